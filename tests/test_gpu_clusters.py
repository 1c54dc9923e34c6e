"""Small problems in one launch of a 16-CTA cluster, and in two launches where the device
has no place for one (a partition of few SMs).  The second is had from a fake of the
runtime's answers: a library loaded before the real one says that no cluster of 16 can be
placed, and refuses to launch one."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

FAKE = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <cuda_runtime_api.h>

int fake_none;      /* say that none can be placed */
int fake_launched;  /* launches of such clusters that were asked for */

static void* real(const char* name) {
  void* h = dlopen("libcudart.so.13", RTLD_LAZY | RTLD_NOLOAD);
  return h ? dlsym(h, name) : 0;
}
static int wide(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension && c->attrs[i].val.clusterDim.x == 16)
      return 1;
  return 0;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  if (fake_none && wide(c)) { *n = 0; return cudaSuccess; }
  cudaError_t (*fn)(int*, const void*, const cudaLaunchConfig_t*) = real("cudaOccupancyMaxActiveClusters");
  return fn(n, f, c);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  if (wide(c)) {
    ++fake_launched;
    if (fake_none) return cudaErrorInvalidClusterSize;
  }
  cudaError_t (*fn)(const cudaLaunchConfig_t*, const void*, void**) = real("cudaLaunchKernelExC");
  return fn(c, f, args);
}
"""

CHILD = r"""
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
none, launched = (ctypes.c_int.in_dll(fake, n) for n in ("fake_none", "fake_launched"))
none.value = int(sys.argv[2])
sys.path[:0] = [sys.argv[3], sys.argv[3] + "/.."]
import combine_top_route_gb300 as occ
import test_gpu_balance as bal
import test_gpu_block_norm as norm
for T, Ne, k in ((4100, 64, 6), (300, 256, 8), (2048, 8, 2)):
    z, ids = bal.case(T, Ne, k, seed=T)
    bal.check(occ, z, ids, 8)
n = launched.value
for T, d, res in ((16, 2048, "bf16"), (257, 64, "f32"), (9, 8256, "f32"), (3, 16384, "bf16")):
    norm.check_backward(occ, norm.Case(T, d, "f32", res, gate="channel", seed=T))
print("launched", n, launched.value - n)
"""


@pytest.mark.parametrize("none", [0, 1])
def test_small_problems_with_and_without_clusters(tmp_path, none):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_top_route_gb300 import build
    build.build()
    src, lib = tmp_path / "fake.c", tmp_path / "fake.so"
    src.write_text(FAKE)
    inc = os.path.join(build._cuda_home(), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", f"-I{inc}", str(src), "-o", str(lib), "-ldl"],
                   check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib), str(none), HERE], text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    _, balance, backward = r.stdout.split()
    if none:
        assert (balance, backward) == ("0", "0")      # not tried where there is no place
    else:
        assert int(balance) >= 2 and int(backward) >= 4
