"""What the library knows of a device is made once for each device, not once a process.

Kernels' attributes (the shared memory above 48 KB that a kernel may ask for) and the number of
CTA pairs that fit belong to a device.  The holder of such state is plain C++ and runs here with
numbers in the place of devices; the sources are read for any that is kept otherwise.
"""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_top_route_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"
struct Fit { int err; int pairs; };
std::atomic<int> made[occult::kMaxDevices];
int pairs_of(int device) {
  static occult::PerDevice<Fit> fits;
  return fits.get(device, [&](Fit& f) { ++made[device]; f.pairs += 100 + device; }).pairs;
}
int main() {
  std::vector<std::thread> threads;
  std::atomic<int> wrong{0};
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 3 * occult::kMaxDevices; ++i) {
        const int d = (i * 7 + t) % occult::kMaxDevices;
        if (pairs_of(d) != 100 + d) ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  for (auto& m : made)
    if (m != 1) ++wrong;
  std::printf("wrong %d\n", wrong.load());
  return wrong != 0;
}
"""


def test_every_device_has_a_state_of_its_own(tmp_path):
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and "wrong 0" in out.stdout


def test_no_kernel_attribute_is_set_once_a_process():
    """A function-static flag may guard only what no device owns (the tensor-map encoder)."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for at in re.finditer(r"static std::once_flag", text):
            body = text[at.start():at.start() + 900].split("\n}\n")[0]
            assert "cuTensorMapEncodeTiled" in body and "cudaFunc" not in body and "Occupancy" not in body, name
