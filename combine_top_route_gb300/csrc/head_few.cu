// The output head's loss for up to four tokens (scoring while decoding), in one pass over
// the weights.  Their stream is all that counts (one token x 2048 x 50304: 206 MB, 30 us
// at the copy rate), and the fp32 units keep up with it: no tensor core tile would be
// more than a thirty-second full.
//
// A block has a run of vocabulary rows, which come in as bulk copies, a row each, through a
// ring of 64 KB stages in shared memory (one warp asks for them, from before the launch
// ahead is done: nothing ahead of that one is still running).  The case above takes 40 us
// with its rows' launch, as long as any read of 206 MB here (a plain sum of as many bytes
// 40 us; of 4.3 GB at 6.6 TB/s); four rows a warp straight to registers took 47 us, a
// stage in one copy 41, a ring for each warp 41.  A warp takes two rows of a stage at a
// time, a lane 16 bytes of each per step; products are added in fp32 in 32 sums, joined over
// the lanes, so that a warp knows its rows' logits and keeps a maximum and a sum of powers
// of two for each token.  The entries' logits are products of their own, a warp each, so
// that no row has to be looked up.  The last block to arrive joins the blocks' sums and
// finishes the losses.
#include <algorithm>

#include "head.h"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kWarps = 16;                   // and one that asks for the copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kFewBlocks = 152;              // one an SM at most
constexpr int kMaxStages = 4;
constexpr int kRingBytes = 216 * 1024;       // ring and x

struct FewTail {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort_flag;
  int last;
};

struct FewArgs {
  HeadCounts* cnt;
  HeadLossOut out;
  const __nv_bfloat16 *x, *w;
  const int32_t* idx;
  const uint8_t* flag;
  float *zt, *pm, *ps, *ps2;   // parts [block][ldp]
  int V, d, ldp, rows, stages;
  float inv_tau;
  int* dev_err;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Sums of two rows' products with NT tokens, known to all lanes.
template <int NT, typename LOAD>
__device__ __forceinline__ void two_rows(float (&acc)[2][NT], LOAD load, const __nv_bfloat16* xs, int d) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = 0.f;
#pragma unroll 4
  for (int c = (threadIdx.x & 31) * 8; c < d; c += 256) {
    float f[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) unpack16(load(i, c), f[i], __nv_bfloat16());
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float g[8];
      unpack16(*reinterpret_cast<const uint4*>(xs + t * d + c), g, __nv_bfloat16());
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][t] = fmaf(f[i][j], g[j], acc[i][t]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = warp_sum(acc[i][t]);
}

template <int NT, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) head_few_kernel(const FewArgs a) {
  extern __shared__ __align__(128) uint8_t few_smem[];
  __shared__ FewTail tail;
  __shared__ float s_m[kWarps][NT], s_s[kWarps][NT], s_s2[kWarps][NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row_bytes = a.d * 2, stage_bytes = a.rows * row_bytes;
  uint8_t* ring = few_smem;
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(few_smem + a.stages * stage_bytes);
  const int v0 = static_cast<int>(static_cast<int64_t>(a.V) * blockIdx.x / gridDim.x);
  const int v1 = static_cast<int>(static_cast<int64_t>(a.V) * (blockIdx.x + 1) / gridDim.x);
  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&tail.full[s], 1);
      mbar_init(&tail.empty[s], kWarps);
    }
    tail.abort_flag = 0;
    tail.last = 0;
    mbar_fence_init();
  }
  __syncthreads();
  volatile int* abort_flag = &tail.abort_flag;
  const float NEG = -__int_as_float(0x7f800000);
  bool ok = true;
  if (warp == kWarps) {
    // ---- the ring's copies (the weights are no output of the launch ahead) ----
    int stage = 0;
    uint32_t phase = 0;
    for (int v = v0; v < v1; v += a.rows) {
      if (!mbar_wait(&tail.empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
      const int rows = min(a.rows, v1 - v);
      if (lane == 0) mbar_arrive_expect_tx(&tail.full[stage], static_cast<uint32_t>(rows) * row_bytes);
      __syncwarp();
      for (int r = lane; r < rows; r += 32)
        bulk_load(ring + stage * stage_bytes + r * row_bytes, a.w + static_cast<size_t>(v + r) * a.d, row_bytes,
                  &tail.full[stage]);
      __syncwarp();
      if (++stage == a.stages) { stage = 0; phase ^= 1u; }
    }
    pdl_wait();
    pdl_trigger();
  } else {
    pdl_wait();
    pdl_trigger();
    const int n = a.cnt->n;
    for (int i = tid * 8; i < NT * a.d; i += kWarps * 32 * 8) {
      const int t = i / a.d;
      *reinterpret_cast<uint4*>(xs + i) =
          t < n ? *reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(a.idx[t]) * a.d + (i - t * a.d))
                : make_uint4(0, 0, 0, 0);
    }
    asm volatile("bar.sync 1, %0;" :: "n"(kWarps * 32) : "memory");   // these warps alone
    float acc[2][NT];
    const int E = a.out.E;
    for (int i = blockIdx.x * kWarps + warp; i < n * E; i += gridDim.x * kWarps) {
      const int id = a.out.ent[i], t = i / E;
      if (id == kHeadNoEntry) continue;
      const __nv_bfloat16* row = a.w + static_cast<size_t>(id) * a.d;
      two_rows<NT>(acc, [&](int, int c) { return ld_nc_v4(row + c); }, xs, a.d);
      float z = acc[0][0];
#pragma unroll
      for (int u = 1; u < NT; ++u) z = t == u ? acc[0][u] : z;
      if (lane == 0) a.zt[i] = z;
    }
    float m[NT], s[NT], s2[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) { m[t] = NEG; s[t] = 0.f; s2[t] = 0.f; }
    int stage = 0;
    uint32_t phase = 0;
    for (int v = v0; v < v1; v += a.rows) {
      if (!mbar_wait(&tail.full[stage], phase, abort_flag)) { ok = false; break; }
      const int rows = min(a.rows, v1 - v);
      const uint8_t* base = ring + stage * stage_bytes;
      for (int r = 2 * warp; r < rows; r += 2 * kWarps) {
        const bool both = r + 1 < rows;   // (else the row is read twice and counts once)
        const uint8_t* p = base + static_cast<size_t>(r) * row_bytes;
        two_rows<NT>(acc, [&](int i, int c) {
          return *reinterpret_cast<const uint4*>(p + (i && both ? row_bytes : 0) + c * 2);
        }, xs, a.d);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float z1 = both ? acc[1][t] : NEG;
          const float hi = fmaxf(m[t], fmaxf(acc[0][t], z1) * kLog2e), to = hi == NEG ? 0.f : hi;
          const float y0 = over_top(acc[0][t], to), y1 = over_top(z1, to);
          s[t] = s[t] * ex2(m[t] - to) + (ex2(y0) + ex2(y1));
          if (TWO)
            s2[t] = s2[t] * ex2((m[t] - to) * a.inv_tau) + (ex2(y0 * a.inv_tau) + ex2(y1 * a.inv_tau));
          m[t] = hi;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail.empty[stage]);
      if (++stage == a.stages) { stage = 0; phase ^= 1u; }
    }
    if (lane == 0)
#pragma unroll
      for (int t = 0; t < NT; ++t) { s_m[warp][t] = m[t]; s_s[warp][t] = s[t]; s_s2[warp][t] = s2[t]; }
  }
  if (!ok) {
    if (lane == 0) latch_error(a.dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
    *abort_flag = 1;
  }
  __syncthreads();
  const int n = a.cnt->n;
  if (tid < NT && tid < n) {
    float hi = NEG, p = 0.f, p2 = 0.f;
    for (int i = 0; i < kWarps; ++i) hi = fmaxf(hi, s_m[i][tid]);
    const float to = hi == NEG ? 0.f : hi;
    for (int i = 0; i < kWarps; ++i) {
      p += s_s[i][tid] * ex2(s_m[i][tid] - to);
      if (TWO) p2 += s_s2[i][tid] * ex2((s_m[i][tid] - to) * a.inv_tau);
    }
    const size_t at = static_cast<size_t>(blockIdx.x) * a.ldp + tid;
    a.pm[at] = hi;
    a.ps[at] = p;
    if (TWO) a.ps2[at] = p2;
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) tail.last = atomicAdd(&a.cnt->ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!tail.last || warp != 0) return;
  // ---- the last block's first warp: the blocks' sums of every row, and the losses ----
  __threadfence();
  RowSums sum{0.f, 0.f, 0.f};
  for (int r = 0; r < n; ++r) {
    // (all of a lane's loads at once: one after the other they would take 3 us)
    float vm[kFewBlocks / 32 + 1], vs[kFewBlocks / 32 + 1], vt[kFewBlocks / 32 + 1];
    float hi = NEG, p = 0.f, p2 = 0.f;
#pragma unroll
    for (int i = 0; i <= kFewBlocks / 32; ++i) {
      const int b = lane + 32 * i;
      const size_t at = static_cast<size_t>(b) * a.ldp + r;
      const bool there = b < static_cast<int>(gridDim.x);
      vm[i] = there ? __ldcg(a.pm + at) : NEG;
      vs[i] = there ? __ldcg(a.ps + at) : 0.f;
      vt[i] = TWO && there ? __ldcg(a.ps2 + at) : 0.f;
    }
#pragma unroll
    for (int i = 0; i <= kFewBlocks / 32; ++i) hi = fmaxf(hi, vm[i]);
    const float my = hi == NEG ? 0.f : hi;
#pragma unroll
    for (int i = 0; i <= kFewBlocks / 32; ++i) {
      p = fmaf(vs[i], ex2(vm[i] - my), p);
      if (TWO) p2 = fmaf(vt[i], ex2((vm[i] - my) * a.inv_tau), p2);
    }
    const float top = warp_max(hi), to = top == NEG ? 0.f : top;
    const float l1 = log2f(warp_sum(p * ex2(hi - to)));
    const float l2 = TWO ? log2f(warp_sum(p2 * ex2((hi - to) * a.inv_tau))) : l1;
    row_losses(a.out, r, a.flag[r], a.idx[r], to, l1, l2, a.inv_tau, sum);
  }
  if (lane == 0) mean_losses(a.out, *a.cnt, sum.ce, sum.kd, sum.z);
}

template <int NT, bool TWO>
int launch_few(const LaunchCtx& ctx, const HeadPlan& p, FewArgs g) {
  auto kern = head_few_kernel<NT, TWO>;
  static PerDevice<cudaError_t> fits;
  if (fits.get(ctx.device, [&](cudaError_t& e) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
      }) != cudaSuccess)
    return OCCULT_ERR_CUDA;
  // stages of about 64 KB, three of them, beside x (d <= 16384: at most 128 KB)
  const int row_bytes = p.d * 2, room = kRingBytes - NT * row_bytes;
  g.rows = std::max(1, std::min(64 * 1024, room / 3) / row_bytes);
  g.stages = std::min(kMaxStages, room / (g.rows * row_bytes));
  if (g.stages < 1) return OCCULT_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(g.stages) * g.rows * row_bytes + NT * row_bytes;
  return cuda_status(launch_pdl(kern, p.halves, kThreads, smem, ctx.stream, g));
}

}  // namespace

// One block an SM, of no less than 64 KB of weights (or a row).
int head_few_blocks(int V, int d) {
  const int64_t bytes = static_cast<int64_t>(V) * d * 2;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kFewBlocks, bytes / (64 * 1024), V})));
}

int launch_head_few(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a) {
  FewArgs g{};
  char* ws = a.ws;
  g.cnt = reinterpret_cast<HeadCounts*>(ws + p.o_cnt);
  g.out = head_loss_out(p, a);
  g.x = static_cast<const __nv_bfloat16*>(a.x);
  g.w = static_cast<const __nv_bfloat16*>(a.w);
  g.idx = reinterpret_cast<const int32_t*>(ws + p.o_idx);
  g.flag = reinterpret_cast<const uint8_t*>(ws + p.o_flag);
  g.zt = reinterpret_cast<float*>(ws + p.o_zt);
  g.pm = reinterpret_cast<float*>(ws + p.o_m);
  g.ps = reinterpret_cast<float*>(ws + p.o_s);
  g.ps2 = reinterpret_cast<float*>(ws + p.o_s2);
  g.V = p.V; g.d = p.d; g.ldp = p.piece; g.inv_tau = 1.f / p.tau;
  g.dev_err = ctx.dev_err;
#define OCCULT_FEW(NT) (p.two ? launch_few<NT, true>(ctx, p, g) : launch_few<NT, false>(ctx, p, g))
  return p.T == 1 ? OCCULT_FEW(1) : p.T == 2 ? OCCULT_FEW(2) : p.T == 3 ? OCCULT_FEW(3) : OCCULT_FEW(4);
#undef OCCULT_FEW
}

}  // namespace occult
