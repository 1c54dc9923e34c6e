// Products of the output head for fp32 layers, on the fp32 units (the tensor cores have no
// fp32 of full precision): tiles of 64 x 64, four by four values a thread, or of 32 x 32,
// two by two, where the large ones would leave SMs idle; 32 deep, the next step's operands
// on their way to registers while this one is multiplied.  fp32 layers are the small ones:
// 257 tokens x 1009 x 64 make 80 large tiles of the logits and 16 of dw, a step of which
// takes longer to arrive than to multiply: the logits take 7 us and both gradients 12 in
// small tiles, dx over parts of the vocabulary (10, 146 and 26 us in large ones with dx's
// sum in one piece), and the step with its sums and gradients of the logits 32 us, of
// which the products at the fp32 rate would be 1.5: six dependent launches.
#include <algorithm>

#include "head.h"
#include "kernels.h"

namespace occult {

namespace {

constexpr int TK = 32;

// A thread's rows (columns): two next to each other, 32 further on two more.
template <int TS>
__device__ __forceinline__ int spot(int t, int i) { return 2 * t + (i & 1) + 32 * (i >> 1); }

// acc[i][j] += sum_k a(spot(ty, i), k) b(spot(tx, j), k) over [k_lo, k_hi): the loaders give
// an element or 0 outside.  A_K / B_K: the operand's rows run along k (its threads then read
// along k, else along m / n).
template <int TS, bool A_K, bool B_K, typename LA, typename LB>
__device__ __forceinline__ void tile_product(float (&acc)[TS / 16][TS / 16], int k_lo, int k_hi,
                                             LA a, LB b) {
  constexpr int V = TS / 16, PER = TS * TK / 256;
  __shared__ __align__(8) float sa[TK][TS + 2], sb[TK][TS + 2];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float ra[PER], rb[PER];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + 256 * i;
      const int ma = A_K ? at / TK : at % TS, ka = k0 + (A_K ? at % TK : at / TS);
      ra[i] = ka < k_hi ? a(ma, ka) : 0.f;
      const int nb = B_K ? at / TK : at % TS, kb = k0 + (B_K ? at % TK : at / TS);
      rb[i] = kb < k_hi ? b(nb, kb) : 0.f;
    }
  };
  if (k_lo < k_hi) fetch(k_lo);
  for (int k0 = k_lo; k0 < k_hi; k0 += TK) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + 256 * i;
      if (A_K) sa[at % TK][at / TK] = ra[i]; else sa[at / TS][at % TS] = ra[i];
      if (B_K) sb[at % TK][at / TK] = rb[i]; else sb[at / TS][at % TS] = rb[i];
    }
    __syncthreads();
    if (k0 + TK < k_hi) fetch(k0 + TK);
    // (unrolled in part: a small call's time is the code's way in as much as its run)
#pragma unroll 8
    for (int k = 0; k < TK; ++k) {
      float2 fa[V / 2], fb[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        fa[i] = *reinterpret_cast<const float2*>(&sa[k][2 * ty + 32 * i]);
        fb[i] = *reinterpret_cast<const float2*>(&sb[k][2 * tx + 32 * i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
          acc[i][j] = fmaf(i & 1 ? fa[i >> 1].y : fa[i >> 1].x, j & 1 ? fb[j >> 1].y : fb[j >> 1].x, acc[i][j]);
    }
    __syncthreads();
  }
}

struct SimtArgs {
  const HeadCounts* cnt;
  const float *x, *xc, *w, *dloss;   // x, and its compact copy where tokens are left out
  const int32_t* ent;
  float *zt, *pm, *ps, *ps2, *kept;   // kept: the logits, then their gradient
  float *part, *acc;
  void* out;
  int T, row0, piece, V, d, E, ld, halves, splits, two, bf16, first, last;
  float inv_tau, coef, coef_kd, coef_z, tau;
};

// The piece's first compact row of x.
__device__ __forceinline__ const float* x_rows(const SimtArgs& a) {
  return (a.cnt->n == a.T ? a.x : a.xc) + static_cast<size_t>(a.row0) * a.d;
}

// Logits: a tile's columns are a part of its rows' maxima and sums.
template <int TS>
__global__ void __launch_bounds__(256) head_logits_f32_kernel(const SimtArgs a) {
  constexpr int V = TS / 16, Q = 256 / TS;   // Q threads a row afterwards
  __shared__ float s_z[TS][TS + 1];
  pdl_wait();
  pdl_trigger();
  const int n = min(a.cnt->n - a.row0, a.piece);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int c0 = blockIdx.x * TS;
  const float NEG = -__int_as_float(0x7f800000);
  const float* x = x_rows(a);
  for (int m0 = blockIdx.y * TS; m0 < n; m0 += gridDim.y * TS) {
    float acc[V][V] = {};
    tile_product<TS, true, true>(
        acc, 0, c0 < a.V ? a.d : 0,
        [&](int m, int k) { return m0 + m < n ? x[static_cast<size_t>(m0 + m) * a.d + k] : 0.f; },
        [&](int v, int k) { return c0 + v < a.V ? a.w[static_cast<size_t>(c0 + v) * a.d + k] : 0.f; });
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int r = spot<TS>(ty, i), c = spot<TS>(tx, j);
        s_z[r][c] = c0 + c < a.V ? acc[i][j] : NEG;
        if (a.kept && m0 + r < n && c0 + c < a.V) a.kept[static_cast<size_t>(m0 + r) * a.ld + c0 + c] = acc[i][j];
      }
    __syncthreads();
    const int r = tid / Q, q = tid % Q;
    float m = NEG;
    for (int c = q; c < TS; c += Q) m = fmaxf(m, s_z[r][c]);
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float my = (m == NEG ? 0.f : m) * kLog2e;
    float s = 0.f, s2 = 0.f;
    for (int c = q; c < TS; c += Q) {
      const float y = fmaf(s_z[r][c], kLog2e, -my);
      s += exp2f(y);
      if (a.two) s2 += exp2f(y * a.inv_tau);
    }
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (q == 0 && m0 + r < n) {
      const size_t at = static_cast<size_t>(blockIdx.x) * a.piece + m0 + r;
      a.pm[at] = m == NEG ? NEG : my;
      a.ps[at] = s;
      if (a.two) a.ps2[at] = s2;
      const int32_t* ent = a.ent + static_cast<size_t>(a.row0 + m0 + r) * a.E;
      float* zt = a.zt + static_cast<size_t>(a.row0 + m0 + r) * a.E;
      for (int e = 0; e < a.E && ent[e] < c0 + TS; ++e)
        if (ent[e] >= c0) zt[e] = s_z[r][ent[e] - c0];
    }
    __syncthreads();
  }
}

// dx: parts [split][row][d] of the sum over the vocabulary; tile `blk` of its launch's.
template <int TS>
__device__ __forceinline__ void dx_tile(const SimtArgs& a, int blk) {
  constexpr int V = TS / 16;
  const int n = min(a.cnt->n - a.row0, a.piece);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int cols = (a.d + TS - 1) / TS;
  const int sp = blk % a.splits, c0 = blk / a.splits % cols * TS, m0 = blk / a.splits / cols * TS;
  if (m0 >= n) return;
  const int k_lo = static_cast<int>(static_cast<int64_t>(a.V) * sp / a.splits);
  const int k_hi = static_cast<int>(static_cast<int64_t>(a.V) * (sp + 1) / a.splits);
  float acc[V][V] = {};
  tile_product<TS, true, false>(
      acc, k_lo, k_hi,
      [&](int m, int k) { return m0 + m < n ? a.kept[static_cast<size_t>(m0 + m) * a.ld + k] : 0.f; },
      [&](int c, int k) { return c0 + c < a.d ? a.w[static_cast<size_t>(k) * a.d + c0 + c] : 0.f; });
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int r = m0 + spot<TS>(ty, i), c = c0 + spot<TS>(tx, j);
      if (r < n && c < a.d) a.part[(static_cast<size_t>(sp) * a.piece + r) * a.d + c] = acc[i][j];
    }
}

template <int TS>
__device__ __forceinline__ void dw_tile(const SimtArgs& a, int blk) {
  constexpr int V = TS / 16;
  const int n = max(0, min(a.cnt->n - a.row0, a.piece));
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int cols = (a.d + TS - 1) / TS, c0 = blk % cols * TS, m0 = blk / cols * TS;
  const HeadScale sc = head_scale(a.cnt->n, a.cnt->n_ce, a.cnt->n_kd, a.coef, a.coef_kd, a.coef_z, a.tau, 1.f);
  const float g = sc.unit * (a.dloss ? *a.dloss : 1.f);
  const float* x = x_rows(a);
  float acc[V][V] = {};
  tile_product<TS, false, false>(
      acc, 0, n,
      [&](int m, int k) { return m0 + m < a.V ? a.kept[static_cast<size_t>(k) * a.ld + m0 + m] : 0.f; },
      [&](int c, int k) { return c0 + c < a.d ? x[static_cast<size_t>(k) * a.d + c0 + c] : 0.f; });
  float* sum = a.bf16 ? a.acc : static_cast<float*>(a.out);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = m0 + spot<TS>(ty, i), c = c0 + spot<TS>(tx, j);
      if (v >= a.V || c >= a.d) continue;
      const size_t at = static_cast<size_t>(v) * a.d + c;
      const float f = g * acc[i][j] + (a.first ? 0.f : sum[at]);
      if (a.bf16 && a.last) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(f);
      else sum[at] = f;
    }
}

// The first `dx_blocks` blocks take a tile of dx each, the others one of dw.
template <int TX, int TW>
__global__ void __launch_bounds__(256) head_grads_f32_kernel(const SimtArgs a, int dx_blocks) {
  pdl_wait();
  pdl_trigger();
  const int blk = blockIdx.x;
  if (blk < dx_blocks) dx_tile<TX>(a, blk);
  else dw_tile<TW>(a, blk - dx_blocks);
}

SimtArgs simt_args(const HeadPlan& p, const HeadArgs& a, int row0) {
  SimtArgs g{};
  char* ws = a.ws;
  g.cnt = reinterpret_cast<const HeadCounts*>(ws + p.o_cnt);
  g.x = static_cast<const float*>(a.x);
  g.w = static_cast<const float*>(a.w);
  g.dloss = a.dloss;
  g.xc = reinterpret_cast<const float*>(ws + p.o_xc);
  g.T = p.T;
  g.ent = reinterpret_cast<const int32_t*>(ws + p.o_ent);
  g.zt = reinterpret_cast<float*>(ws + p.o_zt);
  g.pm = reinterpret_cast<float*>(ws + p.o_m);
  g.ps = reinterpret_cast<float*>(ws + p.o_s);
  g.ps2 = reinterpret_cast<float*>(ws + p.o_s2);
  g.kept = p.step ? reinterpret_cast<float*>(ws + p.o_kept) : nullptr;
  g.part = reinterpret_cast<float*>(ws + p.o_part);
  g.acc = reinterpret_cast<float*>(ws + p.o_acc);
  g.row0 = row0; g.piece = p.piece; g.V = p.V; g.d = p.d; g.E = p.E; g.ld = p.ld;
  g.halves = p.halves; g.two = p.two;
  g.bf16 = p.grad_dtype == OCCULT_BF16;
  g.inv_tau = 1.f / p.tau; g.tau = p.tau;
  g.coef = p.coef; g.coef_kd = p.coef_kd; g.coef_z = p.coef_z;
  return g;
}
unsigned tiles(int n, int ts, int most) { return static_cast<unsigned>(std::min((n + ts - 1) / ts, most)); }

}  // namespace

int launch_head_logits_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0) {
  const SimtArgs g = simt_args(p, a, row0);
  const int ts = p.bn;   // the plan's parts are this kernel's tiles
  const dim3 grid(p.halves, tiles(std::min(p.piece, p.T - row0), ts, 1024));
  return cuda_status(launch_pdl(ts == 32 ? head_logits_f32_kernel<32> : head_logits_f32_kernel<64>, grid, 256,
                                0, ctx.stream, g));
}

int launch_head_grads_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0,
                          bool first, bool last) {
  SimtArgs g = simt_args(p, a, row0);
  g.out = a.dw;
  g.first = first;
  g.last = last;
  g.splits = head_splits(p, a);
  const auto count = [](int64_t n, int ts) { return (n + ts - 1) / ts; };
  const int tx = head_f32_tile(p.T, p.d), tw = head_f32_tile(p.V, p.d);
  const int64_t dx = a.dx ? count(std::min(p.piece, p.T - row0), tx) * count(p.d, tx) * g.splits : 0;
  const int64_t dw = a.dw ? count(p.V, tw) * count(p.d, tw) : 0;
  if (dx + dw >= (1ll << 31)) return OCCULT_ERR_UNSUPPORTED;
  auto* kern = tx == 32 ? (tw == 32 ? head_grads_f32_kernel<32, 32> : head_grads_f32_kernel<32, 64>)
                        : (tw == 32 ? head_grads_f32_kernel<64, 32> : head_grads_f32_kernel<64, 64>);
  return cuda_status(launch_pdl(kern, static_cast<unsigned>(dx + dw), 256, 0, ctx.stream, g, static_cast<int>(dx)));
}

}  // namespace occult
