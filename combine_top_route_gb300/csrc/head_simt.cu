// Products of the output head for fp32 layers, on the fp32 units: 64 x 64 tiles, 16 deep,
// four by four values a thread, operands through shared memory.  fp32 layers are the
// small ones (the tensor cores have no fp32 of full precision), so the tile is chosen to
// fill the chip on few rows, not for the highest rate: 257 tokens x 1009 x 64 make 80
// tiles.
#include <algorithm>

#include "head.h"
#include "kernels.h"

namespace occult {

namespace {

constexpr int TS = 64, TK = 16;

// acc[i][j] += sum_k a(m0 + ty + 16 i, k) b(n0 + tx + 16 j, k) over [0, K): the loaders
// give an element or 0 outside.  A_K / B_K: the operand's rows run along k (its threads
// then read along k, else along m / n).
template <bool A_K, bool B_K, typename LA, typename LB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], int K, LA a, LB b) {
  __shared__ float sa[TK][TS + 1], sb[TK][TS + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int k0 = 0; k0 < K; k0 += TK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = tid + 256 * i;
      const int ma = A_K ? at / TK : at % TS, ka = A_K ? at % TK : at / TS;
      sa[ka][ma] = a(ma, k0 + ka);
      const int nb = B_K ? at / TK : at % TS, kb = B_K ? at % TK : at / TS;
      sb[kb][nb] = b(nb, k0 + kb);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      float fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { fa[i] = sa[k][ty + 16 * i]; fb[i] = sb[k][tx + 16 * i]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(fa[i], fb[j], acc[i][j]);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256)
head_logits_f32_kernel(const HeadCounts* cnt, const float* __restrict__ x, const float* __restrict__ w,
                       const int32_t* __restrict__ idx, const int32_t* __restrict__ ent_all,
                       float* __restrict__ zt_all, int E, int row0, int piece, int V, int d,
                       float inv_tau, bool two, float* __restrict__ pm, float* __restrict__ ps,
                       float* __restrict__ ps2, int ldp, float* __restrict__ kept, int ld) {
  __shared__ float s_z[TS][TS + 1];
  pdl_wait();
  pdl_trigger();
  const int n = min(cnt->n - row0, piece);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int c0 = blockIdx.x * TS;
  const float NEG = -__int_as_float(0x7f800000);
  for (int m0 = blockIdx.y * TS; m0 < n; m0 += gridDim.y * TS) {
    float acc[4][4] = {};
    if (c0 < V)
      tile_product<true, true>(
          acc, d,
          [&](int m, int k) {
            return m0 + m < n && k < d ? x[static_cast<size_t>(idx[row0 + m0 + m]) * d + k] : 0.f;
          },
          [&](int v, int k) { return c0 + v < V && k < d ? w[static_cast<size_t>(c0 + v) * d + k] : 0.f; });
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ty + 16 * i, c = tx + 16 * j;
        s_z[r][c] = c0 + c < V ? acc[i][j] : NEG;
        if (kept && m0 + r < n && c0 + c < V) kept[static_cast<size_t>(m0 + r) * ld + c0 + c] = acc[i][j];
      }
    __syncthreads();
    // four threads a row
    const int r = tid >> 2, q = tid & 3;
    float m = NEG;
    for (int c = q; c < TS; c += 4) m = fmaxf(m, s_z[r][c]);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float my = (m == NEG ? 0.f : m) * kLog2e;
    float s = 0.f, s2 = 0.f;
    for (int c = q; c < TS; c += 4) {
      const float y = fmaf(s_z[r][c], kLog2e, -my);
      s += exp2f(y);
      if (two) s2 += exp2f(y * inv_tau);
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s2 += __shfl_xor_sync(0xffffffffu, s2, 1);
    s2 += __shfl_xor_sync(0xffffffffu, s2, 2);
    if (q == 0 && m0 + r < n) {
      const size_t at = static_cast<size_t>(blockIdx.x) * ldp + m0 + r;
      pm[at] = m == NEG ? NEG : my;
      ps[at] = s;
      if (two) ps2[at] = s2;
      const int32_t* ent = ent_all + static_cast<size_t>(row0 + m0 + r) * E;
      float* zt = zt_all + static_cast<size_t>(row0 + m0 + r) * E;
      for (int e = 0; e < E && ent[e] < c0 + TS; ++e)
        if (ent[e] >= c0) zt[e] = s_z[r][ent[e] - c0];
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void put(void* out, size_t at, float v, int bf16) {
  if (bf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else static_cast<float*>(out)[at] = v;
}

struct GradArgs {
  const HeadCounts* cnt;
  const float *x, *w, *dz, *dloss;
  const int32_t *idx, *pos;
  int T, row0, piece, V, d, ld, bf16, first, last;
  float coef, coef_kd, coef_z, tau;
  void* out;
  float* acc;
};
__device__ __forceinline__ float common_factor(const GradArgs& a) {
  const HeadScale s = head_scale(a.cnt->n, a.cnt->n_ce, a.cnt->n_kd, a.coef, a.coef_kd, a.coef_z, a.tau);
  return s.unit * (a.dloss ? *a.dloss : 1.f);
}

__global__ void __launch_bounds__(256) head_dx_f32_kernel(const GradArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = min(a.cnt->n - a.row0, a.piece);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int c0 = blockIdx.x * TS;
  const float g = common_factor(a);
  for (int m0 = blockIdx.y * TS; m0 < n; m0 += gridDim.y * TS) {
    float acc[4][4] = {};
    tile_product<true, false>(
        acc, a.V,
        [&](int m, int k) { return m0 + m < n && k < a.V ? a.dz[static_cast<size_t>(m0 + m) * a.ld + k] : 0.f; },
        [&](int c, int k) { return c0 + c < a.d && k < a.V ? a.w[static_cast<size_t>(k) * a.d + c0 + c] : 0.f; });
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = m0 + ty + 16 * i, c = c0 + tx + 16 * j;
        if (r < n && c < a.d) put(a.out, static_cast<size_t>(a.idx[a.row0 + r]) * a.d + c, g * acc[i][j], a.bf16);
      }
  }
  // the rows that no term counts, once
  if (a.first)
    for (int t = blockIdx.y; t < a.T; t += gridDim.y)
      if (a.pos[t] < 0 && threadIdx.x < TS && c0 + threadIdx.x < a.d)
        put(a.out, static_cast<size_t>(t) * a.d + c0 + threadIdx.x, 0.f, a.bf16);
}

__global__ void __launch_bounds__(256) head_dw_f32_kernel(const GradArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = max(0, min(a.cnt->n - a.row0, a.piece));
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int c0 = blockIdx.x * TS;
  const float g = common_factor(a);
  for (int m0 = blockIdx.y * TS; m0 < a.V; m0 += gridDim.y * TS) {
    float acc[4][4] = {};
    tile_product<false, false>(
        acc, n,
        [&](int m, int k) { return m0 + m < a.V && k < n ? a.dz[static_cast<size_t>(k) * a.ld + m0 + m] : 0.f; },
        [&](int c, int k) {
          return c0 + c < a.d && k < n ? a.x[static_cast<size_t>(a.idx[a.row0 + k]) * a.d + c0 + c] : 0.f;
        });
    float* sum = a.bf16 ? a.acc : static_cast<float*>(a.out);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = m0 + ty + 16 * i, c = c0 + tx + 16 * j;
        if (v >= a.V || c >= a.d) continue;
        const size_t at = static_cast<size_t>(v) * a.d + c;
        const float f = g * acc[i][j] + (a.first ? 0.f : sum[at]);
        if (a.bf16 && a.last) put(a.out, at, f, 1);
        else sum[at] = f;
      }
  }
}

GradArgs grad_args(const HeadPlan& p, const HeadArgs& a, int row0) {
  GradArgs g{};
  g.cnt = reinterpret_cast<const HeadCounts*>(a.ws + p.o_cnt);
  g.x = static_cast<const float*>(a.x);
  g.w = static_cast<const float*>(a.w);
  g.dz = reinterpret_cast<const float*>(a.ws + p.o_kept);
  g.dloss = a.dloss;
  g.idx = reinterpret_cast<const int32_t*>(a.ws + p.o_idx);
  g.pos = reinterpret_cast<const int32_t*>(a.ws + p.o_pos);
  g.T = p.T; g.row0 = row0; g.piece = p.piece; g.V = p.V; g.d = p.d; g.ld = p.ld;
  g.bf16 = p.grad_dtype == OCCULT_BF16;
  g.coef = p.coef; g.coef_kd = p.coef_kd; g.coef_z = p.coef_z; g.tau = p.tau;
  return g;
}
unsigned tiles(int n, int most) { return static_cast<unsigned>(std::min((n + TS - 1) / TS, most)); }

}  // namespace

int launch_head_logits_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0) {
  char* ws = a.ws;
  const dim3 grid(p.halves, tiles(std::min(p.piece, p.T - row0), 1024));
  return cuda_status(launch_pdl(
      head_logits_f32_kernel, grid, 256, 0, ctx.stream, reinterpret_cast<const HeadCounts*>(ws + p.o_cnt),
      static_cast<const float*>(a.x), static_cast<const float*>(a.w),
      reinterpret_cast<const int32_t*>(ws + p.o_idx), reinterpret_cast<const int32_t*>(ws + p.o_ent),
      reinterpret_cast<float*>(ws + p.o_zt), p.E, row0, p.piece, p.V, p.d, 1.f / p.tau, p.two,
      reinterpret_cast<float*>(ws + p.o_m), reinterpret_cast<float*>(ws + p.o_s),
      reinterpret_cast<float*>(ws + p.o_s2), p.piece,
      p.step ? reinterpret_cast<float*>(ws + p.o_kept) : nullptr, p.ld));
}

int launch_head_dx_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0) {
  GradArgs g = grad_args(p, a, row0);
  g.out = a.dx;
  g.first = row0 == 0;
  const dim3 grid((p.d + TS - 1) / TS, tiles(std::min(p.piece, p.T - row0), 1024));
  return cuda_status(launch_pdl(head_dx_f32_kernel, grid, 256, 0, ctx.stream, g));
}

int launch_head_dw_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0,
                       bool first, bool last) {
  GradArgs g = grad_args(p, a, row0);
  g.out = a.dw;
  g.acc = reinterpret_cast<float*>(a.ws + p.o_acc);
  g.first = first;
  g.last = last;
  const dim3 grid((p.d + TS - 1) / TS, tiles(p.V, 4096));
  return cuda_status(launch_pdl(head_dw_f32_kernel, grid, 256, 0, ctx.stream, g));
}

}  // namespace occult
