// The norms around a block: RMS norm of its output, gate and residual sum, RMS
// norm before the next block (forward), and the gradients (backward).
//
// With one row's sums known everything is elementwise, so both directions are
// bound by the bytes they move: with bf16 rows and an fp32 block output the
// forward moves 10 bytes an element, the backward 16.
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float4 mul4(const float4& a, const float4& b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 scale4(const float4& a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float4 fma4(const float4& a, float b, const float4& c) {
  return make_float4(fmaf(a.x, b, c.x), fmaf(a.y, b, c.y), fmaf(a.z, b, c.z), fmaf(a.w, b, c.w));
}

// Sums of N values over the CTA, in a fixed order; every thread gets them.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*s_red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s_red[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) v[i] += s_red[w][i];
  }
}

// One CTA a row; the fp32 r' of the row waits in shared memory for its mean square.
template <typename R, typename L>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(NormArgs a) {
  extern __shared__ float s_row[];
  __shared__ float s_red[kNormThreads / 32][1];
  pdl_wait();
  pdl_trigger();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = static_cast<size_t>(t) * a.d;
    float rp = 1.f;
    if (w_post) {
      float s[1] = {0.f};
      for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4) {
        const float4 y = ld4(a.y + base + c);
        s[0] += dot4(y, y);
      }
      block_sum<1>(s, s_red);
      rp = rsqrtf(s[0] / a.d + a.eps);
      if (threadIdx.x == 0 && a.rstd_post_out) a.rstd_post_out[t] = rp;
    }
    const float tok = a.gate_kind == OCCULT_GATE_TOKEN ? a.gate[t] : 1.f;
    float q[1] = {0.f};
    for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4) {
      float4 r = ld4(static_cast<const R*>(a.r) + base + c);
      if (a.y) {
        float4 b = scale4(ld4(a.y + base + c), rp);
        if (w_post) b = mul4(b, ld4(w_post + c));
        if (a.gate_kind == OCCULT_GATE_CHANNEL) b = mul4(b, ld4(a.gate + c));
        r = fma4(b, tok, scale4(r, a.res_scale));
        st4(static_cast<R*>(a.r_out) + base + c, r);
      }
      q[0] += dot4(r, r);
      *reinterpret_cast<float4*>(s_row + c) = r;
    }
    if (!w_pre) continue;
    block_sum<1>(q, s_red);
    const float rq = rsqrtf(q[0] / a.d + a.eps);
    if (threadIdx.x == 0 && a.rstd_pre_out) a.rstd_pre_out[t] = rq;
    for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4)
      st4(static_cast<L*>(a.x) + base + c,
          mul4(scale4(*reinterpret_cast<const float4*>(s_row + c), rq), ld4(w_pre + c)));
  }
}

// Backward, one CTA a row.  D is linear in mean(w_pre dx n), so one round of sums
// gives every mean: with g = w_pre dx, D0 = dr_out + rstd_pre g and
// q = gate w_post m,
//   s0 = sum g n,  s1 = sum q D0,  s2 = sum q n
//   c1 = s0 / d,   sum q D = s1 - c1 rstd_pre s2.
// The column sums stay with the threads that own the columns, in shared memory,
// and go to one row of partial sums a CTA.
template <typename R, typename L>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(NormArgs a, float* part) {
  extern __shared__ float s_cols[];  // [2][d]: sum dx n, sum (gate) D m
  __shared__ float s_red[kNormThreads / 32][3];
  pdl_wait();
  pdl_trigger();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  const bool use_y = w_post || a.gate_kind != OCCULT_GATE_NONE;
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL, token = a.gate_kind == OCCULT_GATE_TOKEN;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4) {
    st4(s_cols + c, zero);
    st4(s_cols + a.d + c, zero);
  }
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = static_cast<size_t>(t) * a.d;
    const float rp = w_post ? a.rstd_post[t] : 1.f;
    const float rq = w_pre ? a.rstd_pre[t] : 0.f;
    const float tok = token ? a.gate[t] : 1.f;
    float s[3] = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4) {
      const float4 up = a.dr_out ? ld4(static_cast<const R*>(a.dr_out) + base + c) : zero;
      float4 g = zero, n = zero, q = zero;
      if (w_pre) {
        g = mul4(ld4(a.dx + base + c), ld4(w_pre + c));
        n = scale4(ld4(static_cast<const R*>(a.r) + base + c), rq);
      }
      if (use_y) {
        q = scale4(ld4(a.y + base + c), rp);
        if (w_post) q = mul4(q, ld4(w_post + c));
        if (chan) q = mul4(q, ld4(a.gate + c));
      }
      s[0] += dot4(g, n);
      s[1] += dot4(q, fma4(g, rq, up));
      s[2] += dot4(q, n);
    }
    block_sum<3>(s, s_red);
    const float c1 = s[0] / a.d;
    const float qd = s[1] - c1 * rq * s[2];  // sum q D without the token's gate
    if (token && threadIdx.x == 0) a.dgate[t] = qd;
    const float c2 = tok * qd / a.d;         // mean(u m)
    for (int c = threadIdx.x * 4; c < a.d; c += kNormThreads * 4) {
      float4 D = a.dr_out ? ld4(static_cast<const R*>(a.dr_out) + base + c) : zero;
      if (w_pre) {
        const float4 dx = ld4(a.dx + base + c);
        const float4 n = scale4(ld4(static_cast<const R*>(a.r) + base + c), rq);
        D = fma4(fma4(n, -c1, mul4(dx, ld4(w_pre + c))), rq, D);
        st4(s_cols + c, add4(ld4(s_cols + c), mul4(dx, n)));
      }
      st4(static_cast<R*>(a.dr) + base + c, scale4(D, a.y ? a.res_scale : 1.f));
      if (!a.y) continue;
      float4 u = scale4(D, tok);
      float4 m = zero;
      if (use_y) {
        m = scale4(ld4(a.y + base + c), rp);
        st4(s_cols + a.d + c, add4(ld4(s_cols + a.d + c), mul4(chan ? D : u, m)));
      }
      u = mul4(u, chan ? ld4(a.gate + c) : one);
      if (w_post) u = scale4(fma4(m, -c2, mul4(u, ld4(w_post + c))), rp);
      st4(static_cast<L*>(a.dy) + base + c, u);
    }
  }
  __syncthreads();  // the copy below goes over both sums in one stride
  float* row = part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
  for (int c = threadIdx.x * 4; c < 2 * a.d; c += kNormThreads * 4) st4(row + c, ld4(s_cols + c));
}

// Adds the CTAs' partial rows in order and turns the second sum into dw_post and a
// channel gate's gradient.
template <typename L>
__global__ void __launch_bounds__(kNormThreads)
norm_bwd_cols_kernel(NormArgs a, const float* __restrict__ part, int n_part) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= 2 * a.d) return;
  float s = 0.f;
  for (int p = 0; p < n_part; ++p) s += part[static_cast<size_t>(p) * 2 * a.d + c];
  if (c < a.d) {
    if (a.dw_pre) a.dw_pre[c] = s;
    return;
  }
  const int j = c - a.d;
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL;
  if (a.dw_post) a.dw_post[j] = chan ? s * a.gate[j] : s;
  if (chan) a.dgate[j] = a.w_post ? s * to_f32(static_cast<const L*>(a.w_post)[j]) : s;
}

template <typename K>
int allow_smem(K kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return OCCULT_OK;
  return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(bytes)));
}

template <typename R, typename L>
int fwd(const LaunchCtx& ctx, const NormArgs& a) {
  const size_t smem = static_cast<size_t>(a.d) * sizeof(float);
  const int rc = allow_smem(norm_fwd_kernel<R, L>, smem);
  if (rc) return rc;
  const int grid = a.T < ctx.num_sms * 8 ? a.T : ctx.num_sms * 8;
  return cuda_status(launch_pdl(norm_fwd_kernel<R, L>, grid, kNormThreads, smem, ctx.stream, a));
}

template <typename R, typename L>
int bwd(const LaunchCtx& ctx, const NormArgs& a, float* part) {
  const size_t smem = 2 * static_cast<size_t>(a.d) * sizeof(float);
  int rc = allow_smem(norm_bwd_kernel<R, L>, smem);
  if (rc) return rc;
  const int grid = norm_bwd_parts(a.T);
  rc = cuda_status(launch_pdl(norm_bwd_kernel<R, L>, grid, kNormThreads, smem, ctx.stream, a, part));
  if (rc || !(a.dw_pre || a.dw_post || a.gate_kind == OCCULT_GATE_CHANNEL)) return rc;
  return cuda_status(launch_pdl(norm_bwd_cols_kernel<L>, (2 * a.d + kNormThreads - 1) / kNormThreads,
                                kNormThreads, 0, ctx.stream, a, part, grid));
}

}  // namespace

int norm_bwd_parts(int T) { return T < kNormMaxParts ? T : kNormMaxParts; }

size_t block_norm_bwd_ws_bytes(const occult_desc_t& ds) {
  return static_cast<size_t>(norm_bwd_parts(ds.T)) * 2 * ds.d * sizeof(float);
}

int launch_block_norm(const LaunchCtx& ctx, const NormArgs& a, int res_dtype, int dtype) {
  if (res_dtype == OCCULT_BF16)
    return dtype == OCCULT_BF16 ? fwd<__nv_bfloat16, __nv_bfloat16>(ctx, a)
                                : fwd<__nv_bfloat16, float>(ctx, a);
  return dtype == OCCULT_BF16 ? fwd<float, __nv_bfloat16>(ctx, a) : fwd<float, float>(ctx, a);
}

int launch_block_norm_bwd(const LaunchCtx& ctx, const NormArgs& a, int res_dtype, int dtype,
                          void* ws) {
  float* part = static_cast<float*>(ws);
  if (res_dtype == OCCULT_BF16)
    return dtype == OCCULT_BF16 ? bwd<__nv_bfloat16, __nv_bfloat16>(ctx, a, part)
                                : bwd<__nv_bfloat16, float>(ctx, a, part);
  return dtype == OCCULT_BF16 ? bwd<float, __nv_bfloat16>(ctx, a, part)
                              : bwd<float, float>(ctx, a, part);
}

}  // namespace occult
