// AdamW over many tensors in one launch, with fp32 states or 8-bit ones.
//
// The 8-bit states are floats of their own: magnitudes x > 0 of a block of 256
// elements are cut to MANT mantissa bits (m: 3 and a sign, sqrt(v): 4) by adding
// a draw to the fp32 word below the cut and truncating, so that the expectation
// is x; the word's leading bits less those of 2^(E - 15), with E the exponent of
// the block's largest (rounded up) value, are the code, 0 .. 16 * 2^MANT - 1.
// All of it is integer arithmetic on the fp32 words, and every code stands for a
// value that bf16 holds exactly.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kBlock = OCCULT_STATE_BLOCK;       // elements of a warp's step
constexpr int kChunk = kAdamWarps * kBlock * 4;  // elements of a CTA
constexpr int kMaxTensors = 256;                 // of one launch

enum : int { KIND_F32 = 0, KIND_MASTER = 1, KIND_BF16 = 2 };

struct Tensor {
  void* param;
  float* master;
  const float* grad;
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  int64_t n, first;
  int kind;
};
struct AdamTable {
  float b1, c1, b2, c2;      // beta, 1 - beta
  float keep, rate;          // 1 - lr wd, lr / (1 - beta1^t)
  float inv_root, eps;       // (1 - beta2^t)^(-1/2)
  uint32_t key;
  const float* grad_scale;
  int n;
  int chunk0[kMaxTensors + 1];  // first CTA of every tensor
  Tensor t[kMaxTensors];
};

constexpr uint32_t kMul1 = 0xBB67AE85u, kMul2 = 0x3C6EF373u;  // frac(sqrt 3), frac(sqrt 5), odd

// A 32-bit hash (multiply, fold the high half in, twice).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x *= kMul1;
  x ^= x >> 15;
  x *= kMul2;
  return x ^ (x >> 16);
}

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

// exponent byte of a block whose largest magnitude has the bits `top`
template <int MANT>
__device__ __forceinline__ uint32_t block_exp(uint32_t top) {
  constexpr uint32_t cut = 23 - MANT;
  if (top >= 0x7f800000u) return 255u;
  const uint32_t e = (top + ((1u << cut) - 1)) >> 23;
  return e < 16u ? 16u : e;
}
template <int MANT>
__device__ __forceinline__ uint32_t encode(uint32_t bits, uint32_t draw16, uint32_t exp) {
  constexpr uint32_t cut = 23 - MANT;
  const uint32_t mag = bits & 0x7fffffffu;
  int k = static_cast<int>((mag + (draw16 << (cut - 16))) >> cut) -
          ((static_cast<int>(exp) - 15) << MANT);
  k = min(max(k, 0), (16 << MANT) - 1);
  if (MANT == 3) return k ? static_cast<uint32_t>(k) | ((bits >> 24) & 0x80u) : 0u;
  return (k == 0 && mag != 0) ? 1u : static_cast<uint32_t>(k);
}
template <int MANT>
__device__ __forceinline__ float decode(uint32_t code, uint32_t exp) {
  constexpr uint32_t cut = 23 - MANT;
  const uint32_t mag = code & ((16u << MANT) - 1);
  if (exp == 255u) return __int_as_float(0x7fffffff);
  if (mag == 0) return 0.f;
  uint32_t bits = (mag + ((exp - 15u) << MANT)) << cut;
  if (MANT == 3) bits |= (code & 0x80u) << 24;
  return __uint_as_float(bits);
}

// bf16 by a draw: the low half of the word carries into the high one
__device__ __forceinline__ uint32_t bf16_by_draw(float w, uint32_t draw16) {
  const uint32_t bits = __float_as_uint(w);
  if ((bits & 0x7f800000u) == 0x7f800000u)
    return __bfloat16_as_ushort(__float2bfloat16_rn(w));
  return (bits + draw16) >> 16;
}

// Four consecutive elements of a tensor, the first `live` of them in range.
__device__ __forceinline__ void load4(const float* p, int live, float (&f)[4]) {
  if (live == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < live ? p[j] : 0.f;
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int live, float (&f)[4]) {
  if (live == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < live ? to_f32(p[j]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int live) {
  if (live == 4) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < live) w |= static_cast<uint32_t>(p[j]) << (8 * j);
  return w;
}
__device__ __forceinline__ void store4(float* p, int live, const float (&f)[4]) {
  if (live == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p[j] = f[j];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, int live, const uint32_t (&h)[4]) {
  if (live == 4) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p[j] = static_cast<uint16_t>(h[j]);
  }
}
__device__ __forceinline__ void store4(uint8_t* p, int live, const uint32_t (&c)[4]) {
  if (live == 4) {
    *reinterpret_cast<uint32_t*>(p) =
        __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p[j] = static_cast<uint8_t>(c[j]);
  }
}

// One block of 256 elements by one warp: lane l has elements 4l .. 4l+3 of both
// halves, so that every access of the warp is to consecutive words.  Products are
// rounded before they are summed (no fused multiply-add in the moments and the
// root, which a code is cut from): the same bits as the formula term by term.
template <int BITS, int KIND>
__device__ __forceinline__ void step_block(const AdamTable& a, const Tensor& T, int64_t blk,
                                           float gs) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = blk * kBlock + lane * 4;
  int live[2];
  float g[2][4], w[2][4], m[2][4], v[2][4], s[2][4];
  uint32_t cm[2], cv[2], em = 0, ev = 0;
  if (BITS == 8) { em = T.m_exp[blk]; ev = T.v_exp[blk]; }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b0 + h * 128, left = T.n - i;
    live[h] = left >= 4 ? 4 : (left > 0 ? static_cast<int>(left) : 0);
    load4(T.grad + i, live[h], g[h]);
    if (KIND == KIND_MASTER) load4(static_cast<const float*>(T.master) + i, live[h], w[h]);
    else if (KIND == KIND_F32) load4(static_cast<const float*>(T.param) + i, live[h], w[h]);
    else load4(static_cast<const __nv_bfloat16*>(T.param) + i, live[h], w[h]);
    if (BITS == 32) {
      load4(static_cast<const float*>(T.m) + i, live[h], m[h]);
      load4(static_cast<const float*>(T.v) + i, live[h], v[h]);
    } else {
      cm[h] = load4(static_cast<const uint8_t*>(T.m) + i, live[h]);
      cv[h] = load4(static_cast<const uint8_t*>(T.v) + i, live[h]);
    }
  }
  uint32_t top_m = 0, top_v = 0, draw[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b0 + h * 128;
    float out[4];
    uint32_t half[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BITS == 8) {
        m[h][j] = decode<3>((cm[h] >> (8 * j)) & 0xffu, em);
        const float r = decode<4>((cv[h] >> (8 * j)) & 0xffu, ev);
        v[h][j] = r * r;
      }
      if (BITS == 8 || KIND == KIND_BF16)
        draw[h][j] = mix(static_cast<uint32_t>(T.first + i) + j + a.key);
      const float gj = gs * g[h][j];
      m[h][j] = __fadd_rn(__fmul_rn(a.b1, m[h][j]), __fmul_rn(a.c1, gj));
      v[h][j] = __fadd_rn(__fmul_rn(a.b2, v[h][j]), __fmul_rn(__fmul_rn(a.c2, gj), gj));
      s[h][j] = sqrtf(v[h][j]);
      out[j] = fmaf(-a.rate, __fdividef(m[h][j], fmaf(s[h][j], a.inv_root, a.eps)), w[h][j] * a.keep);
      top_m = max(top_m, __float_as_uint(m[h][j]) & 0x7fffffffu);
      top_v = max(top_v, __float_as_uint(s[h][j]) & 0x7fffffffu);
      if (KIND == KIND_MASTER) half[j] = __bfloat16_as_ushort(__float2bfloat16_rn(out[j]));
      if (KIND == KIND_BF16) half[j] = bf16_by_draw(out[j], (draw[h][j] * kMul1) >> 16);
    }
    if (BITS == 32) {
      store4(static_cast<float*>(T.m) + i, live[h], m[h]);
      store4(static_cast<float*>(T.v) + i, live[h], v[h]);
    }
    if (KIND == KIND_F32) store4(static_cast<float*>(T.param) + i, live[h], out);
    if (KIND == KIND_MASTER) store4(T.master + i, live[h], out);
    if (KIND != KIND_F32) store4(static_cast<uint16_t*>(T.param) + i, live[h], half);
  }
  if (BITS == 8) {
    // (elements out of range are zeros here: they raise no exponent)
    const uint32_t new_m = block_exp<3>(warp_max_u32(top_m));
    const uint32_t new_v = block_exp<4>(warp_max_u32(top_v));
    if (lane == 0) {
      T.m_exp[blk] = static_cast<uint8_t>(new_m);
      T.v_exp[blk] = static_cast<uint8_t>(new_v);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t km[4], kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        km[j] = encode<3>(__float_as_uint(m[h][j]), draw[h][j] & 0xffffu, new_m);
        kv[j] = encode<4>(__float_as_uint(s[h][j]), draw[h][j] >> 16, new_v);
      }
      store4(static_cast<uint8_t*>(T.m) + b0 + h * 128, live[h], km);
      store4(static_cast<uint8_t*>(T.v) + b0 + h * 128, live[h], kv);
    }
  }
}

template <int BITS>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable a) {
  pdl_wait();
  pdl_trigger();
  // the tensor of this CTA: the last whose first CTA is not after it
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.chunk0[mid] <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  const Tensor& T = a.t[lo];
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t blk0 = static_cast<int64_t>(blockIdx.x - a.chunk0[lo]) * (kChunk / kBlock);
  const int64_t n_blk = (T.n + kBlock - 1) / kBlock;
  for (int u = threadIdx.x >> 5; u < kChunk / kBlock; u += kAdamWarps) {
    const int64_t blk = blk0 + u;
    if (blk >= n_blk) break;
    if (T.kind == KIND_F32) step_block<BITS, KIND_F32>(a, T, blk, gs);
    else if (T.kind == KIND_MASTER) step_block<BITS, KIND_MASTER>(a, T, blk, gs);
    else step_block<BITS, KIND_BF16>(a, T, blk, gs);
  }
}

// The values of 8-bit states: a thread turns 8 codes into 16 bytes.
template <int MANT>
__global__ void __launch_bounds__(256)
adamw_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n,
                  __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const uint32_t e = exps[i / kBlock];
  if (i + 8 <= n) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + i);
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = decode<MANT>((c.x >> (8 * j)) & 0xffu, e);
      f[4 + j] = decode<MANT>((c.y >> (8 * j)) & 0xffu, e);
    }
    st_v4(out + i, pack16(f, __nv_bfloat16()));
  } else {
    for (int64_t j = i; j < n; ++j) out[j] = __float2bfloat16_rn(decode<MANT>(codes[j], e));
  }
}

}  // namespace

int launch_adamw(const LaunchCtx& ctx, const occult_adamw_t& o, const occult_param_t* params,
                 int n_params) {
  static_assert(sizeof(AdamTable) <= 32764, "kernel parameters");
  AdamTable a;
  a.b1 = static_cast<float>(o.beta1);
  a.c1 = static_cast<float>(1.0 - o.beta1);
  a.b2 = static_cast<float>(o.beta2);
  a.c2 = static_cast<float>(1.0 - o.beta2);
  a.keep = static_cast<float>(1.0 - o.lr * o.weight_decay);
  a.rate = static_cast<float>(o.lr / (1.0 - pow(o.beta1, o.step)));
  a.inv_root = static_cast<float>(1.0 / sqrt(1.0 - pow(o.beta2, o.step)));
  a.eps = static_cast<float>(o.eps);
  a.key = mix(o.seed + mix(static_cast<uint32_t>(o.step)));
  a.grad_scale = o.grad_scale;
  int i = 0;
  while (i < n_params) {
    a.n = 0;
    int64_t chunks = 0;
    for (; i < n_params && a.n < kMaxTensors; ++i) {
      const occult_param_t& p = params[i];
      if (p.n == 0) continue;
      const int64_t c = (p.n + kChunk - 1) / kChunk;
      if (chunks + c > 0x7fffffff) {
        if (a.n > 0) break;
        return OCCULT_ERR_UNSUPPORTED;
      }
      Tensor& t = a.t[a.n];
      t.param = p.param; t.master = p.master; t.grad = p.grad; t.m = p.m; t.v = p.v;
      t.m_exp = p.m_exp; t.v_exp = p.v_exp; t.n = p.n; t.first = p.first;
      t.kind = p.dtype == OCCULT_F32 ? KIND_F32 : p.master ? KIND_MASTER : KIND_BF16;
      a.chunk0[a.n++] = static_cast<int>(chunks);
      chunks += c;
    }
    if (a.n == 0) break;
    const cudaError_t e =
        o.state_bits == 32
            ? launch_pdl(adamw_kernel<32>, static_cast<unsigned>(chunks), kAdamThreads, 0, ctx.stream, a)
            : launch_pdl(adamw_kernel<8>, static_cast<unsigned>(chunks), kAdamThreads, 0, ctx.stream, a);
    if (e != cudaSuccess) return OCCULT_ERR_CUDA;
  }
  return OCCULT_OK;
}

int launch_adamw_read(const LaunchCtx& ctx, const uint8_t* codes, const uint8_t* exps, int64_t n,
                      int which, void* out) {
  const int64_t need = (n + 2047) / 2048;
  if (need > 0x7fffffff) return OCCULT_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(need);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  return cuda_status(
      which == OCCULT_STATE_M
          ? launch_pdl(adamw_read_kernel<3>, grid, 256, 0, ctx.stream, codes, exps, n, o)
          : launch_pdl(adamw_read_kernel<4>, grid, 256, 0, ctx.stream, codes, exps, n, o));
}

}  // namespace occult
