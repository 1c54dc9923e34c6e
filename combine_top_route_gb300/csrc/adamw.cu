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

// The elements i0 .. i0+3 of a tensor (as many as `live`).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int live, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = j < live ? to_f32(p[j]) : 0.f;
}
template <>
__device__ __forceinline__ void load4<float>(const float* p, int live, float (&f)[4]) {
  if (live == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < live ? p[j] : 0.f;
  }
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

// One block of 256 elements by one warp: lane l has elements 4l .. 4l+3 of both
// halves, so that every access of the warp is to consecutive words.
template <int BITS, int KIND>
__device__ __forceinline__ void step_block(const AdamTable& a, const Tensor& T, int64_t blk,
                                           float gs) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = blk * kBlock;
  uint32_t em = 0, ev = 0;
  if (BITS == 8) { em = T.m_exp[blk]; ev = T.v_exp[blk]; }
  float m[2][4], s[2][4];
  uint32_t top_m = 0, top_v = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b0 + h * 128 + lane * 4;
    const int64_t left = T.n - i;
    const int live = left >= 4 ? 4 : (left > 0 ? static_cast<int>(left) : 0);
    float g[4], w[4], v[4];
    load4(T.grad + i, live, g);
    if (KIND == KIND_MASTER) load4(static_cast<const float*>(T.master) + i, live, w);
    else if (KIND == KIND_F32) load4(static_cast<const float*>(T.param) + i, live, w);
    else load4(static_cast<const __nv_bfloat16*>(T.param) + i, live, w);
    if (BITS == 32) {
      load4(static_cast<const float*>(T.m) + i, live, m[h]);
      load4(static_cast<const float*>(T.v) + i, live, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[h][j] = decode<3>(j < live ? static_cast<const uint8_t*>(T.m)[i + j] : 0u, em);
        const float r = decode<4>(j < live ? static_cast<const uint8_t*>(T.v)[i + j] : 0u, ev);
        v[j] = r * r;
      }
    }
    float out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float gj = gs * g[j];
      m[h][j] = fmaf(a.b1, m[h][j], a.c1 * gj);
      v[j] = fmaf(a.b2, v[j], a.c2 * gj * gj);
      s[h][j] = sqrtf(v[j]);
      out[j] = fmaf(-a.rate, m[h][j] / fmaf(s[h][j], a.inv_root, a.eps), w[j] * a.keep);
      if (j < live) {
        top_m = max(top_m, __float_as_uint(m[h][j]) & 0x7fffffffu);
        top_v = max(top_v, __float_as_uint(s[h][j]) & 0x7fffffffu);
      }
    }
    if (BITS == 32) {
      store4(static_cast<float*>(T.m) + i, live, m[h]);
      store4(static_cast<float*>(T.v) + i, live, v);
    }
    if (KIND == KIND_F32) store4(static_cast<float*>(T.param) + i, live, out);
    if (KIND == KIND_MASTER) store4(T.master + i, live, out);
    if (KIND != KIND_F32) {
      uint16_t* p = static_cast<uint16_t*>(T.param) + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= live) continue;
        if (KIND == KIND_MASTER) {
          p[j] = __bfloat16_as_ushort(__float2bfloat16_rn(out[j]));
        } else {
          const uint32_t h32 = mix(static_cast<uint32_t>(T.first + i + j) + a.key);
          p[j] = static_cast<uint16_t>(bf16_by_draw(out[j], (h32 * kMul1) >> 16));
        }
      }
    }
  }
  if (BITS == 8) {
    const uint32_t new_m = block_exp<3>(warp_max_u32(top_m));
    const uint32_t new_v = block_exp<4>(warp_max_u32(top_v));
    if (lane == 0) {
      T.m_exp[blk] = static_cast<uint8_t>(new_m);
      T.v_exp[blk] = static_cast<uint8_t>(new_v);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t i = b0 + h * 128 + lane * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j >= T.n) continue;
        const uint32_t h32 = mix(static_cast<uint32_t>(T.first + i + j) + a.key);
        static_cast<uint8_t*>(T.m)[i + j] =
            static_cast<uint8_t>(encode<3>(__float_as_uint(m[h][j]), h32 & 0xffffu, new_m));
        static_cast<uint8_t*>(T.v)[i + j] =
            static_cast<uint8_t>(encode<4>(__float_as_uint(s[h][j]), h32 >> 16, new_v));
      }
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

template <int MANT>
__global__ void __launch_bounds__(256)
adamw_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n,
                  __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    out[i] = __float2bfloat16_rn(decode<MANT>(codes[i], exps[i / kBlock]));
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
  const int64_t need = (n + 255) / 256, cap = static_cast<int64_t>(ctx.num_sms) * 16;
  const int grid = static_cast<int>(need < cap ? need : cap);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  return cuda_status(
      which == OCCULT_STATE_M
          ? launch_pdl(adamw_read_kernel<3>, grid, 256, 0, ctx.stream, codes, exps, n, o)
          : launch_pdl(adamw_read_kernel<4>, grid, 256, 0, ctx.stream, codes, exps, n, o));
}

}  // namespace occult
