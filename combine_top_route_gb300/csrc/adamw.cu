// AdamW over many tensors at once, with fp32 states or 8-bit ones.
//
// The 8-bit states are floats of their own: magnitudes x > 0 of a block of 256
// elements are cut to MANT mantissa bits (m: 3 and a sign, sqrt(v): 4) by adding
// a draw to the fp32 word below the cut and truncating, so that the expectation
// is x; the word's leading bits less those of 2^(E - 15), with E the exponent of
// the block's largest (rounded up) value, are the code, 0 .. 16 * 2^MANT - 1.
// All of it is integer arithmetic on the fp32 words, and every code stands for a
// value that bf16 holds exactly.
//
// Bound by the bytes: an element moves 30 with fp32 states, a bf16 parameter and its
// master (28 for an fp32 parameter), 18 with 8-bit states and a master, 16 for an fp32
// and 12 for a bf16 parameter alone.  Measured on one GB300, 402.8 M weights: 1699 us =
// 7.1 TB/s, 1025 us = 7.1 TB/s, 927 us = 7.0 TB/s, and 808 us = 6.0 TB/s for the last,
// which takes 67 instructions an element, a dozen of them the correctly rounded root,
// and most of the issue slots.  Moments, roots and parameters are fp32 until they are
// stored.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kAdamThreads = 128;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kBlock = OCCULT_STATE_BLOCK;       // elements of a warp's step
constexpr int kCtaLog2 = 10;                     // log2 of the weights of kAdamWarps blocks
static_assert(kAdamWarps * kBlock == 1 << kCtaLog2, "a CTA's weights");
constexpr int kMaxTensors = 256;                 // of one launch
constexpr int kSpans = 127;                      // of CTAs, in the search for a CTA's tensor
constexpr int64_t kOwnWeights = 1 << 25;         // of a kind, for a launch of its own

enum : int { KIND_F32 = 0, KIND_MASTER = 1, KIND_BF16 = 2, KIND_ANY = 3 };

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
  int cta_blocks;            // blocks of a CTA
  int span_log2;             // CTAs of a span
  uint8_t span_first[kSpans + 1];  // tensor of a span's first CTA
  int chunk0[kMaxTensors];   // first CTA of every tensor
  Tensor t[kMaxTensors];
};

constexpr uint32_t kMul1 = 0xBB67AE85u, kMul2 = 0x3C6EF373u;  // frac(sqrt 3), frac(sqrt 5), odd

// A 32-bit hash (multiply, fold high bits in, twice), cut before its last fold:
// mix(x) = h ^ (h >> 16) with h = mix_open(x * kMul1).
__host__ __device__ __forceinline__ uint32_t mix_open(uint32_t x_mul1) {
  return (x_mul1 ^ (x_mul1 >> 15)) * kMul2;
}
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  const uint32_t h = mix_open(x * kMul1);
  return h ^ (h >> 16);
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
// The codes of four values, in the bytes of a word, from their fp32 words with the
// draws added below the cut.  From the words' upper halves on two values share a
// register (16-bit lanes): this work is bound by the integer pipe, which runs at
// half the rate of the other one.
__device__ __forceinline__ uint32_t minus_base(uint32_t exp, int mant) {
  return ((0u - ((exp - 15u) << mant)) & 0xffffu) * 0x10001u;
}
__device__ __forceinline__ uint32_t encode4_m(const uint32_t (&a)[4], uint32_t exp) {
  const uint32_t nb = minus_base(exp, 3);
  const uint32_t p01 = __byte_perm(a[0], a[1], 0x7632), p23 = __byte_perm(a[2], a[3], 0x7632);
  const uint32_t k01 = __viaddmax_s16x2((p01 >> 4) & 0x07ff07ffu, nb, 0u);
  const uint32_t k23 = __viaddmax_s16x2((p23 >> 4) & 0x07ff07ffu, nb, 0u);
  const uint32_t k = __byte_perm(k01, k23, 0x6420);       // 0 .. 127 each
  const uint32_t sign = __byte_perm(p01, p23, 0x7531);    // in bit 7 of each byte
  return k | (sign & (k + 0x7f7f7f7fu) & 0x80808080u);    // no sign on a zero
}
__device__ __forceinline__ uint32_t encode4_v(const uint32_t (&a)[4], uint32_t exp) {
  const uint32_t nb = minus_base(exp, 4);
  const uint32_t w01 = (__byte_perm(a[0], a[1], 0x7632) >> 3) & 0x1fff1fffu;
  const uint32_t w23 = (__byte_perm(a[2], a[3], 0x7632) >> 3) & 0x1fff1fffu;
  // at least 1 unless the value is 0 (the root of the least fp32 number is 2^-75, and
  // a draw alone stays below the cut)
  const uint32_t k01 = __viaddmax_s16x2(w01, nb, __vminu2(w01, 0x00010001u));
  const uint32_t k23 = __viaddmax_s16x2(w23, nb, __vminu2(w23, 0x00010001u));
  return __byte_perm(k01, k23, 0x6420);
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
// Bytes j and j + 1 (j even) of a word of codes as two bf16 values in a register;
// `base2` = lanes_base(exp), not of a NaN block.
__device__ __forceinline__ uint32_t lanes_base(uint32_t exp) {
  return (((exp - 15u) << 7) & 0xffffu) * 0x10001u;
}
template <int MANT>
__device__ __forceinline__ uint32_t decode_lanes(uint32_t w, int j, uint32_t base2) {
  const uint32_t c = __byte_perm(w, 0u, j == 0 ? 0x4140 : 0x4342);
  const uint32_t mag = MANT == 3 ? c & 0x007f007fu : c;
  const uint32_t some = __vminu2(mag, 0x00010001u) * 0xffffu;   // a lane of ones where not 0
  uint32_t x = (mag * (1u << (7 - MANT)) + base2) & some;
  if (MANT == 3) x |= (c & 0x00800080u) * 256u;
  return x;
}
template <int MANT>
__device__ __forceinline__ float2 decode_pair(uint32_t w, int j, uint32_t base2) {
  const uint32_t x = decode_lanes<MANT>(w, j, base2);
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Two values to bf16, each by the draw in its half of `draws`: the draw is added below
// the cut of the fp32 word, which is then truncated.
__device__ __forceinline__ uint32_t bf16x2_by_draw(float lo, float hi, uint32_t draws) {
  uint32_t r;
  asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(r) : "f"(hi), "f"(lo), "r"(draws));
  return r;
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
__device__ __forceinline__ void store4(uint16_t* p, int live, const uint32_t (&w)[2]) {
  if (live == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void store4(uint8_t* p, int live, uint32_t c) {
  if (live == 4) {
    *reinterpret_cast<uint32_t*>(p) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p[j] = static_cast<uint8_t>(c >> (8 * j));
  }
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
// The sums of the moments, one by one: a packed sum is contracted with the packed
// products before it whatever rounding they ask for.
__device__ __forceinline__ float2 add_rn(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
// max of three that a NaN among them comes through
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// What a lane reads of one block: elements 4 lane .. 4 lane + 3 of both halves, so
// that every access of the warp is to consecutive words.
template <int BITS>
struct Raw {
  float g[2][4], w[2][4];
  float m[2][4], v[2][4];   // fp32 states
  uint32_t cm[2], cv[2];    // or codes
  uint32_t em, ev;          // and exponents
};
// Elements of this lane's four at `i` that exist (FULL: the block is whole).
template <bool FULL>
__device__ __forceinline__ int live_of(const Tensor& T, int64_t i) {
  if (FULL) return 4;
  const int64_t left = T.n - i;
  return left >= 4 ? 4 : (left > 0 ? static_cast<int>(left) : 0);
}

template <int BITS, int KIND, bool FULL>
__device__ __forceinline__ void load_block(const Tensor& T, int64_t blk, Raw<BITS>& x) {
  const int64_t b0 = blk * kBlock + (threadIdx.x & 31) * 4;
  if (BITS == 8) { x.em = T.m_exp[blk]; x.ev = T.v_exp[blk]; }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b0 + h * 128;
    const int live = live_of<FULL>(T, i);
    load4(T.grad + i, live, x.g[h]);
    if (KIND == KIND_MASTER) load4(static_cast<const float*>(T.master) + i, live, x.w[h]);
    else if (KIND == KIND_F32) load4(static_cast<const float*>(T.param) + i, live, x.w[h]);
    else load4(static_cast<const __nv_bfloat16*>(T.param) + i, live, x.w[h]);
    if (BITS == 32) {
      load4(static_cast<const float*>(T.m) + i, live, x.m[h]);
      load4(static_cast<const float*>(T.v) + i, live, x.v[h]);
    } else {
      x.cm[h] = load4(static_cast<const uint8_t*>(T.m) + i, live);
      x.cv[h] = load4(static_cast<const uint8_t*>(T.v) + i, live);
    }
  }
}

// One block by one warp.  Products are rounded before they are summed (no fused
// multiply-add in the moments and the root, which a code is cut from): the same bits
// as the formula term by term.
template <int BITS, int KIND, bool FULL>
__device__ __forceinline__ void step_block(const AdamTable& a, const Tensor& T, int64_t blk,
                                           float gs, Raw<BITS>& x) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = blk * kBlock + lane * 4;
  float s[2][4];
  float top_m = 0.f, top_v = 0.f;
  uint32_t hash[2][4];
  const uint32_t base_m = lanes_base(x.em), base_v = lanes_base(x.ev);
  // a NaN block comes back as NaN through the gradient's factor
  const float nan = __int_as_float(0x7fffffff);
  const float gs_m = BITS == 8 && x.em == 255u ? nan : gs;
  const float gs_v = BITS == 8 && x.ev == 255u ? nan : gs;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b0 + h * 128;
    const int live = live_of<FULL>(T, i);
    const uint32_t x0 = (static_cast<uint32_t>(T.first + i) + a.key) * kMul1;
    float out[4];
    uint32_t word[2];
    if (BITS == 8 || KIND == KIND_BF16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) hash[h][j] = mix_open(x0 + j * kMul1);
    }
    // two elements at a time: the packed fp32 operations take one issue slot for both
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float2 m, v;
      if (BITS == 8) {
        m = decode_pair<3>(x.cm[h], j, base_m);
        v = decode_pair<4>(x.cv[h], j, base_v);
        v = __fmul2_rn(v, v);
      } else {
        m = make_float2(x.m[h][j], x.m[h][j + 1]);
        v = make_float2(x.v[h][j], x.v[h][j + 1]);
      }
      const float2 g = make_float2(x.g[h][j], x.g[h][j + 1]);
      const float2 gm = __fmul2_rn(two(gs_m), g), gv = __fmul2_rn(two(gs_v), g);
      m = add_rn(__fmul2_rn(two(a.b1), m), __fmul2_rn(two(a.c1), gm));
      v = add_rn(__fmul2_rn(two(a.b2), v), __fmul2_rn(__fmul2_rn(two(a.c2), gv), gv));
      const float2 root = make_float2(sqrtf(v.x), sqrtf(v.y));
      const float2 den = __ffma2_rn(root, two(a.inv_root), two(a.eps));
      const float2 upd = __fmul2_rn(m, make_float2(rcp_approx(den.x), rcp_approx(den.y)));
      const float2 w = __ffma2_rn(two(-a.rate), upd,
                                  __fmul2_rn(make_float2(x.w[h][j], x.w[h][j + 1]), two(a.keep)));
      x.m[h][j] = m.x; x.m[h][j + 1] = m.y;
      x.v[h][j] = v.x; x.v[h][j + 1] = v.y;
      s[h][j] = root.x; s[h][j + 1] = root.y;
      out[j] = w.x; out[j + 1] = w.y;
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      if (KIND == KIND_MASTER) word[j / 2] = pack_bf16x2(out[j], out[j + 1]);
      if (KIND == KIND_BF16) {
        const uint32_t a0 = (hash[h][j] ^ (hash[h][j] >> 16)) * kMul1;
        const uint32_t a1 = (hash[h][j + 1] ^ (hash[h][j + 1] >> 16)) * kMul1;
        word[j / 2] = bf16x2_by_draw(out[j], out[j + 1], __byte_perm(a0, a1, 0x7632));
      }
    }
    if (BITS == 8) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        top_m = max3_nan(top_m, fabsf(x.m[h][j]), fabsf(x.m[h][j + 1]));
        top_v = max3_nan(top_v, s[h][j], s[h][j + 1]);
      }
    } else {
      store4(static_cast<float*>(T.m) + i, live, x.m[h]);
      store4(static_cast<float*>(T.v) + i, live, x.v[h]);
    }
    if (KIND == KIND_F32) store4(static_cast<float*>(T.param) + i, live, out);
    if (KIND == KIND_MASTER) store4(T.master + i, live, out);
    if (KIND != KIND_F32) store4(static_cast<uint16_t*>(T.param) + i, live, word);
  }
  if (BITS == 8) {
    // (elements out of range are zeros here, or NaN in a NaN block: they raise no exponent)
    const uint32_t new_m = block_exp<3>(warp_max_u32(__float_as_uint(top_m)));
    const uint32_t new_v = block_exp<4>(warp_max_u32(__float_as_uint(top_v)));
    if (lane == 0) {
      T.m_exp[blk] = static_cast<uint8_t>(new_m);
      T.v_exp[blk] = static_cast<uint8_t>(new_v);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t am[4], av[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t hi = hash[h][j] >> 16;
        am[j] = __float_as_uint(x.m[h][j]) + ((hash[h][j] ^ hi) & 0xffffu) * 16u;
        av[j] = __float_as_uint(s[h][j]) + hi * 8u;
      }
      const int live = live_of<FULL>(T, b0 + h * 128);
      store4(static_cast<uint8_t*>(T.m) + b0 + h * 128, live, encode4_m(am, new_m));
      store4(static_cast<uint8_t*>(T.v) + b0 + h * 128, live, encode4_v(av, new_v));
    }
  }
}

// The blocks blk, blk + kAdamWarps, ... below end of a tensor by one warp; with 8-bit
// states the next block's words are on their way while this one's are worked on, for a
// bf16 parameter without a master, whose words are few, both blocks' from the start.  402.8
// M weights, us with neither, the next block's and both from the start: bf16 alone 848,
// 940, 812; with a master 1401, 1027, 1100; fp32 1325, 930, 979.
template <int BITS, int KIND>
__device__ __forceinline__ void step_blocks(const AdamTable& a, const Tensor& T, int64_t blk,
                                            int64_t end, float gs) {
  const int64_t whole = T.n / kBlock;
  const int64_t full_end = end < whole ? end : whole;
  Raw<BITS> x;
  if (BITS == 8 && KIND == KIND_BF16 && blk + kAdamWarps < full_end) {
    Raw<BITS> y;
    load_block<BITS, KIND, true>(T, blk, x);
    load_block<BITS, KIND, true>(T, blk + kAdamWarps, y);
    step_block<BITS, KIND, true>(a, T, blk, gs, x);
    step_block<BITS, KIND, true>(a, T, blk + kAdamWarps, gs, y);
    blk += 2 * kAdamWarps;
  } else if (BITS == 8) {
    if (blk < full_end) load_block<BITS, KIND, true>(T, blk, x);
    for (; blk < full_end; blk += kAdamWarps) {
      Raw<BITS> y = x;
      if (blk + kAdamWarps < full_end) load_block<BITS, KIND, true>(T, blk + kAdamWarps, x);
      step_block<BITS, KIND, true>(a, T, blk, gs, y);
    }
  } else {
    for (; blk < full_end; blk += kAdamWarps) {
      load_block<BITS, KIND, true>(T, blk, x);
      step_block<BITS, KIND, true>(a, T, blk, gs, x);
    }
  }
  if (blk < end) {  // the tensor's ragged last block
    load_block<BITS, KIND, false>(T, blk, x);
    step_block<BITS, KIND, false>(a, T, blk, gs, x);
  }
}

// CTAs of an SM: eight, nine for the kind that the issue rate bounds (64 bytes of stack a
// thread for the spills, and 812 us where eight CTAs take 831, ten 832); nine cost the
// other two with 8-bit states more than they give (1083 for 1027 us with masters, 981 for
// 930 in fp32).
__host__ __device__ constexpr int adam_ctas(int bits, int kind) {
  return bits == 8 && kind == KIND_BF16 ? 9 : 8;
}
template <int BITS, int KIND>
__global__ void __launch_bounds__(kAdamThreads, adam_ctas(BITS, KIND))
adamw_kernel(const __grid_constant__ AdamTable a) {
  pdl_wait();
  pdl_trigger();
  // the tensor of this CTA: the last that begins at or before it, between those of the
  // ends of its span of CTAs.  (Each thread looking at its share of the table, whose
  // lines then come one by one, and a sync: 200 tensors of 0.5 M fp32 weights 6.9 us, now
  // 3.3, of 315 M bf16 ones with 8-bit states 764, now 643 us.)
  const int cta = static_cast<int>(blockIdx.x), span = cta >> a.span_log2;
  int which = a.span_first[span], last = a.span_first[span + 1];
  while (which < last) {
    const int mid = (which + last + 1) >> 1;
    if (a.chunk0[mid] <= cta) which = mid;
    else last = mid - 1;
  }
  const Tensor T = a.t[which];
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int64_t blk0 = static_cast<int64_t>(cta - a.chunk0[which]) * a.cta_blocks;
  const int64_t n_blk = (T.n + kBlock - 1) / kBlock;
  const int64_t end = n_blk < blk0 + a.cta_blocks ? n_blk : blk0 + a.cta_blocks;
  const int64_t mine = blk0 + (threadIdx.x >> 5);
  const int kind = KIND == KIND_ANY ? T.kind : KIND;
  if (kind == KIND_F32) step_blocks<BITS, KIND_F32>(a, T, mine, end, gs);
  else if (kind == KIND_MASTER) step_blocks<BITS, KIND_MASTER>(a, T, mine, end, gs);
  else step_blocks<BITS, KIND_BF16>(a, T, mine, end, gs);
}

// The values of 8-bit states: kReadSteps times a thread turns 8 codes into 16 bytes.
// 402.8 M values in 171 us = 7.1 TB/s (205 us with one step a thread).
constexpr int kReadSteps = 2;
constexpr int kReadChunk = 256 * 8 * kReadSteps;
template <int MANT>
__global__ void __launch_bounds__(256)
adamw_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n,
                  __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kReadChunk + threadIdx.x * 8;
  uint2 c[kReadSteps];
  uint32_t e[kReadSteps];
#pragma unroll
  for (int u = 0; u < kReadSteps; ++u) {
    const int64_t i = first + u * 2048;
    if (i + 8 <= n) {
      c[u] = *reinterpret_cast<const uint2*>(codes + i);
      e[u] = exps[i / kBlock];
    }
  }
#pragma unroll
  for (int u = 0; u < kReadSteps; ++u) {
    const int64_t i = first + u * 2048;
    if (i + 8 <= n) {
      const uint32_t base = lanes_base(e[u]);
      uint4 o = make_uint4(decode_lanes<MANT>(c[u].x, 0, base), decode_lanes<MANT>(c[u].x, 2, base),
                           decode_lanes<MANT>(c[u].y, 0, base), decode_lanes<MANT>(c[u].y, 2, base));
      if (e[u] == 255u) o = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      st_v4(out + i, o);
    } else {
      for (int64_t j = i; j < n; ++j)
        out[j] = __float2bfloat16_rn(decode<MANT>(codes[j], exps[j / kBlock]));
    }
  }
}

int kind_of(const occult_param_t& p) {
  return p.dtype == OCCULT_F32 ? KIND_F32 : p.master ? KIND_MASTER : KIND_BF16;
}
template <int BITS>
cudaError_t launch(const LaunchCtx& ctx, int kind, const AdamTable& a, unsigned grid) {
  const auto k = kind == KIND_F32      ? adamw_kernel<BITS, KIND_F32>
                 : kind == KIND_MASTER ? adamw_kernel<BITS, KIND_MASTER>
                 : kind == KIND_BF16   ? adamw_kernel<BITS, KIND_BF16>
                                       : adamw_kernel<BITS, KIND_ANY>;
  return launch_pdl(k, grid, kAdamThreads, 0, ctx.stream, a);
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
  // With 8-bit states two blocks a warp, whose loads and arithmetic overlap, where that
  // leaves four CTAs for each place on the GPU; one for smaller sets and for 32-bit states,
  // which wait for memory alone.  One, two, three blocks took, us for 402.8 M weights: bf16
  // alone with 8-bit states 1030, 808, 932, with masters 1058, 1025, 1221 (the CTAs' streams
  // lie too far apart then); with fp32 states and masters 1699, 1711 (two).
  int64_t blocks = 0, of_kind[3] = {0, 0, 0};
  for (int k = 0; k < n_params; ++k) {
    const int64_t b = (params[k].n + kBlock - 1) / kBlock;
    blocks += b;
    of_kind[kind_of(params[k])] += b;
  }
  const bool two = o.state_bits == 8 && blocks >= static_cast<int64_t>(kAdamWarps) * 2 * 4 * 8 * ctx.num_sms;
  a.cta_blocks = kAdamWarps << two;
  const int chunk_log2 = kCtaLog2 + two;  // weights of a CTA (no division: the host's time counts)
  // A kernel of its own for a kind of 2^25 weights and more, or where there is no other;
  // the rest go together.  Own registers save 402.8 M weights 23 us (bf16 alone with 8-bit
  // states, or masters and fp32 states); a launch more costs 2 to 3 us, and 60 tensors of
  // three kinds and 2560 weights each take 5 us in one, 12 us in three launches, of 2^20
  // each with 8-bit states 152 and 162 us.
  bool own[3];
  for (int k = 0; k < KIND_ANY; ++k)
    own[k] = of_kind[k] == blocks || of_kind[k] >= kOwnWeights / kBlock || of_kind[k] == 0;
  for (int kind = KIND_F32; kind <= KIND_ANY; ++kind) {
    if (kind == KIND_ANY ? own[0] && own[1] && own[2] : !own[kind] || of_kind[kind] == 0) continue;
    int i = 0;
    while (i < n_params) {
      a.n = 0;
      int64_t chunks = 0;
      for (; i < n_params && a.n < kMaxTensors; ++i) {
        const occult_param_t& p = params[i];
        const int its = kind_of(p);
        if (p.n == 0 || (own[its] ? its : KIND_ANY) != kind) continue;
        const int64_t c = ((p.n - 1) >> chunk_log2) + 1;
        if (chunks + c > 0x7fffffff) {
          if (a.n > 0) break;
          return OCCULT_ERR_UNSUPPORTED;
        }
        a.t[a.n] = {p.param, p.master, p.grad, p.m, p.v, p.m_exp, p.v_exp, p.n, p.first, its};
        a.chunk0[a.n++] = static_cast<int>(chunks);
        chunks += c;
      }
      if (a.n == 0) break;
      const unsigned grid = static_cast<unsigned>(chunks);
      a.span_log2 = 0;
      while (((grid - 1) >> a.span_log2) >= kSpans) ++a.span_log2;
      for (int s = 0, k = 0; s <= kSpans; ++s) {  // tensors of the spans' first CTAs
        while (k + 1 < a.n && a.chunk0[k + 1] <= static_cast<int64_t>(s) << a.span_log2) ++k;
        a.span_first[s] = static_cast<uint8_t>(k);
      }
      const cudaError_t e = o.state_bits == 32 ? launch<32>(ctx, kind, a, grid)
                                               : launch<8>(ctx, kind, a, grid);
      if (e != cudaSuccess) return OCCULT_ERR_CUDA;
    }
  }
  return OCCULT_OK;
}

int launch_adamw_read(const LaunchCtx& ctx, const uint8_t* codes, const uint8_t* exps, int64_t n,
                      int which, void* out) {
  const int64_t need = (n + kReadChunk - 1) / kReadChunk;
  if (need > 0x7fffffff) return OCCULT_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(need);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
  return cuda_status(
      which == OCCULT_STATE_M
          ? launch_pdl(adamw_read_kernel<3>, grid, 256, 0, ctx.stream, codes, exps, n, o)
          : launch_pdl(adamw_read_kernel<4>, grid, 256, 0, ctx.stream, codes, exps, n, o));
}

}  // namespace occult
