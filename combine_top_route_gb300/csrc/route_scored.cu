// The scored router: softmax or sigmoid scores, a bias on the choice, groups of
// experts, the top k of the kept groups, their gates and the gradient.
//
// One warp a token.  The groups lie side by side on the lanes: a group has 32 / G' lanes
// (G' the power of two from G up), each up to PL of its experts, so that a group's worth
// is a few shuffles.  The choice runs on one 32-bit word an expert -- 23 bits of rank and
// the expert's number -- sorted in the lane, then k + 1 rounds of one warp-wide maximum
// (redux) whose winner's lane moves up its next word.
//
// Those 23 bits decide only what they can: with a bias, ranks in steps of 2^-23 of their
// span, about the error of a score made with the fast exponential and reciprocal; without
// one, the upper bits of the logits.  Places nearer to each other than that (a few tokens
// in ten thousand, one in a hundred without a bias) are put in order by their logits, or
// by their ranks in fp64 where there is a bias: one exponential on the lanes that hold the
// candidates.  Two worths within some 4e-6 at the border of the kept groups are made again in
// fp64, from the candidates of these two groups where they are few, else by the whole choice in
// fp64: one token in 10^5 of logits of deviation 1.  Of wider ones more worths are that near, or
// that small: 32768 tokens x 256 experts in 8 groups by their best two go from 42 us (deviation
// 1) to 247 (8) by sigmoids, from 58 to 306 by a softmax with a bias, from 38 to 88 by one
// without.  One best score without a bias is its logit and needs none of it (36 us at any).
// fp64 for every token would cost more than the rest together: the chip has two fp64 lanes
// an SM.
//
// A token's chain of steps bounds the choice, not its bytes: 32768 tokens x 256 experts in 8
// groups, 4 of them and 8 experts kept, sigmoid with a bias, take 34 to 37 us (33.5 MB of logits,
// 5 us at the copy rate) with 54 to 57 % of the issue slots used and the integer pipe 36 to 42 %
// busy: the rest are waits for the step before (sort, then one dependent maximum a place).  145 us
// with the choice in fp64 for every tie within fp32's error, 66 before near places were
// told apart from their candidates alone; two tokens a warp, half a warp each, and tokens
// dealt out by a shared counter were no faster.  16383 tokens x 60 experts: 11 us.  Few
// tokens wait for the launch and one token's chain: 512 x 256 in 5 us.  The gradient moves
// 8 bytes a logit near the copy rate (10 to 13 us for the 67 MB of the first case; by a softmax,
// whose every score is made again, 18 us renormalised, 23 not).
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLowest = -3.402823466e+38f;   // a logit as low as this is switched off
#define OCCULT_NEG_INF (-__int_as_float(0x7f800000))

// Words of the choice: on (bit 31) or switched off (bit 30);
// bits 8..30 the rank, the lowest eight 255 - expert (equal ranks: the lower expert).
// 0: none, or in no kept group (the kept ones hold at least k).
constexpr uint32_t kOn = 1u << 31, kOff = 1u << 30;

__device__ __forceinline__ bool is_off(float z) { return !(z > kLowest); }  // NaN too

// Bits that order as the floats do (-0 as 0).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_bits64(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.));
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o) {
  return static_cast<uint64_t>(__shfl_xor_sync(kFull, static_cast<unsigned long long>(v), o));
}
__device__ __forceinline__ uint64_t shfl64(uint64_t v, int lane) {
  return static_cast<uint64_t>(__shfl_sync(kFull, static_cast<unsigned long long>(v), lane));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

struct RouteArgs {
  const float* logits;
  const float* bias;
  const int32_t* e2v;
  int32_t* ids;
  float* gates;
  uint32_t* vmask;
  int T, Ne, k, G, keep, best, vdev_groups, renorm;
  int per, group_lanes;    // experts and lanes of a group (2^group_shift)
  int group_shift, holes;  // holes: some of the lanes' places hold no expert
  int vec;                 // a lane's experts are aligned fours of consecutive logits
  float scale;
};

// Score for a gate (IEEE): top and total of the softmax's exponentials.
template <bool SIG>
__device__ __forceinline__ float score_of(float z, float top, float total) {
  if (z <= kLowest) return 0.f;
  return SIG ? 1.f / (1.f + expf(-z)) : expf(z - top) / total;
}

// ---- the choice in fp64 --------------------------------------------------------------
// An fp64 instruction takes a warp 64 cycles of its scheduler here, a logistic function
// some fifty of them; comparisons are made on integers of the same order.

// A score as the sum of `whole` and `rest`: a sigmoid above a half is 1 less its complement, so
// that the rests of z and -z cancel and sigmoid(x) + sigmoid(-x) is 1 for every x.
struct Score64 {
  double whole, rest;
  __device__ __forceinline__ double value() const { return whole + rest; }
};
template <bool SIG>
__device__ __forceinline__ Score64 score64(float z, float top, double inv) {
  if (!SIG) return {0., exp(static_cast<double>(z) - static_cast<double>(top)) * inv};
  const double c = 1. / (1. + exp(fabs(static_cast<double>(z))));
  return z > 0.f ? Score64{1., -c} : Score64{0., c};
}
// Rank of an expert that is on, as an ordered integer: by score and bias, without a bias by its
// logit, which no score is too near 0 or 1 for.  A NaN ranks below every number.
template <bool SIG>
__device__ __forceinline__ uint64_t rank64(float z, int e, const float* bias, float top, double inv) {
  if (!bias) return order_bits64(static_cast<double>(z));
  const double v = score64<SIG>(z, top, inv).value() + static_cast<double>(bias[e]);
  return order_bits64(v == v ? v : static_cast<double>(OCCULT_NEG_INF));
}

// The worth of a group, as two ordered integers: the sum of its scores and biases in fp64, and
// what that sum's rounding left out.  All 0: no expert that is on.
struct Worth {
  uint64_t hi, lo;
  __device__ __forceinline__ bool above(const Worth& o) const { return hi > o.hi || (hi == o.hi && lo > o.lo); }
  __device__ __forceinline__ bool same(const Worth& o) const { return hi == o.hi && lo == o.lo; }
  __device__ __forceinline__ Worth of(int lane) const { return {shfl64(hi, lane), shfl64(lo, lane)}; }
};

// Worth of a group of lanes from the best two of each: ranks r1, r2 (0: none) of experts e1, e2,
// equal ranks by the lower expert.  One best score without a bias orders as its logit.
template <bool SIG>
__device__ __forceinline__ Worth group_worth(uint64_t r1, uint64_t r2, int e1, int e2, const RouteArgs& a,
                                             const float* row, const float* bias, float top, double inv) {
  for (int o = 1; o < a.group_lanes; o <<= 1) {
    const uint64_t q1 = shfl_xor64(r1, o), q2 = shfl_xor64(r2, o);
    const int f1 = __shfl_xor_sync(kFull, e1, o), f2 = __shfl_xor_sync(kFull, e2, o);
    const bool theirs = q1 > r1 || (q1 == r1 && f1 < e1);
    // behind the first: the other lane's first, or the second of its own lane
    const uint64_t s1 = theirs ? r1 : q1, s2 = theirs ? q2 : r2;
    const int g1 = theirs ? e1 : f1, g2 = theirs ? f2 : e2;
    const bool second = s2 > s1 || (s2 == s1 && g2 < g1);
    r2 = second ? s2 : s1;
    e2 = second ? g2 : g1;
    if (theirs) { r1 = q1; e1 = f1; }
  }
  if (r1 == 0) return {0, 0};
  if (!bias && a.best == 1) return {r1, 0};
  Score64 s = score64<SIG>(row[e1], top, inv);
  if (bias) s.whole += static_cast<double>(bias[e1]);
  if (a.best == 2 && r2 != 0) {
    const Score64 n = score64<SIG>(row[e2], top, inv);
    s.whole += n.whole + (bias ? static_cast<double>(bias[e2]) : 0.);
    s.rest += n.rest;
  }
  const double sum = s.whole + s.rest, back = sum - s.whole;
  const double left = (s.whole - (sum - back)) + (s.rest - back);   // (exactly what the sum left out)
  if (!(fabs(sum) < 1e300))   // biases that are no numbers or infinite
    return {order_bits64(sum == sum ? sum : static_cast<double>(OCCULT_NEG_INF)), order_bits64(0.)};
  return {order_bits64(sum), order_bits64(left)};
}

// The whole choice of one token, ranks and worths as doubles.  Returns slot `lane`'s
// expert.
template <bool SIG, int PL>
__device__ __noinline__ int choose_exactly(const RouteArgs& a, const float* row, const int* s_exp) {
  const int lane = threadIdx.x & 31;
  float z[PL];
  uint64_t r[PL];   // rank by score and bias; 0: none or switched off
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = s_exp[lane * PL + i];
    z[i] = e >= 0 ? row[e] : kLowest;
  }
  double inv = 1.;
  float top = kLowest;
  if (!SIG) {
#pragma unroll
    for (int i = 0; i < PL; ++i) top = fmaxf(top, z[i]);
    top = warp_max(top);
  }
  if (!SIG && a.bias) {   // (without a bias the total is a common factor: left out)
    double total = 0.;
    for (int i = 0; i < PL; ++i)
      if (!is_off(z[i])) total += exp(static_cast<double>(z[i]) - static_cast<double>(top));
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    inv = 1. / total;
  }
  uint64_t b1 = 0, b2 = 0;
  int e1 = 0x7fffffff, e2 = 0x7fffffff;
#pragma unroll 1
  for (int i = 0; i < PL; ++i) {
    const int e = s_exp[lane * PL + i];
    r[i] = 0;
    if (is_off(z[i])) continue;
    r[i] = rank64<SIG>(z[i], e, a.bias, top, inv);
    if (r[i] > b1) { b2 = b1; e2 = e1; b1 = r[i]; e1 = e; } else if (r[i] > b2) { b2 = r[i]; e2 = e; }
  }
  bool in = true;
  if (a.G > 1) {
    const Worth worth = group_worth<SIG>(b1, b2, e1, e2, a, row, a.bias, top, inv);
    const int mine = lane / a.group_lanes;
    int place = 0;
    for (int g = 0; g < a.G; ++g) {
      const Worth w = worth.of(g * a.group_lanes);
      place += (w.above(worth) || (w.same(worth) && g < mine)) ? 1 : 0;
    }
    in = mine < a.G && place < a.keep;
  }
  // an expert's word: on (far above 1 for every number), off, or none
#pragma unroll 1
  for (int i = 0; i < PL; ++i) {
    const int e = s_exp[lane * PL + i];
    r[i] = e < 0 || !in ? 0 : is_off(z[i]) ? 1 : r[i];
  }
  int mine = 0;
  uint32_t gone = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t v = 0;
    int id = 0x7fffffff;
#pragma unroll 1
    for (int i = 0; i < PL; ++i) {
      const int e = s_exp[lane * PL + i];
      if (((gone >> i) & 1u) || r[i] == 0) continue;
      if (r[i] > v || (r[i] == v && e < id)) { v = r[i]; id = e; }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t w = shfl_xor64(v, o);
      const int e = __shfl_xor_sync(kFull, id, o);
      if (w > v || (w == v && e < id)) { v = w; id = e; }
    }
#pragma unroll 1
    for (int i = 0; i < PL; ++i)
      if (s_exp[lane * PL + i] == id) gone |= 1u << i;
    if (lane == j) mine = id;
  }
  return mine;
}

// The border of the kept groups, `last` the last kept and `next` the first left out, whose
// worths fp32 cannot tell apart: made again in fp64 from the experts of these two that can
// be among their best (`e1`, `e2`: a lane's two, where `c1`, `c2`).  (Not for softmax with a bias,
// which needs the total.)
// True: the group left out is the better one.
template <bool SIG, bool BIAS>
__device__ __noinline__ bool next_is_better(const RouteArgs& a, const float* row, const float* s_bias,
                                            float top, int e1, int e2, bool c1, bool c2, int last,
                                            int next) {
  const float* bias = BIAS ? s_bias : nullptr;
  uint64_t r1 = c1 ? rank64<SIG>(row[e1], e1, bias, top, 1.) : 0, r2 = c2 ? rank64<SIG>(row[e2], e2, bias, top, 1.) : 0;
  if (r2 > r1 || (r2 == r1 && e2 < e1)) {
    const uint64_t r = r1;
    const int e = e1;
    r1 = r2; e1 = e2;
    r2 = r; e2 = e;
  }
  const Worth worth = group_worth<SIG>(r1, r2, e1, e2, a, row, bias, top, 1.);
  const Worth w0 = worth.of(last * a.group_lanes), w1 = worth.of(next * a.group_lanes);
  return w1.above(w0) || (w1.same(w0) && next < last);
}

template <int PL>
__device__ __forceinline__ void cas(uint32_t (&v)[PL], int i, int j) {
  const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
  v[i] = hi;
  v[j] = lo;
}
// A lane's words in descending order (odd-even merges).
template <int PL>
__device__ __forceinline__ void sort_down(uint32_t (&v)[PL]) {
  if constexpr (PL > 1) {
#pragma unroll
    for (int p = 1; p < PL; p *= 2)
#pragma unroll
      for (int q = p; q >= 1; q /= 2)
#pragma unroll
        for (int j = q % p; j + q < PL; j += 2 * q)
#pragma unroll
          for (int i = 0; i < q; ++i)
            if (i + j + q < PL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) cas<PL>(v, i + j, i + j + q);
  }
}

// Blocks an SM: registers for 24 warps, 32 where a lane holds few experts.
constexpr int blocks_per_sm(int pl) { return pl <= 2 ? 5 : pl <= 8 ? 4 : 1; }

// The first places of a warp's sorted words, a maximum at a time; lane j keeps place j.
template <int PL>
__device__ __forceinline__ void draw(uint32_t (&key)[PL], int j, uint32_t& mine) {
  const uint32_t w = __reduce_max_sync(kFull, key[0]);
  if (key[0] == w) {
#pragma unroll
    for (int i = 0; i + 1 < PL; ++i) key[i] = key[i + 1];
    key[PL - 1] = 0;
  }
  if ((threadIdx.x & 31) == j) mine = w;
}

// Places too near to each other for their words: more of them until one is clearly lower,
// then in order by logits, or by fp64 ranks where there is a bias.  False: the whole
// choice has to be made in fp64.  A softmax's ranks are made with the total in fp32, which
// is within 2^-19 of itself and errs for all of them alike: it moves the difference of two
// ranks by no more than that of the difference of their scores; two that are nearer than
// this need the total in fp64, and with it every expert.
template <bool SIG, bool BIAS, int PL>
__device__ __noinline__ bool order_near(uint32_t (&key)[PL], uint32_t mine, int have, int k, int Ne,
                                        uint32_t gap_max, const float* row, const float* s_bias,
                                        float top, float total, int& my_id) {
  const int lane = threadIdx.x & 31;
  float z = mine >= kOn ? row[my_id] : 0.f;
  {
    // the same logit under the same bias is a tie, and stands in order
    const float b = BIAS && mine >= kOn ? s_bias[my_id] : 0.f;
    const uint32_t nxt = __shfl_down_sync(kFull, mine, 1);
    const float nz = __shfl_down_sync(kFull, z, 1), nb = __shfl_down_sync(kFull, b, 1);
    if (!__any_sync(kFull, lane < k && lane < 31 && mine >= kOn && nxt >= kOn &&
                               (mine >> 8) - (nxt >> 8) <= gap_max && !(z == nz && b == nb)))
      return true;
  }
  for (;;) {
    const uint32_t last = __shfl_sync(kFull, mine, have - 1), prev = __shfl_sync(kFull, mine, have - 2);
    if (last < kOn || (prev >> 8) - (last >> 8) > gap_max || have == Ne) break;
    if (have == 32) return false;
    draw<PL>(key, have++, mine);
  }
  my_id = 255 - static_cast<int>(mine & 255u);
  const bool on = lane < have && mine >= kOn;
  uint64_t r = 0;   // above 0 for places that are on: they stand before the others
  double v = 0.;
  float p = 0.f;    // a softmax's score
  if (on) {
    z = row[my_id];
    if (BIAS) {
      if (SIG) {
        v = score64<SIG>(z, top, 1.).value();
      } else {
        v = exp(static_cast<double>(z) - static_cast<double>(top)) * (1. / static_cast<double>(total));
        p = static_cast<float>(v);
      }
      v += static_cast<double>(s_bias[my_id]);
      r = order_bits64(v);
    } else {
      r = static_cast<uint64_t>(order_bits(z)) + 1;
    }
  }
  int place = on ? 0 : lane;
  bool unsure = false;
  for (int j = 0; j < have; ++j) {
    const uint64_t o = shfl64(r, j);
    const int e = __shfl_sync(kFull, my_id, j);
    if (on && (o > r || (o == r && e < my_id))) ++place;
    if (BIAS && !SIG) {
      const float gap = fabsf(static_cast<float>(__shfl_sync(kFull, v, j) - v));
      const float dp = fabsf(__shfl_sync(kFull, p, j) - p);
      const bool there = __shfl_sync(kFull, static_cast<int>(on), j) != 0;
      // (scores of one logit are equal, whatever the total)
      unsure |= on && there && dp > 0.f && gap <= 0x1p-19f * dp + 0x1p-50f;
    }
  }
  if (BIAS && !SIG && __any_sync(kFull, unsure)) return false;
  int sorted = my_id;
  for (int j = 0; j < have; ++j) {
    const int at = __shfl_sync(kFull, place, j), e = __shfl_sync(kFull, my_id, j);
    if (at == lane) sorted = e;
  }
  my_id = sorted;
  return true;
}

template <bool SIG, bool BIAS, int PL>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm(PL))
route_scored_kernel(const RouteArgs a) {
  __shared__ int s_dev[OCCULT_MAX_EXPERTS], s_exp[PL * 32];
  __shared__ float s_bias[OCCULT_MAX_EXPERTS], s_span[2];
  __shared__ bool s_odd;
  __shared__ int s_count[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the experts of every lane's places, and the bias's span
  static_assert(kWarps * 32 >= OCCULT_MAX_EXPERTS, "a thread an expert");
  const int dev = tid < a.Ne ? a.e2v[tid] & 31 : 32;
  if (tid < a.Ne) {
    s_dev[tid] = dev;
    s_bias[tid] = BIAS ? a.bias[tid] : 0.f;
  }
  for (int i = tid; i < PL * 32; i += kWarps * 32) {
    const int g = (i / PL) >> a.group_shift, j = i - (g << a.group_shift) * PL;
    s_exp[i] = !a.vdev_groups && g < a.G && j < a.per ? g * a.per + j : -1;
  }
  if (a.vdev_groups) {
    // an expert's number among its device's: those before it in its warp, and the warps'
    // counts
    for (int i = tid; i < kWarps * 32; i += kWarps * 32) s_count[i / 32][i % 32] = 0;
    __syncthreads();
    const uint32_t same = __match_any_sync(kFull, dev);
    int j = __popc(same & lanemask_lt());
    if (j == 0 && dev < 32) s_count[warp][dev] = __popc(same);
    __syncthreads();
    if (dev < a.G) {
      for (int w = 0; w < warp; ++w) j += s_count[w][dev];
      if (j < a.per) s_exp[(dev << a.group_shift) * PL + j] = tid;
    }
  } else {
    __syncthreads();
  }
  if (BIAS && warp == 0) {
    float lo = 3e38f, hi = -3e38f;
    bool odd = false;
    for (int e = lane; e < a.Ne; e += 32) {
      lo = fminf(lo, s_bias[e]);
      hi = fmaxf(hi, s_bias[e]);
      odd |= !(fabsf(s_bias[e]) < 1e18f);
    }
    lo = -warp_max(-lo);
    hi = warp_max(hi);
    odd = __any_sync(kFull, odd);
    if (lane == 0) { s_span[0] = lo; s_span[1] = hi; s_odd = odd; }
  }
  __syncthreads();
  // Ranks with a bias lie in [base, base + span]: s * q_mul + c, in whole numbers behind
  // 2^23, is a rank's place in 2^23 steps of the span.
  const bool odd = BIAS && s_odd;   // biases without a span: every token in fp64
  const float base = BIAS && !odd ? s_span[0] : 0.f;
  const float span = BIAS && !odd ? 1.f + (s_span[1] - s_span[0]) : 1.f;
  const float q_mul = 8388600.f / span;
  // A score made with ex2 and rcp is within 2^-21 of itself (|z| <= 16; beyond that its
  // distance from 0 or 1 is; a softmax's total errs by some 2^-20 as well, for all of its
  // scores alike), bias and rank within 2^-24 of their size, the steps add a half each:
  // two ranks further apart than this many steps are in order.
  const float slack = (SIG ? 0x1p-20f : 0x1p-19f) + 0x1p-22f * (fabsf(base) + span);
  const uint32_t gap_max = BIAS ? static_cast<uint32_t>(fminf(slack * q_mul, 8388606.f)) + 3u : 0u;
  // (the words' steps come on top where worths are made from them)
  const float slack_worth = 2.f * slack + (BIAS ? 4.f / q_mul : 0.f);
  int ex[PL];
  uint32_t low[PL];
  float c[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    ex[i] = s_exp[lane * PL + i];
    low[i] = 255u - static_cast<uint32_t>(ex[i]);
    c[i] = BIAS && ex[i] >= 0 ? fmaf(s_bias[ex[i]] - base, q_mul, 8388608.f) : 0.f;
  }
  const int my_group = lane >> a.group_shift;
  const int rounds = min(min(a.k + 1, a.Ne), 32);

  // (unsigned: the last step may pass 2^31)
  for (uint32_t t = blockIdx.x * kWarps + warp; t < static_cast<uint32_t>(a.T); t += gridDim.x * kWarps) {
    const float* row = a.logits + static_cast<size_t>(t) * a.Ne;
    float z[PL];
    if (PL % 4 == 0 && a.vec) {
#pragma unroll
      for (int i = 0; i < PL; i += 4) {
        const float4 v = ex[i] >= 0 ? __ldg(reinterpret_cast<const float4*>(row + ex[i]))
                                    : make_float4(kLowest, kLowest, kLowest, kLowest);
        z[i] = v.x; z[i + (PL > 1 ? 1 : 0)] = v.y; z[i + (PL > 2 ? 2 : 0)] = v.z; z[i + (PL > 3 ? 3 : 0)] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) z[i] = ex[i] >= 0 ? row[ex[i]] : kLowest;
    }
    float top = 0.f, total = 1.f, s[PL];
    bool no_number = false;   // a softmax's row with a NaN logit
    if (!SIG) {
      top = kLowest;
#pragma unroll
      for (int i = 0; i < PL; ++i) top = fmaxf(top, z[i]);   // NaN is skipped
      top = warp_max(top);
      total = 0.f;
      // (places without an expert hold kLowest; a NaN logit makes the total NaN)
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        s[i] = z[i] <= kLowest ? 0.f : expf(z[i] - top);
        total += s[i];
      }
      total = warp_sum(total);
      no_number = !(total == total);
      if (no_number) {   // the choice goes by the scores of the others; the gates are NaN
        total = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          if (is_off(z[i])) s[i] = 0.f;
          total += s[i];
        }
        total = warp_sum(total);
      }
      const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] *= inv;
    } else if (BIAS || a.G > 1) {
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] = rcp(1.f + ex2(z[i] * -kLog2e));
    } else {   // the logits alone choose
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] = 0.f;
    }

    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t q = BIAS ? __float_as_uint(fmaf(s[i], q_mul, c[i])) << 8
                              : (order_bits(z[i]) >> 1) & 0x7fffff00u;
      key[i] = is_off(z[i]) ? kOff | low[i] : q + (kOn | low[i]);
    }
    if (a.holes) {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (ex[i] < 0) key[i] = 0;
    }
    sort_down<PL>(key);

    bool exact = odd;
    if (a.G > 1) {
      // the group's best two: with a bias from the words, else from the scores, the one best by its
      // logit, which orders as its score does and needs no other look
      const bool by_logit = !BIAS && a.best == 1;
      float b1 = kLowest, b2 = kLowest;
      if (BIAS) {
        const float back = span / 8388600.f;
        if (key[0] >= kOn) b1 = fmaf(static_cast<float>((key[0] >> 8) & 0x7fffffu), back, base);
        if (PL > 1 && key[PL > 1 ? 1 : 0] >= kOn)
          b2 = fmaf(static_cast<float>((key[PL > 1 ? 1 : 0] >> 8) & 0x7fffffu), back, base);
      } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const float r = is_off(z[i]) ? kLowest : by_logit ? z[i] : s[i];
          b2 = fmaxf(b2, fminf(b1, r));
          b1 = fmaxf(b1, r);
        }
      }
      for (int o = 1; o < a.group_lanes; o <<= 1) {
        const float c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
        b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
        b1 = fmaxf(b1, c1);
      }
      const float worth = a.best == 2 && b2 > kLowest ? b1 + b2 : b1;
      // the keep groups of largest worth, one maximum each: equal ones from the left; then
      // the first left out, which the last kept must be clearly above
      uint32_t wkey = my_group < a.G ? order_bits(worth) : 0u;
      uint32_t in = 0, last = 0, before = 0;
      int g_last = 0;
      for (int g = 0; g < a.keep; ++g) {
        before = last;
        last = __reduce_max_sync(kFull, wkey);
        g_last = (__ffs(__ballot_sync(kFull, wkey == last)) - 1) >> a.group_shift;
        if (my_group == g_last) { wkey = 0; in = 1; }
      }
      if (a.keep < a.G && !by_logit) {
        auto unbits = [](uint32_t u) { return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u); };
        const uint32_t next = __reduce_max_sync(kFull, wkey);
        const float w0 = unbits(last), w1 = unbits(next);
        const float tell = slack_worth + 0x1p-22f * (fabsf(w0) + fabsf(w1));
        // (two groups without an expert are equal exactly)
        if (w1 > kLowest && w0 - w1 <= tell) {
          const int g_next = (__ffs(__ballot_sync(kFull, wkey == next)) - 1) >> a.group_shift;
          const uint32_t after = __reduce_max_sync(kFull, my_group == g_next ? 0u : wkey);
          // what can be among the best of these two groups: a lane's best two, no third
          const float edge = (a.best == 2 && b2 > kLowest ? b2 : b1) - tell;
          const bool here = my_group == g_last || my_group == g_next;
          int e1 = -1, e2 = -1;
          bool many = false;
          float r1 = kLowest;
#pragma unroll
          for (int i = 0; i < PL; ++i) {
            const float r = BIAS ? s[i] + s_bias[max(ex[i], 0)] : s[i];
            if (!here || is_off(z[i]) || !(r >= edge)) continue;
            many |= e2 >= 0;
            if (r > r1) { e2 = e1; e1 = ex[i]; r1 = r; } else e2 = ex[i];
          }
          if ((BIAS && !SIG) || __any_sync(kFull, many) || (a.keep > 1 && unbits(before) - w1 <= tell) ||
              (after != 0 && w0 - unbits(after) <= tell)) {
            exact = true;
          } else if (next_is_better<SIG, BIAS>(a, row, s_bias, top, e1, e2, e1 >= 0, e2 >= 0, g_last, g_next)) {
            if (my_group == g_last) in = 0;
            if (my_group == g_next) in = 1;
          }
        }
      }
      if (!in) {
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = 0;
      }
    }

    int my_id = 0;
    if (!exact) {
      uint32_t mine = 0;
#pragma unroll 3
      for (int j = 0; j < rounds; ++j) draw<PL>(key, j, mine);
      my_id = 255 - static_cast<int>(mine & 255u);
      const uint32_t nxt = __shfl_down_sync(kFull, mine, 1);
      if (__any_sync(kFull, lane < a.k && lane < 31 && mine >= kOn && nxt >= kOn &&
                                (mine >> 8) - (nxt >> 8) <= gap_max))
        exact = !order_near<SIG, BIAS, PL>(key, mine, rounds, a.k, a.Ne, gap_max, row, s_bias, top,
                                             total, my_id);
    }
    if (exact) my_id = choose_exactly<SIG, PL>(a, row, s_exp);
    if (my_id < 0 || my_id >= a.Ne) my_id = 0;   // (devices that do not share the experts evenly)

    if (!SIG && no_number) total = __int_as_float(0x7fc00000);
    float g = lane < a.k ? score_of<SIG>(row[my_id], top, total) : 0.f;
    if (a.renorm) {
      const float sum = warp_sum(g);
      // (the fast division is for sums of normal size)
      if (sum >= 0x1p-120f) g = __fdividef(g, sum);
      else g = sum == 0.f ? 0.f : g / sum;
    }
    const uint32_t vm = __reduce_or_sync(kFull, lane < a.k ? 1u << s_dev[my_id] : 0u);
    if (lane < a.k) {
      a.ids[static_cast<size_t>(t) * a.k + lane] = my_id;
      a.gates[static_cast<size_t>(t) * a.k + lane] = a.scale * g;
    }
    if (lane == 0) a.vmask[t] = vm;
  }
}

// Total of the softmax's exponentials over the experts that are on; a NaN logit makes
// it NaN.  (The warp's lanes hold z[i] of expert lane + 32 i.)
template <int PL>
__device__ __forceinline__ void softmax_stats(const float (&z)[PL], int Ne, float& top, float& total) {
  const int lane = threadIdx.x & 31;
  top = kLowest;
#pragma unroll
  for (int i = 0; i < PL; ++i) top = fmaxf(top, z[i]);   // NaN is skipped
  top = warp_max(top);
  total = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (lane + 32 * i < Ne && !(z[i] <= kLowest)) total += expf(z[i] - top);
  total = warp_sum(total);
}

// ---- gradient -------------------------------------------------------------------
// The row is put together in shared memory: the k chosen experts' terms on zeros, then
// (softmax, not renormalised) the common term of every expert, and written as it lies.
template <bool SIG, int PL>
__global__ void __launch_bounds__(kWarps * 32)
route_scored_grad_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                         const float* __restrict__ dgates, float* __restrict__ dlogits, int T,
                         int Ne, int k, int renorm, float scale) {
  __shared__ float s_row[kWarps][PL * 32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  float* sm = s_row[warp];
  for (uint32_t t = blockIdx.x * kWarps + warp; t < static_cast<uint32_t>(T); t += gridDim.x * kWarps) {
    const float* row = logits + static_cast<size_t>(t) * Ne;
    float z[PL];
    float top = 0.f, total = 1.f;
    if (!SIG) {
#pragma unroll
      for (int i = 0; i < PL; ++i) z[i] = lane + 32 * i < Ne ? row[lane + 32 * i] : kLowest;
      softmax_stats<PL>(z, Ne, top, total);
    }
    int id = lane < k ? ids[static_cast<size_t>(t) * k + lane] : -1;
    if (id < 0 || id >= Ne) id = -1;
    const float u = id >= 0 ? scale * dgates[static_cast<size_t>(t) * k + lane] : 0.f;
    const float s = id >= 0 ? score_of<SIG>(row[id], top, total) : 0.f;
    // The chosen experts' terms.  Renormalised, a gate depends on the scores' shares of their sum
    // alone: p_j (u_j - sum p_i u_i), which no sum is too small for; the terms add up to 0, so that a
    // softmax has no other ones.  Differences are taken from the largest score's u first: where its
    // share is nearly 1, its own term is as small as the others' together, and u_j less a mean
    // that is nearly u_j would keep no digit of it (a token's only expert has none, exactly).
    float own = SIG ? u * s : u, all = 0.f;
    int sure = -1;         // softmax: an expert with more than half of the sum, and its term
    float sure_term = 0.f;
    if (renorm) {
      const float S = warp_sum(s);
      const float p = S == 0.f ? 0.f : s / S;
      const uint32_t bits = __float_as_uint(s);
      const int lead = __ffs(__ballot_sync(kFull, bits == __reduce_max_sync(kFull, bits))) - 1;
      const float base = __shfl_sync(kFull, u, lead);
      const float v = id >= 0 ? u - base : 0.f;
      own = p * (v - warp_sum(v * p));
    } else if (!SIG) {
      all = warp_sum(u * s);
      const uint32_t half = __ballot_sync(kFull, s > 0.5f);
      if (half) {
        // the same cancellation: u (1 - s) less the others' u s, 1 - s from the other exponentials
        sure = __shfl_sync(kFull, id, __ffs(half) - 1);
        float rest = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i)
          if (lane + 32 * i != sure && !(z[i] <= kLowest)) rest += expf(z[i] - top);
        rest = warp_sum(rest) / total;
        const float mine = warp_sum(id == sure ? u : 0.f);
        sure_term = (1.f - rest) * (mine * rest - warp_sum(id == sure ? 0.f : u * s));
      }
    }
    // 1 - s = e^-z s: the difference keeps no digit of it from logits of 17 on
    if (SIG && s > 0.f) own *= expf(-row[id]) * s;
#pragma unroll
    for (int i = 0; i < PL; ++i) sm[lane + 32 * i] = 0.f;
    __syncwarp();
    // (two slots of one expert, which the router does not write, add up)
    if (id >= 0) atomicAdd(&sm[id], own);
    __syncwarp();
    float* out = dlogits + static_cast<size_t>(t) * Ne;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < Ne)
        out[e] = SIG || renorm ? sm[e] : e == sure ? sure_term : score_of<SIG>(z[i], top, total) * (sm[e] - all);
    }
    __syncwarp();
  }
}

// One block: the counts' sums over the groups of tokens, then one step of every bias.
__global__ void __launch_bounds__(OCCULT_MAX_EXPERTS)
bias_step_kernel(const int32_t* __restrict__ counts, int G, int Ne, float rate,
                 float* __restrict__ bias) {
  __shared__ long long s_sum;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_sum = 0;
  __syncthreads();
  const int e = threadIdx.x;
  long long c = 0;
  if (e < Ne) {
    for (int g = 0; g < G; ++g) c += counts[static_cast<size_t>(g) * Ne + e];
    // whole numbers: the order of the additions does not matter
    atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum), static_cast<unsigned long long>(c));
  }
  __syncthreads();
  if (e < Ne) {
    const long long d = s_sum - c * Ne;
    if (d != 0) bias[e] += d > 0 ? rate : -rate;
  }
}

int blocks_for(const LaunchCtx& ctx, int T, int per_sm) {
  const int blocks = (T - 1) / kWarps + 1;
  return blocks < ctx.num_sms * per_sm ? blocks : ctx.num_sms * per_sm;
}

}  // namespace

int launch_route_scored(const LaunchCtx& ctx, const occult_desc_t& ds, const occult_score_t& opt,
                        const float* logits, const float* bias, const int32_t* e2v, int32_t* ids,
                        float* gates, uint32_t* vmask) {
  if (ds.T == 0) return OCCULT_OK;
  RouteArgs a{};
  a.logits = logits; a.bias = bias; a.e2v = e2v;
  a.ids = ids; a.gates = gates; a.vmask = vmask;
  a.T = ds.T; a.Ne = ds.n_experts; a.k = ds.top_k;
  a.G = opt.n_groups; a.keep = opt.keep_groups; a.best = opt.group_best;
  a.vdev_groups = opt.group_kind == OCCULT_GROUP_VDEV && a.G > 1;
  a.renorm = ds.renorm; a.scale = opt.scale;
  a.per = a.Ne / a.G;
  int groups = 1;   // the power of two from G up
  while (groups < a.G) groups *= 2;
  a.group_lanes = 32 / groups;
  while ((1 << a.group_shift) < a.group_lanes) ++a.group_shift;
  const int need = (a.per + a.group_lanes - 1) / a.group_lanes;   // experts a lane: at most 15
  // whole fours of a row: consecutive experts, none cut off, rows on 16 bytes
  a.vec = !a.vdev_groups && a.per % 4 == 0 && a.Ne % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  const bool sig = opt.score == OCCULT_SCORE_SIGMOID;
#define OCCULT_SCORED(PL)                                                                  \
  (a.holes = a.vdev_groups || a.group_lanes * a.G != 32 || a.per != a.group_lanes * PL,    \
   cuda_status(launch_pdl(sig ? (bias ? route_scored_kernel<true, true, PL>                 \
                                     : route_scored_kernel<true, false, PL>)               \
                             : (bias ? route_scored_kernel<false, true, PL>                \
                                     : route_scored_kernel<false, false, PL>),             \
                         blocks_for(ctx, ds.T, blocks_per_sm(PL)), kWarps * 32, 0, ctx.stream, a)))
  if (need <= 1) return OCCULT_SCORED(1);
  if (need <= 2) return OCCULT_SCORED(2);
  if (need <= 4) return OCCULT_SCORED(4);
  if (need <= 8) return OCCULT_SCORED(8);
  return OCCULT_SCORED(16);
#undef OCCULT_SCORED
}

int launch_route_scored_grad(const LaunchCtx& ctx, const occult_desc_t& ds,
                             const occult_score_t& opt, const float* logits, const int32_t* ids,
                             const float* dgates, float* dlogits) {
  if (ds.T == 0) return OCCULT_OK;
  const bool sig = opt.score == OCCULT_SCORE_SIGMOID;
  const int nb = blocks_for(ctx, ds.T, 8);
#define OCCULT_SCORED_GRAD(PL)                                                                         \
  cuda_status(launch_pdl(sig ? route_scored_grad_kernel<true, PL> : route_scored_grad_kernel<false, PL>, \
                         nb, kWarps * 32, 0, ctx.stream, logits, ids, dgates, dlogits, ds.T,           \
                         ds.n_experts, ds.top_k, ds.renorm, opt.scale))
  if (ds.n_experts <= 32) return OCCULT_SCORED_GRAD(1);
  if (ds.n_experts <= 64) return OCCULT_SCORED_GRAD(2);
  if (ds.n_experts <= 128) return OCCULT_SCORED_GRAD(4);
  return OCCULT_SCORED_GRAD(8);
#undef OCCULT_SCORED_GRAD
}

int launch_route_bias_step(const LaunchCtx& ctx, int Ne, const int32_t* counts, int G, float rate,
                           float* bias) {
  return cuda_status(launch_pdl(bias_step_kernel, 1, OCCULT_MAX_EXPERTS, 0, ctx.stream, counts, G,
                                Ne, rate, bias));
}

}  // namespace occult
