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
// candidates.  Two worths too near at the border of the kept groups (one token in 10^5)
// send that token through the whole choice in fp64.  fp64 for every token would cost more
// than the rest together: the chip has two fp64 lanes an SM.
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLowest = -3.402823466e+38f;   // a logit as low as this is switched off
#define OCCULT_NEG_INF (-__int_as_float(0x7f800000))

// Words of the choice: on (bit 31), switched off (bit 30), in no kept group (bit 29);
// bits 8..30 the rank, the lowest eight 255 - expert (equal ranks: the lower expert).
constexpr uint32_t kOn = 1u << 31, kOff = 1u << 30, kOut = 1u << 29;

__device__ __forceinline__ bool is_off(float z) { return !(z > kLowest); }  // NaN too

// Bits that order as the floats do (-0 as 0).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
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
  int per, group_lanes;    // experts and lanes of a group
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
// One token, same rules, ranks and worths as doubles.  Returns slot `lane`'s expert.
// `exp_of` gives the expert at this lane's place i, or -1.
template <bool SIG, int PL>
__device__ __noinline__ int choose_exactly(const RouteArgs& a, const float* row, const int* s_exp) {
  const int lane = threadIdx.x & 31;
  const double kNone = -1e300;   // below every rank of finite biases
  double s[PL];
  float z[PL];
  uint32_t live = 0, off = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = s_exp[lane * PL + i];
    z[i] = e >= 0 ? row[e] : kLowest;
    if (e >= 0) live |= 1u << i;
    if (is_off(z[i])) off |= 1u << i;
  }
  if (SIG) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = 1. / (1. + exp(-static_cast<double>(z[i])));
  } else {
    float top = kLowest;
#pragma unroll
    for (int i = 0; i < PL; ++i) top = fmaxf(top, z[i]);
    top = warp_max(top);
    double total = 0.;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = ((off >> i) & 1u) ? 0. : exp(static_cast<double>(z[i]) - static_cast<double>(top));
      total += s[i];
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] /= total;
  }
  double b1 = kNone, b2 = kNone;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    if (a.bias && ((live >> i) & 1u)) s[i] += static_cast<double>(a.bias[s_exp[lane * PL + i]]);
    if (s[i] != s[i]) s[i] = OCCULT_NEG_INF;   // a NaN ranks below every number
    if (!((off >> i) & 1u)) {
      if (s[i] > b1) { b2 = b1; b1 = s[i]; } else if (s[i] > b2) b2 = s[i];
    }
  }
  uint32_t kept = kFull;
  if (a.G > 1) {
    for (int o = 1; o < a.group_lanes; o <<= 1) {
      const double c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
      b2 = fmax(fmax(b2, c2), fmin(b1, c1));
      b1 = fmax(b1, c1);
    }
    double worth = a.best == 2 && b2 > kNone ? b1 + b2 : b1;
    // as multiples of 2^-48: sums that the formula makes equal, as sigmoid(x) +
    // sigmoid(-x) = 1 for every x, then do not hang on the last bits of exp
    if (fabs(worth) < 256.) worth = rint(worth * 0x1p48) * 0x1p-48;
    const int mine = lane / a.group_lanes;
    int place = 0;
    for (int g = 0; g < a.G; ++g) {
      const double w = __shfl_sync(kFull, worth, g * a.group_lanes);
      place += (w > worth || (w == worth && g < mine)) ? 1 : 0;
    }
    kept = __ballot_sync(kFull, place < a.keep);
  }
  const bool in = (kept >> lane) & 1u;
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    // best of this lane by level, rank, expert
    int level = -1, id = 0x7fffffff;
    double v = kNone;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (!((live >> i) & 1u)) continue;
      const int e = s_exp[lane * PL + i];
      const int lv = !in ? 0 : ((off >> i) & 1u) ? 1 : 2;
      const double r = lv == 2 ? (a.bias ? s[i] : static_cast<double>(z[i])) : kNone;
      if (lv > level || (lv == level && (r > v || (r == v && e < id)))) { level = lv; v = r; id = e; }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const int lv = __shfl_xor_sync(kFull, level, o);
      const double r = __shfl_xor_sync(kFull, v, o);
      const int e = __shfl_xor_sync(kFull, id, o);
      if (lv > level || (lv == level && (r > v || (r == v && e < id)))) { level = lv; v = r; id = e; }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (s_exp[lane * PL + i] == id) live &= ~(1u << i);
    if (lane == j) mine = id;
  }
  return mine;
}

template <int PL>
__device__ __forceinline__ void cas(uint32_t (&v)[PL], int i, int j) {
  const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
  v[i] = hi;
  v[j] = lo;
}
// A lane's words in descending order (odd-even merge networks).
template <int PL>
__device__ __forceinline__ void sort_down(uint32_t (&v)[PL]) {
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

template <bool SIG, int PL>
__global__ void __launch_bounds__(kWarps * 32)
route_scored_kernel(const RouteArgs a) {
  __shared__ int s_dev[OCCULT_MAX_EXPERTS], s_exp[PL * 32];
  __shared__ float s_bias[OCCULT_MAX_EXPERTS], s_span[2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the experts of every lane's places, and the bias's span
  for (int e = tid; e < a.Ne; e += blockDim.x) {
    s_dev[e] = a.e2v[e] & 31;
    s_bias[e] = a.bias ? a.bias[e] : 0.f;
  }
  for (int i = tid; i < PL * 32; i += blockDim.x) {
    const int g = i / PL / a.group_lanes, j = i - g * a.group_lanes * PL;
    s_exp[i] = !a.vdev_groups && g < a.G && j < a.per ? g * a.per + j : -1;
  }
  __syncthreads();
  if (a.vdev_groups)
    for (int e = tid; e < a.Ne; e += blockDim.x) {
      const int g = s_dev[e];
      int j = 0;
      for (int f = 0; f < e; ++f) j += s_dev[f] == g ? 1 : 0;
      if (g < a.G && j < a.per) s_exp[g * a.group_lanes * PL + j] = e;
    }
  if (a.bias && warp == 0) {
    float lo = 3e38f, hi = -3e38f;
    for (int e = lane; e < a.Ne; e += 32) {
      const float b = s_bias[e];
      if (fabsf(b) < 1e30f) { lo = fminf(lo, b); hi = fmaxf(hi, b); }
    }
    lo = -warp_max(-lo);
    hi = warp_max(hi);
    if (lane == 0) { s_span[0] = fminf(lo, hi); s_span[1] = fmaxf(hi, lo); }
  }
  __syncthreads();
  int ex[PL];
  float b[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    ex[i] = s_exp[lane * PL + i];
    b[i] = ex[i] >= 0 ? s_bias[ex[i]] : 0.f;
  }
  // ranks with a bias lie in [base, base + span]; a word holds them in 2^23 steps
  const float base = a.bias ? s_span[0] : 0.f, span = a.bias ? 1.f + (s_span[1] - s_span[0]) : 1.f;
  const float q_mul = 8388607.f / span;
  // A score made with ex2 and rcp is within 2^-21 of itself (|z| <= 16; beyond that its
  // distance from 0 or 1 is), the sum with the bias within 2^-24 of the rank's size, the
  // step adds its half: two ranks further apart than this many steps are in order.  (A
  // softmax's total errs by some 2^-20 as well, for all of its scores alike.)
  const float slack = (SIG ? 0x1p-20f : 0x1p-19f) + 0x1p-23f * fmaxf(fabsf(base), fabsf(base + span));
  const uint32_t near = static_cast<uint32_t>(fminf(slack * q_mul, 8388606.f)) + 2u;
  const int my_group = lane / a.group_lanes;

  for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
    const float* row = a.logits + static_cast<size_t>(t) * a.Ne;
    float z[PL], s[PL];
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
    float top = 0.f, total = 1.f;
    const bool scored = a.bias || a.G > 1;   // else the logits alone choose
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
      const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] *= inv;
    } else if (scored) {
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] = rcp(1.f + ex2(z[i] * -kLog2e));
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) s[i] = 0.f;
    }

    bool in = true, exact = false;
    if (a.G > 1) {
      float b1 = kLowest, b2 = kLowest;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        float r = s[i] + b[i];
        r = is_off(z[i]) ? kLowest : r == r ? r : OCCULT_NEG_INF;
        b2 = fmaxf(b2, fminf(b1, r));
        b1 = fmaxf(b1, r);
      }
      for (int o = 1; o < a.group_lanes; o <<= 1) {
        const float c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
        b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
        b1 = fmaxf(b1, c1);
      }
      const float worth = a.best == 2 && b2 > kLowest ? b1 + b2 : b1;
      int place = 0;
      float gap = 3e38f;   // to the nearest other worth
      for (int g = 0; g < a.G; ++g) {
        const float w = __shfl_sync(kFull, worth, g * a.group_lanes);
        place += (w > worth || (w == worth && g < my_group)) ? 1 : 0;
        if (g != my_group) gap = fminf(gap, fabsf(w - worth));
      }
      in = place < a.keep;
      // the last group kept: within the scores' error of a neighbour (two groups without
      // an expert are equal exactly)
      exact = __any_sync(kFull, my_group < a.G && a.keep < a.G && place == a.keep - 1 &&
                                    worth > kLowest && gap <= 2.f * slack + 0x1p-22f * fabsf(worth));
    }

    int my_id = 0;
    if (!exact) {
      uint32_t key[PL];
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const uint32_t low = 255u - static_cast<uint32_t>(ex[i]);
        uint32_t q;
        if (a.bias) {
          const float r = s[i] + b[i];
          q = __float_as_uint(fminf(fmaxf(fmaf(r - base, q_mul, 8388608.f), 8388608.f), 16777215.f)) & 0x7fffffu;
        } else {
          q = order_bits(z[i]) >> 9;
        }
        key[i] = ex[i] < 0 ? 0u : !in ? kOut | low : is_off(z[i]) ? kOff | low : kOn | (q << 8) | low;
      }
      sort_down<PL>(key);
      // the first k + 1 (at most 32, at most all): lane j keeps place j
      const int rounds = min(min(a.k + 1, a.Ne), 32);
      uint32_t mine = 0;
      auto draw = [&](int j) {
        const uint32_t w = __reduce_max_sync(kFull, key[0]);
        if (key[0] == w) {
#pragma unroll
          for (int i = 0; i + 1 < PL; ++i) key[i] = key[i + 1];
          key[PL - 1] = 0;
        }
        if (lane == j) mine = w;
      };
      for (int j = 0; j < rounds; ++j) draw(j);
      my_id = 255 - static_cast<int>(mine & 255u);
      // A place not clearly above the next: the same logit under the same bias is a tie
      // (the lower expert stands first already), others are looked at closely.
      const uint32_t gap_max = a.bias ? near : 0u;
      const int n_exp = a.Ne;
      bool on = lane < rounds && mine >= kOn;
      float cz = on ? row[my_id] : 0.f, cb = on ? s_bias[my_id] : 0.f;
      auto close = [&]() -> bool {   // of this lane's place and the next
        const uint32_t nxt = __shfl_down_sync(kFull, mine, 1);
        const float nz = __shfl_down_sync(kFull, cz, 1), nb = __shfl_down_sync(kFull, cb, 1);
        return lane < 31 && mine >= kOn && nxt >= kOn && (mine >> 8) - (nxt >> 8) <= gap_max &&
               !(cz == nz && cb == nb);
      };
      if (__any_sync(kFull, close() && lane < a.k)) {
        // more places until one is clearly below (a tie counts as not clear here)
        int have = rounds;
        while (have < min(n_exp, 32)) {
          const uint32_t last = __shfl_sync(kFull, mine, have - 1), prev = __shfl_sync(kFull, mine, have - 2);
          if (last < kOn || (prev >> 8) - (last >> 8) > gap_max) break;
          draw(have++);
        }
        const uint32_t last = __shfl_sync(kFull, mine, have - 1), prev = __shfl_sync(kFull, mine, max(0, have - 2));
        if ((a.bias && !SIG) || (have == 32 && n_exp > 32 && last >= kOn && (prev >> 8) - (last >> 8) <= gap_max)) {
          exact = true;   // (a softmax's total in fp64 takes every expert)
        } else {
          my_id = 255 - static_cast<int>(mine & 255u);
          on = lane < have && mine >= kOn;
          cz = on ? row[my_id] : 0.f;
          // the rank in fp64; lanes that hold no place, or one switched off, stay behind
          double r = -1e305;
          if (on) {
            r = static_cast<double>(cz);
            if (a.bias) {
              r = 1. / (1. + exp(-r)) + static_cast<double>(s_bias[my_id]);
              if (r != r || r < -1e300) r = -1e301;
            }
          }
          int place = 0;
          for (int j = 0; j < have; ++j) {
            const double o = __shfl_sync(kFull, r, j);
            const int e = __shfl_sync(kFull, my_id, j);
            const bool other_on = __shfl_sync(kFull, static_cast<int>(on), j);
            place += on ? (other_on && (o > r || (o == r && e < my_id)) ? 1 : 0) : (j < lane ? 1 : 0);
          }
          // (places behind the ones that are on keep their order)
          int sorted = 0;
          for (int j = 0; j < have; ++j) {
            const int at = __shfl_sync(kFull, place, j), e = __shfl_sync(kFull, my_id, j);
            if (at == lane) sorted = e;
          }
          my_id = sorted;
        }
      }
    }
    if (exact) my_id = choose_exactly<SIG, PL>(a, row, s_exp);
    if (my_id < 0 || my_id >= a.Ne) my_id = 0;   // (devices that do not share the experts evenly)

    float g = lane < a.k ? score_of<SIG>(row[my_id], top, total) : 0.f;
    if (a.renorm) {
      const float sum = warp_sum(g);
      g = sum == 0.f ? 0.f : g / sum;
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
// (softmax) the common term of every expert, and written as it lies.
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
  for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
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
    float ds = u;
    if (renorm) {
      const float S = warp_sum(s);
      const float us = warp_sum(u * s);
      ds = S == 0.f || id < 0 ? 0.f : (u - us / S) / S;
    }
    const float all = SIG ? 0.f : warp_sum(ds * s);
#pragma unroll
    for (int i = 0; i < PL; ++i) sm[lane + 32 * i] = 0.f;
    __syncwarp();
    // (two slots of one expert, which the router does not write, add up)
    if (id >= 0) atomicAdd(&sm[id], SIG ? ds * s * (1.f - s) : ds);
    __syncwarp();
    float* out = dlogits + static_cast<size_t>(t) * Ne;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < Ne) out[e] = SIG ? sm[e] : score_of<SIG>(z[i], top, total) * (sm[e] - all);
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

int blocks_for(const LaunchCtx& ctx, int T) {
  const int blocks = (T + kWarps - 1) / kWarps;
  return blocks < ctx.num_sms * 8 ? blocks : ctx.num_sms * 8;
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
  const int need = (a.per + a.group_lanes - 1) / a.group_lanes;   // experts a lane: at most 15
  // whole fours of a row: consecutive experts, none cut off, rows on 16 bytes
  a.vec = !a.vdev_groups && a.per % 4 == 0 && a.Ne % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0;
  const bool sig = opt.score == OCCULT_SCORE_SIGMOID;
  const int nb = blocks_for(ctx, ds.T);
#define OCCULT_SCORED(PL) \
  cuda_status(launch_pdl(sig ? route_scored_kernel<true, PL> : route_scored_kernel<false, PL>, nb, \
                         kWarps * 32, 0, ctx.stream, a))
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
  const int nb = blocks_for(ctx, ds.T);
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
