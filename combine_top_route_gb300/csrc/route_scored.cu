// The scored router: softmax or sigmoid scores, a bias on the choice, groups of
// experts, the top k of the kept groups, their gates and the gradient.
//
// One warp a token; lane l holds experts l, l + 32, ... (up to eight).  The choice is
// a comparison of ranks s + b, and s is a rounded exponential: two ranks nearer to
// each other than the rounding could change places from one machine to the next.  So
// the warp also finds the gap to the next rank of every place of the list (and of the
// worths at the border of the kept groups); a gap that fp32 cannot vouch for sends
// that token, and no other, through the same choice in fp64.
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kLowest = -3.402823466e+38f;   // a logit as low as this is switched off

// Keys that order as the floats do, above the levels of experts that are no choice:
// 2 switched off, 1 in no kept group, 0 taken.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);       // -0 orders as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;   // -inf: 0x007fffff
}
constexpr uint32_t kKeyOff = 2, kKeyOut = 1, kKeyTaken = 0;

// s + b, a NaN below every number
__device__ __forceinline__ float rank_of(float s, float b) {
  const float r = s + b;
  return r == r ? r : -__int_as_float(0x7f800000);
}

__device__ __forceinline__ bool is_off(float z) { return !(z > kLowest); }  // NaN too

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

struct RouteArgs {
  const float* logits;
  const float* bias;
  const int32_t* e2v;
  int32_t* ids;
  float* gates;
  uint32_t* vmask;
  int T, Ne, k, G, keep, best, vdev_groups, renorm;
  float scale;
};

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

template <bool SIG>
__device__ __forceinline__ float score_of(float z, float top, float total) {
  if (z <= kLowest) return 0.f;
  return SIG ? 1.f / (1.f + expf(-z)) : expf(z - top) / total;
}

// The choice in fp64 (one token): same rules, ranks and worths as doubles.  Returns
// slot `lane`'s expert.  `sm`: Ne doubles of this warp.
template <bool SIG, int PL>
__device__ __noinline__ int choose_exactly(const RouteArgs& a, const float* row, const int* s_grp,
                                           double* sm) {
  const int lane = threadIdx.x & 31;
  double s[PL];
  uint32_t off = 0;
  double top = -1e300, total = 0.;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    const float z = e < a.Ne ? row[e] : kLowest;
    if (is_off(z)) off |= 1u << i;
    s[i] = static_cast<double>(z);
    if (!is_off(z)) top = fmax(top, s[i]);
  }
  if (SIG) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = 1. / (1. + exp(-s[i]));
  } else {
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = ((off >> i) & 1u) ? 0. : exp(s[i] - top);
      total += s[i];
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] /= total;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    if (a.bias && e < a.Ne) s[i] += static_cast<double>(a.bias[e]);
    if (s[i] != s[i]) s[i] = static_cast<double>(-__int_as_float(0x7f800000));
  }
  const double kNone = -1e300;   // below every rank of finite biases
  uint32_t live = 0;             // bit i: expert lane + 32 i may be chosen
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (lane + 32 * i < a.Ne) live |= 1u << i;
  uint32_t kept = kFull;
  if (a.G > 1) {
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i < a.Ne) sm[lane + 32 * i] = ((off >> i) & 1u) ? kNone : s[i];
    __syncwarp();
    double b1 = kNone, b2 = kNone;
    for (int e = 0; e < a.Ne; ++e)
      if (s_grp[e] == lane) {
        const double v = sm[e];
        if (v > b1) { b2 = b1; b1 = v; } else if (v > b2) b2 = v;
      }
    double worth = a.best == 2 && b2 > kNone ? b1 + b2 : b1;
    // as multiples of 2^-48: sums that the formula makes equal, as sigmoid(x) +
    // sigmoid(-x) = 1 for every x, then do not hang on the last bits of exp
    if (fabs(worth) < 256.) worth = rint(worth * 0x1p48) * 0x1p-48;
    int place = 0;
    for (int g = 0; g < a.G; ++g) {
      const double w = __shfl_sync(kFull, worth, g);
      place += (w > worth || (w == worth && g < lane)) ? 1 : 0;
    }
    kept = __ballot_sync(kFull, lane < a.G && place < a.keep);
    __syncwarp();
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    // best of this lane by level, rank, id
    int level = -1, id = 0x7fffffff;
    double v = kNone;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (!((live >> i) & 1u)) continue;
      const int e = lane + 32 * i;
      const int lv = !((kept >> s_grp[e]) & 1u) ? 0 : ((off >> i) & 1u) ? 1 : 2;
      const double r = lv == 2 ? (a.bias ? s[i] : static_cast<double>(row[e])) : kNone;
      if (lv > level || (lv == level && r > v)) { level = lv; v = r; id = e; }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const int lv = __shfl_xor_sync(kFull, level, o);
      const double r = __shfl_xor_sync(kFull, v, o);
      const int e = __shfl_xor_sync(kFull, id, o);
      if (lv > level || (lv == level && (r > v || (r == v && e < id)))) { level = lv; v = r; id = e; }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 32 * i == id) live &= ~(1u << i);
    if (lane == j) mine = id;
  }
  return mine;
}

template <bool SIG, int PL>
__global__ void __launch_bounds__(kWarps * 32)
route_scored_kernel(const RouteArgs a) {
  __shared__ int s_dev[PL * 32], s_grp[PL * 32];
  __shared__ double s_buf[kWarps][PL * 32];
  pdl_wait();
  pdl_trigger();
  const int per = a.Ne / a.G;
  for (int e = threadIdx.x; e < PL * 32; e += blockDim.x) {
    s_dev[e] = e < a.Ne ? a.e2v[e] & 31 : 0;
    s_grp[e] = e < a.Ne ? (a.G == 1 ? 0 : a.vdev_groups ? s_dev[e] : e / per) : 31;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  float b[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i)
    b[i] = a.bias && lane + 32 * i < a.Ne ? a.bias[lane + 32 * i] : 0.f;

  for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
    const float* row = a.logits + static_cast<size_t>(t) * a.Ne;
    float z[PL], s[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) z[i] = lane + 32 * i < a.Ne ? row[lane + 32 * i] : kLowest;
    float top = 0.f, total = 1.f;
    if (!SIG) softmax_stats<PL>(z, a.Ne, top, total);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = score_of<SIG>(z[i], top, total);

    bool unsure = false;
    uint32_t kept = kFull;
    if (a.G > 1) {
      float* sm = reinterpret_cast<float*>(s_buf[warp]);
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i < a.Ne) sm[lane + 32 * i] = is_off(z[i]) ? kLowest : rank_of(s[i], b[i]);
      __syncwarp();
      // lane g finds its group's best two
      float b1 = kLowest, b2 = kLowest;
      if (a.vdev_groups) {
        for (int e = 0; e < a.Ne; ++e)
          if (s_grp[e] == lane) {
            const float v = sm[e];
            b2 = fmaxf(b2, fminf(b1, v));
            b1 = fmaxf(b1, v);
          }
      } else if (lane < a.G) {
        int j = lane % per;   // a start of its own: no two groups on one bank
        for (int n = 0; n < per; ++n) {
          const float v = sm[lane * per + j];
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
          if (++j == per) j = 0;
        }
      }
      const float worth = a.best == 2 && b2 > kLowest ? b1 + b2 : b1;
      int place = 0;
      for (int g = 0; g < a.G; ++g) {
        const float w = __shfl_sync(kFull, worth, g);
        place += (w > worth || (w == worth && g < lane)) ? 1 : 0;
      }
      kept = __ballot_sync(kFull, lane < a.G && place < a.keep);
      // the border of the kept groups: the last kept and the first left out
      const uint32_t last = __ballot_sync(kFull, lane < a.G && place == a.keep - 1);
      const uint32_t next = __ballot_sync(kFull, lane < a.G && place == a.keep);
      if (next && last) {
        const float w0 = __shfl_sync(kFull, worth, __ffs(last) - 1);
        const float w1 = __shfl_sync(kFull, worth, __ffs(next) - 1);
        // scores are at most 1, so that the sum of two with their biases is within
        // 2^-20 (2 + |worth|) of itself; two empty groups are equal exactly
        if (w1 > kLowest && w0 - w1 <= 0x1p-20f * (2.f + fabsf(w0) + fabsf(w1))) unsure = true;
      }
      __syncwarp();
    }

    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      key[i] = e >= a.Ne ? kKeyTaken
             : !((kept >> s_grp[e]) & 1u) ? kKeyOut
             : is_off(z[i]) ? kKeyOff : order_key(a.bias ? rank_of(s[i], b[i]) : z[i]);
    }
    int my_id = 0;
    // with a bias one place more than k: the gap below the last one counts as well
    const int rounds = a.bias && a.k < a.Ne ? a.k + 1 : a.k;
    float pr = 0.f, ps = 0.f, pz = 0.f, pb = 0.f;   // the place before: rank, score, logit, bias
    for (int j = 0; j < rounds; ++j) {
      uint32_t kb = kKeyTaken;
      int ib = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (key[i] > kb) { kb = key[i]; ib = lane + 32 * i; }
      const uint32_t kw = __reduce_max_sync(kFull, kb);
      const int id = __reduce_min_sync(kFull, kb == kw ? ib : 0x7fffffff);
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i == id) key[i] = kKeyTaken;
      if (lane == j) my_id = id;
      if (a.bias) {
        const int owner = id & 31;
        float cz = 0.f, cs = 0.f, cb = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i)
          if ((id >> 5) == i) { cz = z[i]; cs = s[i]; cb = b[i]; }
        cz = __shfl_sync(kFull, cz, owner);
        cs = __shfl_sync(kFull, cs, owner);
        cb = __shfl_sync(kFull, cb, owner);
        const float cr = cs + cb;
        // expf, 1 + e and the division leave a score within 4 units of 2^-24, the
        // argument's rounding |z| units more, the sum one of the rank: 2^-20 covers
        // both sides.  The same logit under the same bias is a tie in fp64 as well.
        if (j > 0 && kw > kKeyOff && pr - cr <= 0x1p-20f * ((ps + cs) * (1.f + 0.125f * fabsf(SIG ? cz : cz - top)) + fabsf(pr) + fabsf(cr)) &&
            !(pz == cz && pb == cb))
          unsure = true;
        pr = cr; ps = cs; pz = cz; pb = cb;
      }
    }
    if (unsure) my_id = choose_exactly<SIG, PL>(a, row, s_grp, s_buf[warp]);

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

#define OCCULT_SCORED_LAUNCH(KERNEL, ...)                                                        \
  do {                                                                                           \
    const int nb_ = blocks_for(ctx, ds.T);                                                       \
    const bool sig_ = opt.score == OCCULT_SCORE_SIGMOID;                                         \
    cudaError_t e_;                                                                              \
    if (ds.n_experts <= 32)                                                                      \
      e_ = launch_pdl(sig_ ? KERNEL<true, 1> : KERNEL<false, 1>, nb_, kWarps * 32, 0, ctx.stream, __VA_ARGS__); \
    else if (ds.n_experts <= 64)                                                                 \
      e_ = launch_pdl(sig_ ? KERNEL<true, 2> : KERNEL<false, 2>, nb_, kWarps * 32, 0, ctx.stream, __VA_ARGS__); \
    else if (ds.n_experts <= 128)                                                                \
      e_ = launch_pdl(sig_ ? KERNEL<true, 4> : KERNEL<false, 4>, nb_, kWarps * 32, 0, ctx.stream, __VA_ARGS__); \
    else                                                                                         \
      e_ = launch_pdl(sig_ ? KERNEL<true, 8> : KERNEL<false, 8>, nb_, kWarps * 32, 0, ctx.stream, __VA_ARGS__); \
    return cuda_status(e_);                                                                      \
  } while (0)

int launch_route_scored(const LaunchCtx& ctx, const occult_desc_t& ds, const occult_score_t& opt,
                        const float* logits, const float* bias, const int32_t* e2v, int32_t* ids,
                        float* gates, uint32_t* vmask) {
  if (ds.T == 0) return OCCULT_OK;
  RouteArgs a{};
  a.logits = logits; a.bias = bias; a.e2v = e2v;
  a.ids = ids; a.gates = gates; a.vmask = vmask;
  a.T = ds.T; a.Ne = ds.n_experts; a.k = ds.top_k;
  a.G = opt.n_groups; a.keep = opt.keep_groups; a.best = opt.group_best;
  a.vdev_groups = opt.group_kind == OCCULT_GROUP_VDEV; a.renorm = ds.renorm; a.scale = opt.scale;
  OCCULT_SCORED_LAUNCH(route_scored_kernel, a);
}

int launch_route_scored_grad(const LaunchCtx& ctx, const occult_desc_t& ds,
                             const occult_score_t& opt, const float* logits, const int32_t* ids,
                             const float* dgates, float* dlogits) {
  if (ds.T == 0) return OCCULT_OK;
  OCCULT_SCORED_LAUNCH(route_scored_grad_kernel, logits, ids, dgates, dlogits, ds.T, ds.n_experts,
                       ds.top_k, ds.renorm, opt.scale);
}

int launch_route_bias_step(const LaunchCtx& ctx, int Ne, const int32_t* counts, int G, float rate,
                           float* bias) {
  return cuda_status(launch_pdl(bias_step_kernel, 1, OCCULT_MAX_EXPERTS, 0, ctx.stream, counts, G,
                                Ne, rate, bias));
}

}  // namespace occult
