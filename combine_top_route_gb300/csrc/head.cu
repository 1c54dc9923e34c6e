// The output head: everything around its products.
//
// A call goes: rows (which tokens a term counts, compacted) -> entries (each row's label
// and teacher tokens, sorted by id, with the teacher's probabilities) -> the product with
// its maxima, sums and entries' logits -> the rows' losses and their means -> (step) the
// gradient of the logits, put together from the kept logits -> dx and dw.
//
// Softmax over the vocabulary is done in powers of two: y = z log2(e), and with m the
// maximum of a row's part, sum 2^(y - m); the parts of a row (128 columns each) are
// joined at the end.  The gradient of a logit is then
//   dz_v = k1 2^(y_v - L) + k2 2^(y_v / tau - L') - (at the entries) their factors,
// L and L' the rows' log2 of the sums at temperature 1 and tau.  Its common factor
// (coef / N) is left to the fp32 sums of dx and dw.
#include <algorithm>

#include "head.h"
#include "kernels.h"

namespace occult {

namespace {

// ---- entries ----------------------------------------------------------------------
// A warp makes a row's entries: the teacher's probabilities at temperature tau, and the
// label (q = -1), in ascending token order, absent ones behind.  Returns whether the
// teacher says anything.  `ids`: 128 words of the warp's own, on 16 bytes.
// A lane has every 32nd teacher entry; an entry's place is the number of those in front of it.
constexpr int kEntPer = OCCULT_MAX_TEACHER / 32;
__device__ __forceinline__ bool make_entries(const int32_t* __restrict__ t_ids, const float* __restrict__ t_logits,
                                             int t, int f, int label, int V, int K, float inv_tau, uint32_t* ids,
                                             int32_t* __restrict__ ent, float* __restrict__ ent_q) {
  const int lane = threadIdx.x & 31;
  const float NEG = -__int_as_float(0x7f800000);
  int id[kEntPer];
  float q[kEntPer];
  float top = NEG;
#pragma unroll
  for (int i = 0; i < kEntPer; ++i) {
    const int j = lane + 32 * i;
    id[i] = kHeadNoEntry;
    q[i] = NEG;
    if (j < K && (f & kRowKd)) {
      const size_t at = static_cast<size_t>(t) * K + j;
      const int v = t_ids[at];
      const float l = t_logits[at] * inv_tau;
      if (static_cast<unsigned>(v) < static_cast<unsigned>(V)) {
        id[i] = v;
        q[i] = l;
        top = fmaxf(top, l);
      }
    }
  }
  top = warp_max(top);
  if (top == NEG) top = 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kEntPer; ++i) {
    q[i] = id[i] == kHeadNoEntry ? 0.f : expf(q[i] - top);
    sum += q[i];
  }
  sum = warp_sum(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kEntPer; ++i) {
    const int j = lane + 32 * i;
    q[i] *= inv;
    // (places behind the K hold what stands behind every entry)
    ids[j] = j < K ? static_cast<uint32_t>(id[i]) : 0xffffffffu;
  }
  __syncwarp();
  const uint32_t own = (f & kRowCe) ? label : kHeadNoEntry;
  uint32_t rank[kEntPer], before = 0;   // before: entries in front of the label, the equal ones too
#pragma unroll
  for (int i = 0; i < kEntPer; ++i) {
    rank[i] = own < static_cast<uint32_t>(id[i]) ? 1 : 0;
    before += __popc(__ballot_sync(kFull, lane + 32 * i < K && static_cast<uint32_t>(id[i]) <= own));
  }
#pragma unroll
  for (int b = 0; b < kEntPer; ++b) {
    if (32 * b >= K) break;
#pragma unroll 4
    for (int k = 0; k < 32; k += 4) {
      const uint4 four = *reinterpret_cast<const uint4*>(ids + 32 * b + k);
      const uint32_t other[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < kEntPer; ++i)
          // equal ones in their order: those of a smaller number stand in front
          if (32 * i < K)
            rank[i] += other[j] < static_cast<uint32_t>(id[i]) + (b < i || (b == i && k + j < lane) ? 1u : 0u) ? 1 : 0;
    }
  }
#pragma unroll
  for (int i = 0; i < kEntPer; ++i)
    if (lane + 32 * i < K) {
      ent[rank[i]] = id[i];
      ent_q[rank[i]] = q[i];
    }
  if (lane == 0) {
    ent[before] = static_cast<int32_t>(own);
    ent_q[before] = -1.f;
  }
  __syncwarp();
  return sum != 0.f;
}

// ---- rows -----------------------------------------------------------------------
// Which tokens a term counts, and their compact rows in token order.  A block has `per`
// tokens of its own and counts all of them, from labels and teacher ids themselves where
// those are few KB for every block, else from the tallies of a launch of its own
// (head_tally_kernel): those before its own give its first row, all of them the totals.
// Where some token is left out, the rows of x are copied to their compact place on the way
// (else the products read x itself), with zeros up to the next multiple of 64, so that
// dw's reduction may run over them; and that token's outputs are zeros.  With a teacher a
// warp then makes the entries of its tokens' rows.
constexpr int kRowThreads = 256;
// What a token is to the loss.
__device__ __forceinline__ int token_flag(const int32_t* __restrict__ labels, const int32_t* __restrict__ t_ids,
                                          int t, int V, int K) {
  int f = 0;
  if (labels && static_cast<unsigned>(labels[t]) < static_cast<unsigned>(V)) f |= kRowCe;
  if (K && static_cast<unsigned>(t_ids[static_cast<size_t>(t) * K]) < static_cast<unsigned>(V)) f |= kRowKd;
  return f;
}
// Tallies of 256 tokens each: counted, with a label, with a teacher.
__global__ void __launch_bounds__(kRowThreads)
head_tally_kernel(const int32_t* __restrict__ labels, const int32_t* __restrict__ t_ids, int T, int V, int K,
                  int4* __restrict__ tally) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * kRowThreads + threadIdx.x;
  const int f = t < T ? token_flag(labels, t_ids, t, V, K) : 0;
  const int n = __syncthreads_count(f != 0), ce = __syncthreads_count(f & kRowCe);
  const int kd = __syncthreads_count(f & kRowKd);
  if (threadIdx.x == 0) tally[blockIdx.x] = make_int4(n, ce, kd, 0);
}
__global__ void __launch_bounds__(kRowThreads)
head_rows_kernel(const int32_t* __restrict__ labels, const int32_t* __restrict__ t_ids,
                 const float* __restrict__ t_logits, int T, int V, int K, float inv_tau, int per,
                 HeadCounts* cnt, int32_t* __restrict__ idx, uint8_t* __restrict__ flag,
                 int32_t* __restrict__ ent, float* __restrict__ ent_q, float* __restrict__ lse,
                 float* __restrict__ token_loss, const uint4* __restrict__ x, uint4* __restrict__ xc, int vecs,
                 char* __restrict__ dx, int dx_bytes, const int4* __restrict__ tally) {
  __shared__ __align__(16) uint32_t s_ids[kRowThreads / 32][32 * kEntPer];
  __shared__ int s_sum[4][kRowThreads / 32], s_warp[kRowThreads / 32], s_pos[kRowThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = min(T, static_cast<int>(blockIdx.x) * per), t1 = min(T, t0 + per);
  auto flag_of = [&](int t) { return token_flag(labels, t_ids, t, V, K); };
  int sum[4] = {0, 0, 0, 0};   // rows before this block's, rows, with a label, with a teacher
  if (tally) {
    const int whole = t0 / kRowThreads;   // tallies before this block's tokens
#pragma unroll 4
    for (int i = tid; i < (T + kRowThreads - 1) / kRowThreads; i += kRowThreads) {
      const int4 c = tally[i];
      sum[0] += i < whole ? c.x : 0;
      sum[1] += c.x;
      sum[2] += c.y;
      sum[3] += c.z;
    }
    if (whole * kRowThreads + tid < t0) sum[0] += flag_of(whole * kRowThreads + tid) != 0 ? 1 : 0;
  } else {
#pragma unroll 8
    for (int t = tid; t < T; t += kRowThreads) {
      const int f = flag_of(t);
      sum[0] += (f != 0 && t < t0) ? 1 : 0;
      sum[1] += f != 0 ? 1 : 0;
      sum[2] += (f & kRowCe) ? 1 : 0;
      sum[3] += (f & kRowKd) ? 1 : 0;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = __reduce_add_sync(kFull, sum[i]);
    if (lane == 0) s_sum[i][warp] = v;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) sum[i] += s_sum[i][w];
  }
  const int n = sum[1];
  if (blockIdx.x == 0 && tid == 0) {
    cnt->n = n;
    cnt->n_ce = sum[2];
    cnt->n_kd = sum[3];
    cnt->ticket = 0;
    cnt->stretch = 1.f;
  }
  const bool copy = n < T;
  int row = sum[0];   // first row of the block's next tokens
  for (int base = t0; base < t1; base += kRowThreads) {
    const int t = base + tid;
    const int f = t < t1 ? flag_of(t) : 0;
    const unsigned on = __ballot_sync(kFull, f != 0);
    if (lane == 0) s_warp[warp] = __popc(on);
    __syncthreads();
    int r = row + __popc(on & lanemask_lt()), all = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) {
      if (w < warp) r += s_warp[w];
      all += s_warp[w];
    }
    s_pos[tid] = f ? r : -1;
    if (t < t1) {
      if (f) {
        idx[r] = t;
        flag[r] = static_cast<uint8_t>(f);
        if (K == 0) {   // the label is a row's only entry
          ent[r] = labels[t];
          ent_q[r] = -1.f;
        }
      } else {
        if (lse) lse[t] = 0.f;
        if (token_loss) token_loss[t] = 0.f;
      }
    }
    __syncthreads();
    for (int i = warp; i < min(kRowThreads, t1 - base); i += kRowThreads / 32) {
      const int to = s_pos[i], ti = base + i;
      if (to < 0) {
        // (rows of 8 bytes at least)
        if (dx)
          for (int v = lane * 8; v < dx_bytes; v += 256)
            *reinterpret_cast<uint2*>(dx + static_cast<size_t>(ti) * dx_bytes + v) = make_uint2(0, 0);
        continue;
      }
      if (copy) {
        const uint4* src = x + static_cast<size_t>(ti) * vecs;
        uint4* dst = xc + static_cast<size_t>(to) * vecs;
#pragma unroll 4
        for (int v = lane; v < vecs; v += 32) dst[v] = src[v];
      }
      if (K) {
        const int fi = flag_of(ti);
        const size_t at = static_cast<size_t>(to) * (K + 1);
        const bool says = make_entries(t_ids, t_logits, ti, fi, labels ? labels[ti] : 0, V, K, inv_tau,
                                       s_ids[warp], ent + at, ent_q + at);
        // nothing to learn from: its term is 0, and so is its gradient
        if (!says && lane == 0) flag[to] = static_cast<uint8_t>(fi & ~kRowKd);
      }
    }
    row += all;
    __syncthreads();
  }
  if (copy && blockIdx.x == gridDim.x - 1)
    for (size_t i = static_cast<size_t>(n) * vecs + tid; i < static_cast<size_t>((n + 63) & ~63) * vecs;
         i += kRowThreads)
      xc[i] = make_uint4(0, 0, 0, 0);
}

// ---- the gradient's scalars ---------------------------------------------------------
struct DzArgs {
  const HeadCounts* cnt;
  const float *pk, *tops, *l1, *l2;
  const uint8_t* flag;
  int ldp, row0, piece, V, ld;
  float inv_tau, q_step, coef, coef_kd, coef_z, tau;
  bool two;
};
// A row's factors of the two softmaxes.
__device__ __forceinline__ void row_factors(const DzArgs& a, const HeadScale& sc, int f, float L,
                                            float& k1, float& k2) {
  k1 = ((f & kRowCe) ? sc.k_ce : 0.f) + sc.k_z * (L * kLn2);
  k2 = (f & kRowKd) ? sc.k_kd : 0.f;
  if (!a.two) {   // one softmax for both
    k1 += k2;
    k2 = 0.f;
  }
}
__device__ __forceinline__ HeadScale scale_of(const DzArgs& a) {
  return head_scale(a.cnt->n, a.cnt->n_ce, a.cnt->n_kd, a.coef, a.coef_kd, a.coef_z, a.tau, a.cnt->stretch);
}

// Gradient at entry e of row r, the first of its token: the softmaxes at the entry's own fp32
// logit, minus the factors of every entry of that token.
__device__ __forceinline__ float entry_dz(const DzArgs& a, const HeadScale& sc, const HeadLossOut& o, size_t at,
                                          int e, int id, float top, float l1, float l2, float k1, float k2) {
  const float y = over_top(o.zt[at], top);
  float g = k1 * exp2f(y - l1);
  if (a.two) g += k2 * exp2f(y * a.inv_tau - l2);
  for (int f = e; f < o.E && o.ent[at + f - e] == id; ++f) {
    const float q = o.ent_q[at + f - e];
    g -= q < 0.f ? sc.k_ce : sc.k_kd * q;
  }
  return g;
}

// ---- a row's sums, losses and the means ---------------------------------------------
// A block takes 32 rows: its warps join every so many parts of all of them (a lane a row,
// so that reads run along the rows), then finish the rows one by one.  The last block to
// arrive adds the blocks' sums in their order.  32 warps a block where there are few of
// them, 16 where two to an SM save a second round of blocks.
//
// TUNE (steps of bf16 layers): a row's warp also makes its entries' gradients and what each
// stretch's rounding to bf16 takes from them; the launch's last block picks the piece's.
template <bool TWO, int kSumWarps, bool TUNE>
__global__ void __launch_bounds__(kSumWarps * 32, 32 / kSumWarps)
head_sum_kernel(HeadCounts* cnt, const HeadLossOut o, const float* __restrict__ pm,
                const float* __restrict__ ps, const float* __restrict__ ps2, int ldp, int halves, int row0,
                int rows_max, const int32_t* __restrict__ idx, const uint8_t* __restrict__ flag,
                float* __restrict__ tops, float* __restrict__ l1, float* __restrict__ l2,
                float* __restrict__ sums, int block0,
                int n_blocks, const DzArgs z, float* __restrict__ tune) {
  static_assert(kSumWarps >= kStretches, "a warp a stretch");
  __shared__ float s_m[kSumWarps][33], s_s[kSumWarps][33], s_s2[kSumWarps][33];
  __shared__ float s_ce[32], s_kd[32], s_z[32];
  __shared__ float s_off[TUNE ? kSumWarps : 1][kStretches], s_all[kStretches];
  __shared__ bool s_last, s_pick;
  auto pick = [&] {   // the stretch of the least loss; 1 where none is less
    int best = 0;
    for (int j = 1; j < kStretches; ++j)
      if (s_all[j] < s_all[best]) best = j;
    cnt->stretch = exp2f(static_cast<float>(best) / kStretches);
  };
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = min(cnt->n - row0, rows_max);
  const int r_first = blockIdx.x * 32;
  const float NEG = -__int_as_float(0x7f800000);
  const float inv_tau = 1.f / o.tau;
  if (r_first < n) {
    // parts of row r_first + lane
    const int r = min(r_first + lane, n - 1);
    float m = NEG, s = 0.f, s2 = 0.f;
    constexpr int kAhead = TWO ? 6 : 8;   // parts in flight
    for (int h0 = warp; h0 < halves; h0 += kAhead * kSumWarps) {
      float vm[kAhead], vs[kAhead], vt[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = h0 + u * kSumWarps;
        const size_t at = static_cast<size_t>(h) * ldp + r;
        vm[u] = h < halves ? pm[at] : NEG;
        vs[u] = h < halves ? ps[at] : 0.f;
        vt[u] = TWO && h < halves ? ps2[at] : 0.f;
      }
      float hi = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) hi = fmaxf(hi, vm[u]);
      const float to = hi == NEG ? 0.f : hi;
      s *= ex2(m - to);
      if (TWO) s2 *= ex2((m - to) * inv_tau);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        s = fmaf(vs[u], ex2(vm[u] - to), s);
        if (TWO) s2 = fmaf(vt[u], ex2((vm[u] - to) * inv_tau), s2);
      }
      m = hi;
    }
    s_m[warp][lane] = m;
    s_s[warp][lane] = s;
    if (TWO) s_s2[warp][lane] = s2;
  }
  __syncthreads();
  RowSums mine{0.f, 0.f, 0.f};
  const HeadScale sc = head_scale(cnt->n, cnt->n_ce, cnt->n_kd, z.coef, z.coef_kd, z.coef_z, z.tau, 1.f);
  // a lane's stretch is number lane % 8; of 32 entries it takes every fourth
  static_assert(kStretches == 8, "four lanes a stretch");
  const float by = exp2f(static_cast<float>(lane % kStretches) / kStretches), shrink = 1.f / by;
  float off = 0.f;
  for (int own = warp; own < 32 && r_first + own < n; own += kSumWarps) {
    const size_t r = static_cast<size_t>(row0) + r_first + own;
    const float m = lane < kSumWarps ? s_m[lane][own] : NEG;
    const float top = warp_max(m);
    const float safe = top == NEG ? 0.f : top;
    const float a = log2f(warp_sum(lane < kSumWarps ? s_s[lane][own] * ex2(m - safe) : 0.f));
    float b = a;
    if (TWO) b = log2f(warp_sum(lane < kSumWarps ? s_s2[lane][own] * ex2((m - safe) * inv_tau) : 0.f));
    if (lane == 0) { tops[r] = safe; l1[r] = a; l2[r] = b; }
    const int f = flag[r];
    if (TUNE) {
      float k1, k2;
      row_factors(z, sc, f, safe + a, k1, k2);
      row_losses(o, r, f, idx[r], safe, a, b, inv_tau, mine, [&](int id, float q, float y) {
        // as entry_dz, of two entries of one token at most: a choice hangs on it, no result
        const float own = q < 0.f ? sc.k_ce : sc.k_kd * q;
        const int before = __shfl_up_sync(kFull, id, 1), next = __shfl_down_sync(kFull, id, 1);
        const float other = __shfl_down_sync(kFull, own, 1);
        float g = k1 * ex2(y - a) - own;
        if (TWO) g += k2 * ex2(y * inv_tau - b);
        if (lane < 31 && next == id) g -= other;
        if (id == kHeadNoEntry || (lane > 0 && before == id)) g = 0.f;
#pragma unroll 2
        for (int k = 0; k < min(32, o.E); k += 4) {
          const float v = __shfl_sync(kFull, g, k + lane / kStretches) * shrink;
          const float lost = __bfloat162float(__float2bfloat16_rn(v)) - v;
          off = fmaf(lost, lost, off);
        }
      });
    } else {
      row_losses(o, r, f, idx[r], safe, a, b, inv_tau, mine);
    }
  }
  if (TUNE) {
    off += __shfl_xor_sync(kFull, off, kStretches);
    off += __shfl_xor_sync(kFull, off, 2 * kStretches);
    if (lane < kStretches) s_off[warp][lane] = off * by * by;
  }
  if (lane == 0) { s_ce[warp] = mine.ce; s_kd[warp] = mine.kd; s_z[warp] = mine.z; }
  __syncthreads();
  const bool have = lane < kSumWarps;
  if (warp == 0) {
    const float a = warp_sum(have ? s_ce[lane] : 0.f), b = warp_sum(have ? s_kd[lane] : 0.f),
                c = warp_sum(have ? s_z[lane] : 0.f);
    if (TUNE && lane < kStretches) {
      float v = 0.f;
      for (int w = 0; w < kSumWarps; ++w) v += s_off[w][lane];
      if (gridDim.x == 1) s_all[lane] = v;
      else tune[kStretches * static_cast<size_t>(blockIdx.x) + lane] = v;
    }
    if (n_blocks > 1) {
      if (lane < 3) sums[3 * static_cast<size_t>(block0 + blockIdx.x) + lane] = lane == 0 ? a : lane == 1 ? b : c;
      __threadfence();
    }
    __syncwarp();
    if (lane == 0 && n_blocks == 1) {
      mean_losses(o, *cnt, a, b, c);   // a block alone
      s_last = s_pick = false;
    } else if (lane == 0) {
      const int before = static_cast<int>(atomicAdd(&cnt->ticket, 1u));
      s_last = before == n_blocks - 1;
      s_pick = gridDim.x > 1 && before == block0 + static_cast<int>(gridDim.x) - 1;
    }
    if (TUNE && lane == 0 && gridDim.x == 1) pick();
  }
  __syncthreads();
  if (!s_last && !s_pick) return;
  __threadfence();
  // every block of the launch (the call) is done: a warp adds a stretch's losses, and each thread
  // a run of the blocks' sums, then a tree
  float v = 0.f, a = 0.f, b = 0.f, c = 0.f;
  if (TUNE && s_pick && warp < kStretches)
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 32)
      v += __ldcg(tune + kStretches * static_cast<size_t>(i) + warp);
  if (s_last)
    for (int i = threadIdx.x; i < n_blocks; i += blockDim.x) {
      a += __ldcg(sums + 3 * static_cast<size_t>(i));
      b += __ldcg(sums + 3 * static_cast<size_t>(i) + 1);
      c += __ldcg(sums + 3 * static_cast<size_t>(i) + 2);
    }
  v = warp_sum(v);
  a = warp_sum(a); b = warp_sum(b); c = warp_sum(c);
  if (lane == 0) {
    s_ce[warp] = a; s_kd[warp] = b; s_z[warp] = c;
    if (TUNE && warp < kStretches) s_all[warp] = v;
  }
  __syncthreads();
  if (warp == 0) {
    a = warp_sum(have ? s_ce[lane] : 0.f);
    b = warp_sum(have ? s_kd[lane] : 0.f);
    c = warp_sum(have ? s_z[lane] : 0.f);
    if (lane == 0) {
      if (s_last) mean_losses(o, *cnt, a, b, c);
      if (TUNE && s_pick) pick();
    }
  }
}

// ---- gradient of the logits -----------------------------------------------------------
// bf16 layers: the kept 16-bit logits (units of q_step octaves below the largest of their
// 128 columns that is no entry, the last one for all that lies lower: no probability) become
// bf16 gradients where they lie.  A warp takes 16 rows of 128
// columns, 16 lanes a row's 256 bytes, all of its loads in flight at once.
constexpr int kDzRows = 16;
__global__ void __launch_bounds__(256)
head_dz_bf16_kernel(const DzArgs a, uint16_t* __restrict__ kept) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = min(a.cnt->n - a.row0, a.piece);
  const int h = blockIdx.x * 8 + warp;
  if (n <= 0 || h * 128 >= a.ld) return;
  const HeadScale sc = scale_of(a);
  const int rows = (n + kHeadRowAlign - 1) & ~(kHeadRowAlign - 1);
  const int c0 = h * 128 + (lane & 15) * 8;
  const bool edge = h * 128 + 128 > a.V;
  for (int r0 = blockIdx.y * kDzRows; r0 < rows; r0 += gridDim.y * kDzRows) {
    char* base = reinterpret_cast<char*>(kept + static_cast<size_t>(r0) * a.ld + c0);
    uint4 u[kDzRows / 2];
#pragma unroll
    for (int i = 0; i < kDzRows / 2; ++i) {
      const int rr = 2 * i + (lane >> 4);
      if (r0 + rr < n) u[i] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(rr) * a.ld * 2);
    }
    const int r = r0 + (lane & (kDzRows - 1));
    float m = 0.f, L1 = 0.f, L2 = 0.f, k1 = 0.f, k2 = 0.f;
    if (r < n) {
      m = a.pk[static_cast<size_t>(h) * a.ldp + r] + 65536.f * a.q_step;
      const float top = a.tops[a.row0 + r];
      L1 = top + a.l1[a.row0 + r];
      L2 = fmaf(top, a.inv_tau, a.l2[a.row0 + r]);
      row_factors(a, sc, a.flag[a.row0 + r], L1, k1, k2);
    }
#pragma unroll
    for (int i = 0; i < kDzRows / 2; ++i) {
      const int rr = 2 * i + (lane >> 4);
      const float mm = __shfl_sync(kFull, m, rr), La = __shfl_sync(kFull, L1, rr);
      const float Lb = __shfl_sync(kFull, L2, rr);
      const float ka = __shfl_sync(kFull, k1, rr), kb = __shfl_sync(kFull, k2, rr);
      uint4* at = reinterpret_cast<uint4*>(base + static_cast<size_t>(rr) * a.ld * 2);
      if (r0 + rr >= n) {
        *at = make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint32_t wds[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // 65536 + q by its bits: the conversion unit is the exponentials' as well
        const float q = __uint_as_float(0x47800000u | (j & 1 ? (wds[j >> 1] >> 9) & 0x7fff80u
                                                             : (wds[j >> 1] & 0xffffu) << 7));
        const float y = q == 131071.f ? -__int_as_float(0x7f800000) : fmaf(q, -a.q_step, mm);
        g[j] = ka * ex2(y - La);
        if (a.two) g[j] = fmaf(kb, ex2(fmaf(y, a.inv_tau, -Lb)), g[j]);
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j >= a.V) g[j] = 0.f;
      }
      // (one rounding to bf16: what the tensor cores take)
      *at = pack16(g, __nv_bfloat16());
    }
  }
}

// bf16 layers: the entries' columns, written over.
__global__ void __launch_bounds__(256)
head_dz_entries_kernel(const DzArgs a, const HeadLossOut o, __nv_bfloat16* __restrict__ dz) {
  pdl_wait();
  pdl_trigger();
  const int n = min(a.cnt->n - a.row0, a.piece);
  const HeadScale sc = scale_of(a);
  const int64_t total = static_cast<int64_t>(n) * o.E;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int r = static_cast<int>(i / o.E), e = static_cast<int>(i - static_cast<int64_t>(r) * o.E);
    const size_t rg = static_cast<size_t>(a.row0) + r, at = rg * o.E + e;
    const int id = o.ent[at];
    if (id == kHeadNoEntry || (e > 0 && o.ent[at - 1] == id)) continue;   // the first one writes
    float k1, k2;
    row_factors(a, sc, a.flag[rg], a.tops[rg] + a.l1[rg], k1, k2);
    dz[static_cast<size_t>(r) * a.ld + id] =
        __float2bfloat16_rn(entry_dz(a, sc, o, at, e, id, a.tops[rg], a.l1[rg], a.l2[rg], k1, k2));
  }
}

// fp32 layers: the kept logits themselves, a block a row, its entries behind them.  (The
// products' blocks are let in only when this one is done: in among its blocks they would
// gather on few SMs, 40 us for the small layer's step instead of 32.)
__global__ void __launch_bounds__(256)
head_dz_f32_kernel(const DzArgs a, const HeadLossOut o, float* __restrict__ kept) {
  pdl_wait();
  const int n = min(a.cnt->n - a.row0, a.piece);
  const HeadScale sc = scale_of(a);
  for (int r = blockIdx.x; r < n; r += gridDim.x) {
    const size_t rg = static_cast<size_t>(a.row0) + r;
    const float top = a.tops[rg], l1 = a.l1[rg], l2 = a.l2[rg];
    float k1, k2;
    row_factors(a, sc, a.flag[rg], top + l1, k1, k2);
    float* row = kept + static_cast<size_t>(r) * a.ld;
    for (int c0 = threadIdx.x; c0 < a.V; c0 += 4 * blockDim.x) {
      float z[4];   // (loaded ahead of the first store)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + j * blockDim.x;
        z[j] = c < a.V ? row[c] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + j * blockDim.x;
        const float y = over_top(z[j], top);
        float g = k1 * exp2f(y - l1);
        if (a.two) g += k2 * exp2f(y * a.inv_tau - l2);
        if (c < a.V) row[c] = g;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < o.E; e += blockDim.x) {
      const size_t at = rg * o.E + e;
      const int id = o.ent[at];
      if (id == kHeadNoEntry || (e > 0 && o.ent[at - 1] == id)) continue;
      row[id] = entry_dz(a, sc, o, at, e, id, top, l1, l2, k1, k2);
    }
  }
}

// ---- dx from its parts ---------------------------------------------------------------------
// A block takes four tokens at a time, their parts' loads in flight together; where the
// tokens are few and the parts many, one, and eight parts at a time (129 tokens, 31 parts
// of 512: 23 us by four).
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
template <typename O, int kDxTokens>
__global__ void __launch_bounds__(256)
head_dx_kernel(const HeadCounts* cnt, const int32_t* __restrict__ idx, const float* __restrict__ part,
               int splits, size_t split_stride, int row0, int piece, int d, float coef, float coef_kd,
               float coef_z, float tau, const float* __restrict__ dloss, O* __restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  const int n = min(cnt->n - row0, piece);
  const HeadScale sc = head_scale(cnt->n, cnt->n_ce, cnt->n_kd, coef, coef_kd, coef_z, tau, cnt->stretch);
  const float g = sc.unit * (dloss ? *dloss : 1.f);
  for (int r0 = blockIdx.x * kDxTokens; r0 < n; r0 += gridDim.x * kDxTokens) {
    int t[kDxTokens];
#pragma unroll
    for (int j = 0; j < kDxTokens; ++j) t[j] = r0 + j < n ? idx[row0 + r0 + j] : -1;
    for (int i = threadIdx.x * 4; i < d; i += blockDim.x * 4) {
      float4 v[kDxTokens];
#pragma unroll
      for (int j = 0; j < kDxTokens; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll (8 / kDxTokens)
      for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int j = 0; j < kDxTokens; ++j)
          if (r0 + j < n) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(
                part + s * split_stride + static_cast<size_t>(r0 + j) * d + i));
            v[j].x += f.x; v[j].y += f.y; v[j].z += f.z; v[j].w += f.w;
          }
#pragma unroll
      for (int j = 0; j < kDxTokens; ++j)
        if (t[j] >= 0)
          store4(dx + static_cast<size_t>(t[j]) * d + i,
                 make_float4(g * v[j].x, g * v[j].y, g * v[j].z, g * v[j].w));
    }
  }
}

// Bytes of labels and ids, over all blocks, from which a launch of tallies pays (12091 tokens
// with 64 teacher entries, 330 MB: rows 69 us, with tallies 3 + 43, of which 22 since entries
// are ordered by two compares each; 5936 with one, 158 MB: 12.4 us, and 3 + 9.1; 2048 with
// 32, 19 MB: 8.5 us without).
constexpr int64_t kTallyBytes = 1 << 25;

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace

// Parts of dx's reduction over the vocabulary, of bf16 layers.  In k blocks' time (0.33 us
// where the tensor cores are the bound): a tile lasts its blocks and some five more, a
// part costs its fp32 sums' way out and back, 8 bytes a value.  Beside dw's tiles the
// longest of dx or a CTA pair's share of all counts (8192 x 2048 x 50304: one part,
// written straight to its rows); alone the rounds of dx's tiles.
static int dx_splits(int rows, int d, int V, bool alone) {
  constexpr int64_t pairs = 76;
  const int64_t cols = (d + 255) / 256, units = (rows + 255) / 256 * cols;
  const int64_t kb = (V + 63) / 64, dw = (V + 255) / 256 * cols * ((rows + 63) / 64 + 5);
  const int most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, kb / 8)));
  int best = 1;
  double best_t = 1e300;
  for (int s = 1; s <= most; ++s) {
    const double tile = static_cast<double>(kb) / s + 5;
    double t = alone ? (units * s + pairs - 1) / pairs * tile
                     : std::max(tile, (units * s * tile + dw) / pairs);
    if (s > 1) t += s * 3.6e-6 * rows * d;
    if (t < best_t - 1e-12) { best_t = t; best = s; }
  }
  return best;
}

// The same for fp32 layers: two tiles for every SM, of no less than 128 products' depth.
static int dx_splits_f32(int rows, int d, int V) {
  const int ts = head_f32_tile(rows, d);
  const int64_t tiles = static_cast<int64_t>((rows + ts - 1) / ts) * ((d + ts - 1) / ts);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({2 * 152 / tiles, V / 128, 64})));
}

// Width of the logits' tiles: 256 columns, or what leaves the last round of a small batch
// fuller (each tile costs some 24 columns' time besides its own).
static int tile_width(int rows, int V) {
  const bool pair = rows > 128;
  const int64_t m = (rows + (pair ? 255 : 127)) / (pair ? 256 : 128);
  const int64_t slots = pair ? 76 : 152;
  int best = 256;
  int64_t best_t = (((V + 255) / 256) * m + slots - 1) / slots * (256 + 24);
  for (int bn = 224; bn >= 64; bn -= 32) {
    const int64_t t = (((V + bn - 1) / bn) * m + slots - 1) / slots * (bn + 24);
    if (t < best_t) { best_t = t; best = bn; }
  }
  return best;
}

HeadPlan head_plan(const occult_desc_t& ds, const occult_head_t& opt, bool step) {
  HeadPlan p{};
  p.T = ds.T; p.d = ds.d; p.V = opt.vocab; p.K = opt.topk; p.E = opt.topk + 1;
  p.dtype = ds.dtype; p.grad_dtype = opt.grad_dtype; p.step = step;
  p.tau = p.K ? opt.temperature : 1.f;
  p.coef = opt.coef; p.coef_kd = p.K ? opt.coef_kd : 0.f; p.coef_z = opt.coef_z;
  p.two = p.K > 0 && opt.temperature != 1.f;
  const bool bf = ds.dtype == OCCULT_BF16;
  const int Tr = static_cast<int>(up(std::max(1, ds.T), kHeadRowAlign));
  p.ld = static_cast<int>(up(p.V, 256));
  const int64_t row_bytes = static_cast<int64_t>(p.ld) * (bf ? 2 : 4);
  int64_t piece = opt.piece > 0 ? opt.piece : (int64_t(1) << 30) / row_bytes;
  piece = std::min<int64_t>(1 << 20, piece);
  piece = std::max<int64_t>(kHeadRowAlign, piece / kHeadRowAlign * kHeadRowAlign);
  // (without gradients a piece is what keeps the parts of the sums within some 512 MB, in
  // whole bands of the product's rows)
  if (!step)
    piece = std::max<int64_t>(8192, (int64_t(1) << 29) / (12 * ((p.V + (bf ? 127 : 31)) / (bf ? 128 : 32))) / 8192 * 8192);
  p.piece = static_cast<int>(std::min<int64_t>(piece, Tr));
  p.n_pieces = (Tr + p.piece - 1) / p.piece;
  // (the gradient of the logits is put together in parts of 128 columns)
  const int rows = std::min(p.piece, std::max(1, ds.T));
  p.bn = !bf ? head_f32_tile(rows, p.V) : step ? 256 : tile_width(rows, p.V);
  p.n_tiles = (p.V + p.bn - 1) / p.bn;
  p.halves = bf ? 2 * p.n_tiles : p.n_tiles;
  // Up to four tokens' losses: the weights' stream through the fp32 units.
  p.few = bf && !step && ds.T <= kHeadFewTokens;
  if (p.few) p.halves = head_few_blocks(p.V, p.d);
  p.splits = !step ? 1 : bf ? dx_splits(rows, p.d, p.V, false) : dx_splits_f32(rows, p.d, p.V);
  p.splits_alone = !step ? 1 : bf ? dx_splits(rows, p.d, p.V, true) : p.splits;
  p.q_step = std::max(24.f, 20.f * p.tau) / 65535.f;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += up(bytes, 256); return at; };
  const size_t T = Tr, P = p.piece;
  p.o_cnt = take(sizeof(HeadCounts));
  p.o_tally = take(16 * (T / kHeadRowAlign));
  p.o_idx = take(4 * T); p.o_flag = take(T);
  p.o_ent = take(4 * T * p.E); p.o_q = take(4 * T * p.E); p.o_zt = take(4 * T * p.E);
  p.o_xc = take(T * p.d * (bf ? 2 : 4));
  p.o_m = take(4 * P * p.halves); p.o_s = take(4 * P * p.halves);
  p.o_s2 = take(p.two ? 4 * P * p.halves : 0);
  p.o_mk = take(bf && step ? 4 * P * p.halves : 0);
  p.o_top = take(4 * T); p.o_l1 = take(4 * T); p.o_l2 = take(4 * T);
  p.o_sum = take(12 * (T / 32 + p.n_pieces));
  p.o_tune = take(bf && step ? 4 * kStretches * (P / 32) : 0);
  p.o_kept = take(step ? P * row_bytes : 0);
  const size_t parts = std::max(p.splits, p.splits_alone);
  p.o_part = take(step && (!bf || parts > 1) ? 4 * parts * P * p.d : 0);
  p.o_acc = take(step && p.n_pieces > 1 && p.grad_dtype == OCCULT_BF16
                     ? 4 * static_cast<size_t>(p.V) * p.d : 0);
  p.total = o;
  return p;
}

int launch_head(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a) {
  char* ws = a.ws;
  auto* cnt = reinterpret_cast<HeadCounts*>(ws + p.o_cnt);
  auto* idx = reinterpret_cast<int32_t*>(ws + p.o_idx);
  auto* flag = reinterpret_cast<uint8_t*>(ws + p.o_flag);
  auto* ent = reinterpret_cast<int32_t*>(ws + p.o_ent);
  auto* ent_q = reinterpret_cast<float*>(ws + p.o_q);
  auto* pm = reinterpret_cast<float*>(ws + p.o_m);
  auto* ps = reinterpret_cast<float*>(ws + p.o_s);
  auto* ps2 = reinterpret_cast<float*>(ws + p.o_s2);
  auto* tops = reinterpret_cast<float*>(ws + p.o_top);
  auto* l1 = reinterpret_cast<float*>(ws + p.o_l1);
  auto* l2 = reinterpret_cast<float*>(ws + p.o_l2);
  auto* sums = reinterpret_cast<float*>(ws + p.o_sum);
  auto* part = reinterpret_cast<float*>(ws + p.o_part);
  const bool bf = p.dtype == OCCULT_BF16;
  // at most about 1024 blocks, each of which counts every token; a warp or two for every
  // row of entries
  const int per = static_cast<int>(up((p.T + 1023) / 1024, p.K ? 8 : 32));
  const int grad_size = p.grad_dtype == OCCULT_BF16 ? 2 : 4;
  const int row_blocks = (p.T + per - 1) / per;
  // counting reads 4 bytes of a token's label and 32 of its teacher's first id, in every block
  int4* tally = nullptr;
  cudaError_t e = cudaSuccess;
  if (static_cast<int64_t>(row_blocks) * p.T * (p.K ? 36 : 4) > kTallyBytes) {
    tally = reinterpret_cast<int4*>(ws + p.o_tally);
    e = launch_pdl(head_tally_kernel, (p.T + kRowThreads - 1) / kRowThreads, kRowThreads, 0, ctx.stream, a.labels,
                   a.t_ids, p.T, p.V, p.K, tally);
    if (e != cudaSuccess) return OCCULT_ERR_CUDA;
  }
  e = launch_pdl(head_rows_kernel, row_blocks, kRowThreads, 0, ctx.stream, a.labels,
                             a.t_ids, a.t_logits, p.T, p.V, p.K, 1.f / p.tau, per, cnt, idx, flag, ent, ent_q,
                             a.lse, a.token_loss, static_cast<const uint4*>(a.x),
                             reinterpret_cast<uint4*>(ws + p.o_xc), p.d / (bf ? 8 : 4),
                             static_cast<char*>(a.dx), p.d * grad_size, tally);
  if (e != cudaSuccess) return OCCULT_ERR_CUDA;
  int n_blocks = 0;
  for (int i = 0; i < p.n_pieces; ++i)
    n_blocks += (std::min(p.piece, p.T - i * p.piece) + 31) / 32;
  int block0 = 0;
  for (int i = 0; i < p.n_pieces; ++i) {
    const int row0 = i * p.piece, rows = std::min(p.piece, p.T - row0);
    if (p.few) return launch_head_few(ctx, p, a);
    int rc = bf ? launch_head_logits_bf16(ctx, p, a, row0) : launch_head_logits_f32(ctx, p, a, row0);
    if (rc) return rc;
    const int blocks = (rows + 31) / 32;
    const int warps = blocks > ctx.num_sms ? 16 : 32;
    DzArgs z{};
    z.cnt = cnt; z.pk = reinterpret_cast<const float*>(ws + p.o_mk); z.tops = tops; z.l1 = l1; z.l2 = l2; z.flag = flag;
    z.ldp = p.piece; z.row0 = row0; z.piece = p.piece; z.V = p.V; z.ld = p.ld;
    z.inv_tau = 1.f / p.tau; z.q_step = p.q_step; z.tau = p.tau;
    z.coef = p.coef; z.coef_kd = p.coef_kd; z.coef_z = p.coef_z;
    z.two = p.two;
#define OCCULT_HEAD_SUM(TWO, TUNE) (warps == 32 ? head_sum_kernel<TWO, 32, TUNE> : head_sum_kernel<TWO, 16, TUNE>)
    auto* sum = bf && p.step ? (p.two ? OCCULT_HEAD_SUM(true, true) : OCCULT_HEAD_SUM(false, true))
                             : (p.two ? OCCULT_HEAD_SUM(true, false) : OCCULT_HEAD_SUM(false, false));
#undef OCCULT_HEAD_SUM
    e = launch_pdl(sum, blocks, warps * 32, 0, ctx.stream, cnt, head_loss_out(p, a), pm, ps, ps2, p.piece,
                   p.halves, row0, rows, idx, flag, tops, l1, l2, sums, block0, n_blocks, z,
                   reinterpret_cast<float*>(ws + p.o_tune));
    if (e != cudaSuccess) return OCCULT_ERR_CUDA;
    block0 += blocks;
    if (!p.step) continue;
    if (bf) {
      auto* kept = reinterpret_cast<uint16_t*>(ws + p.o_kept);
      // some eight blocks an SM, however many of the rows count
      const int gx = (p.ld / 128 + 7) / 8, steps = (rows + kHeadRowAlign - 1) / kHeadRowAlign * (kHeadRowAlign / kDzRows);
      const dim3 grid(gx, std::min(steps, std::max(1, (ctx.num_sms * 8 + gx - 1) / gx)));
      e = launch_pdl(head_dz_bf16_kernel, grid, 256, 0, ctx.stream, z, kept);
      if (e != cudaSuccess) return OCCULT_ERR_CUDA;
      const int eb = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(rows) * p.E + 255) / 256,
                                                        ctx.num_sms * 16));
      e = launch_pdl(head_dz_entries_kernel, eb, 256, 0, ctx.stream, z, head_loss_out(p, a),
                     reinterpret_cast<__nv_bfloat16*>(kept));
    } else {
      e = launch_pdl(head_dz_f32_kernel, std::min(rows, ctx.num_sms * 8), 256, 0, ctx.stream, z,
                     head_loss_out(p, a), reinterpret_cast<float*>(ws + p.o_kept));
    }
    if (e != cudaSuccess) return OCCULT_ERR_CUDA;
    const bool first = i == 0, last = i == p.n_pieces - 1;
    rc = bf ? launch_head_grads_bf16(ctx, p, a, row0, first, last)
            : launch_head_grads_f32(ctx, p, a, row0, first, last);
    if (rc) return rc;
    const int splits = head_splits(p, a);
    if (a.dx && (!bf || splits > 1)) {
      const int tokens = rows >= 4 * ctx.num_sms ? 4 : 1;
      const int nb = std::min((rows + tokens - 1) / tokens, ctx.num_sms * 8);
      const int threads = std::min(256, (p.d / 4 + 31) / 32 * 32);
      const size_t stride = static_cast<size_t>(p.piece) * p.d;
#define OCCULT_HEAD_DX(O)                                                                          \
  launch_pdl(tokens == 4 ? head_dx_kernel<O, 4> : head_dx_kernel<O, 1>, nb, threads, 0, ctx.stream, \
             cnt, idx, part, splits, stride, row0, p.piece, p.d, p.coef, p.coef_kd, p.coef_z,      \
             p.tau, a.dloss, static_cast<O*>(a.dx))
      e = p.grad_dtype == OCCULT_BF16 ? OCCULT_HEAD_DX(__nv_bfloat16) : OCCULT_HEAD_DX(float);
#undef OCCULT_HEAD_DX
      if (e != cudaSuccess) return OCCULT_ERR_CUDA;
    }
  }
  return OCCULT_OK;
}

}  // namespace occult
