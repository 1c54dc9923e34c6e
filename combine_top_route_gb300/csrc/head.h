// What the output head's parts share: the host's plan of a call and the scalars that
// its kernels take (head.cu: rows, entries, sums, gradients of the logits; head_gemm.cu:
// the products of bf16 layers; head_simt.cu: those of fp32 layers).
#pragma once

#include "common.cuh"

namespace occult {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kHeadRowAlign = 256;   // rows of a piece and of its buffers
constexpr int kHeadNoEntry = 0x7fffffff;

// Device counters at the head of the workspace.
struct HeadCounts {
  int n;        // tokens that a term counts: compact rows
  int n_ce;     // of them with a label
  int n_kd;     // of them with a teacher row
  unsigned ticket;
  float stretch;   // factor of the common factor of the piece at hand (see HeadScale)
};

// What a row is to the loss.
enum : uint8_t { kRowCe = 1, kRowKd = 2 };   // it has a label, a teacher

// Sizes and workspace offsets of a call; every launcher works from one of these.
struct HeadPlan {
  int T, d, V, K, E;        // E = K + 1 entries a row: the teacher's and the label
  int dtype, grad_dtype;
  bool step, two;           // two: sums at temperature 1 and tau
  bool few;                 // the loss of up to four tokens on the fp32 units
  int piece, n_pieces;      // tokens of a piece (a multiple of kHeadRowAlign)
  int ld;                   // columns of the kept logits
  int bn;                   // vocabulary columns of a tile
  int n_tiles, halves;      // tiles, and parts of a row's sums (bf16: two a tile)
  int splits, splits_alone; // parts of dx's reduction: beside dw, and without it
  float tau, coef, coef_kd, coef_z;
  float q_step;             // octaves of a unit of the kept 16-bit logits
  // workspace
  size_t o_cnt, o_tally, o_idx, o_flag, o_ent, o_q, o_zt, o_xc, o_m, o_s, o_s2, o_mk, o_top, o_l1, o_l2, o_sum, o_tune,
      o_kept, o_part, o_acc, total;
};

struct HeadArgs {
  const void* x;
  const void* w;
  const int32_t* labels;
  const int32_t* t_ids;
  const float* t_logits;
  const float* dloss;
  float *lse, *token_loss, *loss;
  void *dx, *dw;
  char* ws;
};

// The losses' outputs, and what they are made from.
struct HeadLossOut {
  const int32_t* ent;    // entries of the compact rows: token, probability (-1: the label),
  const float* ent_q;    // the student's logit
  const float* zt;
  float *lse, *token_loss, *loss;
  int E;
  float tau, coef, coef_kd, coef_z;
};
inline HeadLossOut head_loss_out(const HeadPlan& p, const HeadArgs& a) {
  return {reinterpret_cast<const int32_t*>(a.ws + p.o_ent), reinterpret_cast<const float*>(a.ws + p.o_q),
          reinterpret_cast<const float*>(a.ws + p.o_zt), a.lse, a.token_loss, a.loss, p.E, p.tau, p.coef,
          p.coef_kd, p.coef_z};
}

#ifdef __CUDACC__
constexpr uint32_t kFull = 0xffffffffu;
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
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

// A row's sums are of 2^(z log2(e) - top), `top` its maximum in octaves, and at temperature
// tau of that exponent over tau; l1 and l2 are their log2.  top and l1 stay apart: a token
// that is nearly sure of its label has z log2(e) - top - l1 near 0, which top + l1 in one
// fp32 would leave without its digits (2e-6 octaves at a logit of 20, where 1 - p may be 1e-3).
__device__ __forceinline__ float over_top(float z, float top) { return fmaf(z, kLog2e, -top); }

// A warp finishes compact row r: writes the token's outputs and adds its terms to `sum`.  The
// whole warp calls `each` with its lanes' entries, 32 of the row's at a time: token (or none),
// probability and the logit's distance to the row's maximum in octaves.
struct RowSums { float ce, kd, z; };
struct NoEach { __device__ __forceinline__ void operator()(int, float, float) const {} };
template <typename Each = NoEach>
__device__ __forceinline__ void row_losses(const HeadLossOut& o, size_t r, int flag, int token, float top,
                                           float l1, float l2, float inv_tau, RowSums& sum,
                                           const Each& each = Each()) {
  const int lane = threadIdx.x & 31;
  const float lse = (top + l1) * kLn2;
  float tok = 0.f, kd = 0.f;
  for (int e0 = 0; e0 < o.E; e0 += 32) {
    const bool there = e0 + lane < o.E;
    const size_t at = r * o.E + e0 + lane;
    const int id = there ? __ldcg(o.ent + at) : kHeadNoEntry;
    const float q = there ? __ldcg(o.ent_q + at) : 0.f, z = there ? __ldcg(o.zt + at) : 0.f;
    const float y = over_top(z, top);
    if (id != kHeadNoEntry) {
      if (q < 0.f) tok = (l1 - y) * kLn2;
      else if (q != 0.f) kd += q * (logf(q) - (y * inv_tau - l2) * kLn2);
    }
    each(id, q, y);
  }
  tok = warp_sum(tok);
  const float ce = (flag & kRowCe) ? tok : 0.f;
  sum.ce += ce;
  sum.kd += warp_sum(kd);
  sum.z += lse * lse;
  if (lane == 0) {
    if (o.lse) o.lse[token] = lse;
    if (o.token_loss) o.token_loss[token] = ce;
  }
}
// The means, from the sums over all rows.
__device__ __forceinline__ void mean_losses(const HeadLossOut& o, const HeadCounts& cnt, float ce, float kd,
                                            float z) {
  ce = cnt.n_ce > 0 ? ce / static_cast<float>(cnt.n_ce) : 0.f;
  kd = cnt.n_kd > 0 ? o.tau * o.tau * kd / static_cast<float>(cnt.n_kd) : 0.f;
  z = cnt.n > 0 ? z / static_cast<float>(cnt.n) : 0.f;
  o.loss[0] = o.coef * ce + o.coef_kd * kd + o.coef_z * z;
  o.loss[1] = ce;
  o.loss[2] = kd;
  o.loss[3] = z;
}
#endif

// Factors of a term's gradient over the mean of its tokens, and the common factor that
// is kept out of the rounded gradients of the logits: the cross entropy's where it
// counts, so that its -1 at the label is exact.  A factor 2^-40 of another's and less does
// not count: the other's ratio to it need not be a number.
struct HeadScale {
  float unit;      // common factor
  float k_ce, k_kd, k_z;   // coef / N_ce, coef_kd tau / N_kd, 2 coef_z / N over it
};
// `stretch`: 1, or what a bf16 layer's piece takes besides, one of kStretches powers of 2 from 1 up
// to 2: the one under which the entries' gradients lose least to their rounding to bf16 (in
// the 2-norm).  They are most of a row's gradient; where few of them stand just above a power
// of two, half a unit is 2^-8 of them, just below it 2^-9.  Of 145 small steps drawn at
// random the errors of dx and dw were up to 2.1 times that of a rounding of the result
// alone, in 27 over 1.5; 1.46 with eight to choose from, 1.45 with 64.
constexpr int kStretches = 8;
__host__ __device__ inline HeadScale head_scale(int n, int n_ce, int n_kd, float coef,
                                                float coef_kd, float coef_z, float tau, float stretch) {
  HeadScale s;
  const float a = n_ce > 0 ? coef / static_cast<float>(n_ce) : 0.f;
  const float b = n_kd > 0 ? coef_kd * tau / static_cast<float>(n_kd) : 0.f;
  const float c = n > 0 ? 2.f * coef_z / static_cast<float>(n) : 0.f;
  const float least = 0x1p-40f * (a > b ? (a > c ? a : c) : (b > c ? b : c));
  s.unit = a > 0.f && a >= least ? a : b > 0.f && b >= least ? b : c > 0.f ? c : 1.f;
  s.unit *= stretch;
  s.k_ce = a / s.unit;
  s.k_kd = b / s.unit;
  s.k_z = c / s.unit;
  return s;
}

// Edge of the fp32 products' tiles over rows x columns: 64 where that makes two for every
// SM, else 32.
inline int head_f32_tile(int64_t rows, int64_t cols) {
  return ((rows + 63) / 64) * ((cols + 63) / 64) >= 2 * 152 ? 64 : 32;
}

HeadPlan head_plan(const occult_desc_t& ds, const occult_head_t& opt, bool step);
int launch_head(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a);

// Products of bf16 layers over the rows [row0, row0 + piece) of the compact rows.
//  logits: partial maxima and sums, the logits of the entries, and (step) the logits in
//          16 bits;  grads: dx (to its tokens' rows, or parts [splits][piece][d] fp32) and dw
//          (written for the first piece, or added to), scaled.
int launch_head_logits_bf16(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0);
int launch_head_grads_bf16(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0,
                           bool first, bool last);
inline int head_splits(const HeadPlan& p, const HeadArgs& a) { return a.dw ? p.splits : p.splits_alone; }
// The same of fp32 layers.
int launch_head_logits_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0);
int launch_head_grads_f32(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0,
                          bool first, bool last);

// The loss of up to kHeadFewTokens tokens of a bf16 layer, from its rows and entries to its
// outputs (head_few.cu); blocks that share the vocabulary.
constexpr int kHeadFewTokens = 4;
int head_few_blocks(int V, int d);
int launch_head_few(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a);

// 2-D bf16 tensor map of a row-major [rows, cols] matrix, 128-byte swizzle.
int tensor_map_bf16(CUtensorMap* m, const void* base, int64_t rows, int64_t cols,
                    uint32_t box_cols, uint32_t box_rows);

}  // namespace occult
