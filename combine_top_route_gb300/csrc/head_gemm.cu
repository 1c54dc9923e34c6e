// Products of the output head on the sm_103a tensor cores (tcgen05 + TMEM + TMA).
//
//   logits  z = x w^T: a tile's columns never leave the chip whole.  Its epilogue finds
//           the maximum and the sum of powers of two of every row's 128 columns, picks
//           out the logits of the row's entries (its label and teacher tokens, sorted, so
//           that a tile looks its first one up and walks on), and for a training step
//           keeps the logits in 16 bits: octaves below the largest of the part that is no
//           entry (an entry's gradient is made from its own fp32 logit), in steps s of
//           max(24, 20 tau) / 65535, the last of them for all that lies lower.  A probability
//           is within s ln 2 / 2 of itself (over tau where tempered): 1.3e-4 up to tau = 1.2,
//           a thirtieth of bf16's rounding of the gradient made from it, 2.1e-4 at 2, 1.1e-3
//           at 10; below the range, 2^-24 of the part's largest (2^-20 tempered), it is 0.
//           Entries would take the range away from the others: of a token sure of its label
//           the other tokens' probabilities are all its gradient is made of.
//   gradients  dx = dz w over the vocabulary (cut into parts where its tiles would not
//           go round) and dw = dz^T x over the rows, the tiles of both in one launch: dx's
//           first, dealt in turn, then dw's, of which pairs that got one dx tile less
//           take as many more as that one's time.
//
// Persistent CTA pairs (tcgen05.mma.cta_group::2: a 256 x 256 tile, rows 0..127 in the
// even CTA, half of the columns' operand in each) or, up to 128 rows, single CTAs with a
// 128-row tile that is mostly padding: there the weights' stream is the bound, and the
// padding costs tensor time that is idle anyway.
//
// CTA = 12 warps: warp 0 TMA producer, warp 1 owner of TMEM (two accumulators, so that a
// tile's epilogue runs under the next one's products) and issuer of the products (in a
// pair the even CTA's), warps 4..11 epilogue, two to a TMEM lane quarter, half of the
// columns each.  Every wait is bounded.
#include <algorithm>

#include "head.h"
#include "kernels.h"

namespace occult {

namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kABytes = BM * BK * 2;          // 16 KB
constexpr int kMnAtom = BK * 128;             // 64 columns of an MN-major operand
constexpr int kEpiWarps = 8, kEpiWarp0 = 4;   // whole warpgroups, for their registers
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kLaunchRegs = 168, kCtrlRegs = 40, kEpiRegs = 232;   // a thread
static_assert(32 * (kEpiWarp0 * kCtrlRegs + kEpiWarps * kEpiRegs) <= kThreads * kLaunchRegs, "registers");
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 8;

enum : int { HEAD_STATS = 0, HEAD_KEEP = 1, HEAD_GRADS = 2 };

// The ring: 192 KB in stages of A's 16 KB and as much of B as the tile has columns.
constexpr int kRingBytes = 192 * 1024;
constexpr int kPairStage = kABytes + BN / 2 * BK * 2;

struct Tail {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kTailBytes = (static_cast<int>(sizeof(Tail)) + 127) & ~127;
constexpr int kEpiBytes = kEpiWarps * 32 * 32 * 4;   // 4 KB a warp
constexpr int kSmemBytes = 1024 + kRingBytes + kTailBytes + kEpiBytes;
static_assert(kSmemBytes <= 232448, "shared memory");

struct GemmArgs {
  const HeadCounts* cnt;
  int T, row0, piece;     // tokens; the piece's first compact row and its rows
  int V, d, bn, n_tiles;  // vocabulary, width, columns of a tile, tiles
  int stages, stage_bytes;   // of single CTAs
  // logits
  const int32_t* ent;
  float* zt;
  int E;
  float *pm, *ps, *ps2, *pk;   // parts' maxima and sums; pk: the kept logits' upper ends
  int ldp, ld;
  uint16_t* kept;
  float inv_tau, q_inv;
  int seg;                // k blocks added up in TMEM before they go to registers
  // gradients
  int splits;             // dx: parts; with one it is written to its tokens' rows
  float* part;
  const int32_t* idx;
  void *dx, *dw;          // either may be missing
  float* acc;             // dw of earlier pieces in fp32 (nullptr: in dw)
  const float* dloss;
  float coef, coef_kd, coef_z, tau;
  int out_bf16, first, last;
  int* dev_err;
};

// One tile of the schedule.
struct Unit {
  int m0;      // first row of this CTA's 128 (rows of the piece; dw: of the vocabulary)
  int n0;      // first column of the tile
  int nt;      // its number
  int k0, k1;  // k blocks
  int split;   // dx: part
  bool dw;
};

// Logits: bands of 32 row tiles; inside one all row tiles of a column tile follow each
// other, so that a weight tile is read once a band and the band's rows stay in L2.
constexpr int kBand = 32;

// What a tile costs besides its k blocks, in their time.
constexpr int kTileCost = 5;

// A launch's tiles, and the ones of a CTA (pair) `me` of `all`.
template <int MODE, bool PAIR>
struct Schedule {
  static constexpr bool kLogits = MODE != HEAD_GRADS;
  static constexpr int RM = PAIR ? 2 * BM : BM;
  const GemmArgs& p;
  int me, all, rank, m_units, kb_rows, n_first, n_second;   // logits or dx tiles; dw tiles
  int firsts, rest, extra;

  __device__ __forceinline__ Schedule(const GemmArgs& p_, int n, int me_, int all_, int rank_)
      : p(p_), me(me_), all(all_), rank(rank_) {
    m_units = (n + RM - 1) / RM;
    kb_rows = (n + BK - 1) / BK;
    n_first = kLogits || p.dx ? m_units * p.n_tiles * (kLogits ? 1 : p.splits) : 0;
    n_second = !kLogits && p.dw ? (p.V + RM - 1) / RM * p.n_tiles : 0;
    firsts = (n_first - me + all - 1) / all;
    rest = n_first % all;
    // dw tiles to the time of a dx tile
    extra = rest ? ((p.V + BK - 1) / BK / p.splits + kTileCost) / (kb_rows + kTileCost) : 0;
  }
  // The i-th tile's number, -1 behind the last.
  __device__ __forceinline__ int at(int i) const {
    if (i < firsts) return me + i * all;
    if (kLogits) return -1;
    const int j = i - firsts, more = rest ? all - rest : 0;
    int64_t u;
    if (me >= rest && j < extra && more) u = static_cast<int64_t>(j) * more + (me - rest);
    else u = static_cast<int64_t>(more) * extra + static_cast<int64_t>(j - (more && me >= rest ? extra : 0)) * all + me;
    return u < n_second ? n_first + static_cast<int>(u) : -1;
  }
  __device__ __forceinline__ Unit unit(int u) const {
    Unit t;
    t.split = 0;
    t.k0 = 0;
    t.dw = u >= n_first;
    if (kLogits) {
      const int band = u / (kBand * p.n_tiles);
      const int in = u - band * (kBand * p.n_tiles);
      const int rows = min(kBand, m_units - band * kBand);
      t.nt = in / rows;
      t.m0 = (band * kBand + in - t.nt * rows) * RM + rank * BM;
      t.k1 = p.d / BK;
    } else {
      int in = u - (t.dw ? n_first : 0);
      if (!t.dw) {
        const int per = m_units * p.n_tiles, kb = (p.V + BK - 1) / BK;
        t.split = in / per;
        in -= t.split * per;
        t.k0 = static_cast<int>(static_cast<int64_t>(kb) * t.split / p.splits);
        t.k1 = static_cast<int>(static_cast<int64_t>(kb) * (t.split + 1) / p.splits);
      } else {
        t.k1 = kb_rows;
      }
      t.nt = in % p.n_tiles;
      t.m0 = in / p.n_tiles * RM + rank * BM;
    }
    t.n0 = t.nt * p.bn;
    return t;
  }
};

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int kk) {
  if (MN) return smem_desc_sw128_mn(base + kk * 2048, kMnAtom, 1024);
  return smem_desc_sw128(base + kk * 32);
}

// A lane's 16-byte piece j (of 8) of its own row in the warp's 4 KB buffer, and a word
// of it: pieces lie at j ^ (row % 8), free of bank conflicts along a row and across rows.
__device__ __forceinline__ uint32_t* own_piece(uint32_t* buf, int j) {
  const int lane = threadIdx.x & 31;
  return buf + lane * 32 + 4 * (j ^ (lane & 7));
}
// The buffer's 32 rows of 128 bytes to global rows: 8 lanes a row.  Rows >= valid stay.
__device__ __forceinline__ void flush_rows(const uint32_t* buf, char* out, int64_t row_bytes, int valid) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int r = it * 4 + lane / 8, c = lane & 7;
    if (r < valid)
      st_v4(out + r * row_bytes + c * 16, *reinterpret_cast<const uint4*>(buf + r * 32 + 4 * (c ^ (r & 7))));
  }
  __syncwarp();
}

// First entry at or behind column c of a row's sorted E.
__device__ __forceinline__ int first_entry(const int32_t* ent, int E, int c) {
  int lo = 0, hi = E;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ent[mid] < c) lo = mid + 1; else hi = mid;
  }
  return lo;
}

template <int MODE, bool PAIR, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                 const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
                 const GemmArgs p) {
  constexpr bool kLogits = MODE != HEAD_GRADS;
  constexpr int RM = PAIR ? 2 * BM : BM;
  // Pairs: six of 32 KB, known when compiled (a stage count of the launch's cost 3 % of the
  // large products); single CTAs: as many of a narrow tile's as the ring holds.
  const int kStages = PAIR ? kRingBytes / kPairStage : p.stages;
  const int kStageBytes = PAIR ? kPairStage : p.stage_bytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Tail* tail = reinterpret_cast<Tail*>(smem + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tail->tfull[a], 1);
      mbar_init(&tail->tempty[a], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    tail->abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    if (PAIR) tmem_alloc_pair(&tail->tmem_base, kTmemCols);
    else tmem_alloc(&tail->tmem_base, kTmemCols);
  }
  tc_fence_before();
  if (PAIR) cluster_sync(); else __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();

  const int n_all = p.cnt->n;
  const int n = max(0, min(n_all - p.row0, p.piece));   // rows of this piece
  const bool whole = n_all == p.T;   // every token counts: x is read where it lies
  const Schedule<MODE, PAIR> plan(p, n, PAIR ? blockIdx.x >> 1 : blockIdx.x, PAIR ? gridDim.x >> 1 : gridDim.x,
                                  rank);
  const uint32_t tbase = tail->tmem_base;
  volatile int* abort_flag = &tail->abort_flag;
  const uint32_t full_lead = PAIR ? smem_addr_in_rank(&tail->full[0], 0) : 0u;
  const uint32_t tempty_lead = PAIR ? smem_addr_in_rank(&tail->tempty[0], 0) : 0u;
  const int b_rows = PAIR ? p.bn / 2 : p.bn;            // of the tile's columns in this CTA
  // bytes of a stage: the boxes are whole wherever they lie
  const uint32_t cta_bytes = kABytes + static_cast<uint32_t>(b_rows) * (BK * 2);

  // The logits' epilogue holds a row's 128 sums beside its work: the launch's 384 x 168
  // registers are dealt out anew, 128 x 40 + 256 x 232.
  if (warp < kEpiWarp0) {
    if (kLogits) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kCtrlRegs));
    if (warp == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // logits: x or its compact copy, and w; gradients: dz for both (as it lies, 64 x 64
      // boxes), and w or x
      const CUtensorMap* ma = kLogits && !whole ? &tmA2 : &tmA;
      const CUtensorMap* mx = whole ? &tmA2 : &tmB2;
      if (lane == 0) { prefetch_tmap(ma); prefetch_tmap(&tmB); }
      // Single CTAs all read the few rows of x there are: each begins at a k block of its
      // own, or they would queue for the same lines (12 tokens x 2432 x 32366: 36 -> 34 us).
      const int turn = static_cast<int>(static_cast<int64_t>(p.d / BK) * blockIdx.x / gridDim.x);
      for (int i = 0, u; ok && (u = plan.at(i)) >= 0; ++i) {
        const Unit t = plan.unit(u);
        const int bc = t.n0 + (PAIR ? rank * b_rows : 0);   // this CTA's first column
        for (int kb = t.k0; kb < t.k1; ++kb) {
          if (!mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
          if (lane == 0) {
            uint8_t* sa = smem + stage * kStageBytes;
            uint8_t* sb = sa + kABytes;
            uint64_t* bar = &tail->full[stage];
            const uint32_t lbar = full_lead + stage * 8;
            if (leader) mbar_arrive_expect_tx(bar, PAIR ? 2 * cta_bytes : cta_bytes);
            if constexpr (kLogits) {
              if (PAIR) {
                tma_load_2d_pair(sa, ma, kb * BK, p.row0 + t.m0, lbar);
                tma_load_2d_pair(sb, &tmB, kb * BK, bc, lbar);
              } else {
                const int at = kb + turn < t.k1 ? kb + turn : kb + turn - t.k1;
                tma_load_2d(sa, ma, at * BK, p.row0 + t.m0, bar);
                tma_load_2d(sb, &tmB, at * BK, bc, bar);
              }
            } else {
              // (128 rows of 64 columns, or 64 rows of 128: two boxes either way)
              for (int a = 0; a < 2; ++a)
                tma_load_2d_pair(sa + a * kMnAtom, ma, t.dw ? t.m0 + 64 * a : kb * BK,
                                 t.dw ? kb * BK : t.m0 + 64 * a, lbar);
              for (int a = 0; a < b_rows / 64; ++a)
                tma_load_2d_pair(sb + a * kMnAtom, t.dw ? mx : &tmB, bc + 64 * a,
                                 kb * BK + (t.dw ? p.row0 : 0), lbar);
            }
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (PAIR && ok) {
        // no release of a stage lands after the CTA has exited
        for (int i = 0; i < kStages && ok; ++i) {
          if (!mbar_wait(&tail->empty[stage], phase ^ 1u, abort_flag)) ok = false;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        if (lane == 0) latch_error(p.dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
      }
    } else if (warp == 1) {
      if (lane == 0 && leader) {
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0, u; ok && (u = plan.at(i)) >= 0; ++i) {
          const Unit t = plan.unit(u);
          // bits 15 and 16: A (dw) and B (both gradients) lie along M and N
          const uint32_t idesc = idesc_bf16_f32(RM, p.bn) | (t.dw && !kLogits ? 1u << 15 : 0u) |
                                 (kLogits ? 0u : 1u << 16);
          int kb = t.k0;
          do {   // (a unit without k blocks still hands over its accumulator)
            const int end = min(t.k1, p.seg < t.k1 - kb ? kb + p.seg : t.k1);
            const int a = it & 1;
            const uint32_t aph = (it >> 1) & 1;
            ++it;
            if (!(PAIR ? mbar_wait_cluster(&tail->tempty[a], aph ^ 1u, abort_flag)
                       : mbar_wait(&tail->tempty[a], aph ^ 1u, abort_flag))) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tbase + a * BN;
            for (const int first = kb; kb < end; ++kb) {
              if (!(PAIR ? mbar_wait_cluster(&tail->full[stage], phase, abort_flag)
                         : mbar_wait(&tail->full[stage], phase, abort_flag))) { ok = false; break; }
              tc_fence_after();
              const uint32_t sa = smem_u32(smem + stage * kStageBytes), sb = sa + kABytes;
  #pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                const bool add = kb != first || kk != 0;
                const uint64_t da = !kLogits && t.dw ? operand_desc<true>(sa, kk) : operand_desc<false>(sa, kk);
                if (PAIR) tc_mma_f16_pair(acc, da, operand_desc<!kLogits>(sb, kk), idesc, add);
                else tc_mma_f16(acc, da, operand_desc<!kLogits>(sb, kk), idesc, add);
              }
              if (PAIR) tc_commit_pair(&tail->empty[stage], 0x3);
              else tc_commit(&tail->empty[stage]);
              if (++stage == kStages) { stage = 0; phase ^= 1u; }
            }
            if (ok) {
              if (PAIR) tc_commit_pair(&tail->tfull[a], 0x3);
              else tc_commit(&tail->tfull[a]);
            }
          } while (ok && kb < t.k1);
        }
        if (!ok) {
          latch_error(p.dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
          *abort_flag = 1;
        }
      }
      __syncwarp();
    }
  } else {
    if (kLogits) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kEpiRegs));
    // ---- epilogue ----------------------------------------------------------
    const int quarter = warp & 3, half = (warp - kEpiWarp0) / 4;
    uint32_t* buf = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(tail) + kTailBytes) +
                    (warp - kEpiWarp0) * 1024;
    float g = 0.f;
    if (!kLogits) {
      const HeadScale sc = head_scale(n_all, p.cnt->n_ce, p.cnt->n_kd, p.coef, p.coef_kd, p.coef_z, p.tau,
                                      p.cnt->stretch);
      g = sc.unit * (p.dloss ? *p.dloss : 1.f);
    }
    int it = 0;
    bool ok = true;
    const int hw = p.bn / 2;   // columns of this warp's half
    for (int i = 0, u; ok && (u = plan.at(i)) >= 0; ++i) {
      const Unit t = plan.unit(u);
      const int rows_all = !kLogits && t.dw ? p.V : n;
      const int valid = min(32, rows_all - t.m0 - quarter * 32);   // rows of this warp (may be < 1)
      const int c0 = t.n0 + half * hw;                             // its first column
      const int64_t row = t.m0 + quarter * 32 + lane;
      int a = 0;
      // the next accumulator, once its products are done; false when the wait gave up
      auto take = [&]() -> bool {
        a = it & 1;
        const uint32_t aph = (it >> 1) & 1;
        ++it;
        if (!mbar_wait(&tail->tfull[a], aph, abort_flag)) return false;
        tc_fence_after();
        return true;
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_remote(tempty_lead + a * 8); else mbar_arrive(&tail->tempty[a]);
        }
      };
      const uint32_t lanes = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + half * hw;

      if constexpr (kLogits) {
        const int lim = valid < 1 ? 0 : min(hw, p.V - c0);   // columns that exist
        const float NEG = -__int_as_float(0x7f800000);
        // the row's first entry at or behind c0, looked up while the products run
        int e = 0, next = kHeadNoEntry;
        const int32_t* ent = nullptr;
        float* zt = nullptr;
        if (lane < valid) {
          ent = p.ent + (p.row0 + row) * p.E;
          zt = p.zt + (p.row0 + row) * p.E;
          e = first_entry(ent, p.E, c0);
          if (e < p.E) next = ent[e];
        }
        // The tensor cores add with truncation: over 2048 products the logits of a
        // token that leans to its label would come out low by 3e-6 of themselves.  Sums
        // of p.seg k blocks are added up here, rounded to nearest.
        float z[128];
        for (int kb = t.k0; kb < t.k1; kb += p.seg) {
          if (!take()) { ok = false; break; }
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            if (c < lim) {
              uint32_t v[32];
              tmem_ld32(lanes + a * BN + c, v);
              tmem_ld_wait();
              if (kb == t.k0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) z[c + j] = __uint_as_float(v[j]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) z[c + j] += __uint_as_float(v[j]);
              }
            }
          }
          release();
        }
        if (!ok) break;
        if (valid < 1) continue;
        if (lim < 128) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= lim) z[j] = NEG;
        }
        // the maximum, the entries' logits, and (kept) the maximum of the others
        float m = NEG, mk = NEG;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float top = NEG;
#pragma unroll
          for (int j = 0; j < 32; ++j) top = fmaxf(top, z[c + j]);
          m = fmaxf(m, top);
          const int end = c0 + min(c + 32, lim);
          if (c < lim && __any_sync(0xffffffffu, next < end)) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(own_piece(buf, j)) =
                  make_float4(z[c + 4 * j], z[c + 4 * j + 1], z[c + 4 * j + 2], z[c + 4 * j + 3]);
            bool again = false;
            float v = NEG;
            for (int id = -1; next < end;) {
              if (next != id) {   // (the first of its token)
                id = next;
                const int at = next - c0 - c;
                uint32_t* p = own_piece(buf, at >> 2) + (at & 3);
                v = __uint_as_float(*p);
                if (MODE == HEAD_KEEP) {
                  *p = __float_as_uint(NEG);
                  again |= v == top;
                }
              }
              zt[e] = v;
              ++e;
              next = e < p.E ? ent[e] : kHeadNoEntry;
            }
            if (MODE == HEAD_KEEP && again) {
              top = NEG;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(own_piece(buf, j));
                top = fmaxf(top, fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)));
              }
            }
            __syncwarp();
          }
          if (MODE == HEAD_KEEP) mk = fmaxf(mk, top);
        }
        // the sums, and the logits to keep
        const float my = (m == NEG ? 0.f : m) * kLog2e;
        const float mine = (mk == NEG ? 0.f : mk) * kLog2e;
        const float qc = -kLog2e * p.q_inv, qm = mine * p.q_inv;
        float s = 0.f, s2 = 0.f;
        char* keep = nullptr;
        if (MODE == HEAD_KEEP)
          keep = reinterpret_cast<char*>(p.kept + (static_cast<int64_t>(t.m0) + quarter * 32) * p.ld + c0);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (MODE == HEAD_KEEP || c < lim) {
            float sa = 0.f, sb = 0.f, ta = 0.f, tb = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float y0 = over_top(z[c + j], my), y1 = over_top(z[c + j + 1], my);
              sa += ex2(y0);
              sb += ex2(y1);
              if (TWO) {
                ta += ex2(y0 * p.inv_tau);
                tb += ex2(y1 * p.inv_tau);
              }
            }
            s += sa + sb;
            if (TWO) s2 += ta + tb;
          }
          if (MODE == HEAD_KEEP) {
            // the low bits of t + 2^23 are t to the nearest: no conversion unit (an
            // entry's t may be below 0, and the maximum's own round there)
            const int j0 = (c & 32) ? 4 : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t wd[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                wd[i] = __float_as_uint(fminf(fmaxf(fmaf(z[c + 8 * j + i], qc, qm), 0.f), 65535.f) + 8388608.f);
              *reinterpret_cast<uint4*>(own_piece(buf, j0 + j)) =
                  make_uint4(__byte_perm(wd[0], wd[1], 0x5410), __byte_perm(wd[2], wd[3], 0x5410),
                             __byte_perm(wd[4], wd[5], 0x5410), __byte_perm(wd[6], wd[7], 0x5410));
            }
            if (c & 32) flush_rows(buf, keep + (c - 32) * 2, static_cast<int64_t>(p.ld) * 2, valid);
          }
        }
        if (lane < valid) {
          const size_t at = static_cast<size_t>(2 * t.nt + half) * p.ldp + row;
          p.pm[at] = m == NEG ? NEG : my;
          p.ps[at] = s;
          if (TWO) p.ps2[at] = s2;
          if (MODE == HEAD_KEEP) p.pk[at] = mine;
        }
      } else {
        // dx: its token's row, or an fp32 part; dw: added to earlier pieces', in its type
        const int token = !t.dw && p.splits == 1 && lane < valid ? p.idx[p.row0 + row] : 0;
        if (!take()) { ok = false; break; }
        const uint32_t acc = lanes + a * BN;
        if (valid < 1) { release(); continue; }
        const bool none = t.k0 == t.k1;   // no products: the accumulator holds nothing
        const bool parts = !t.dw && p.splits > 1;
        float* sum = p.out_bf16 ? p.acc : static_cast<float*>(p.dw);
        const bool to_sum = t.dw && (!p.out_bf16 || !p.last);
        const bool adds = t.dw && (!p.first || to_sum);
        const int lim = min(hw, p.d - c0);
        if (p.out_bf16 && !parts && !adds) {
          // the usual end: 64 columns of bf16 at a time
          for (int c = 0; c < lim; c += 64) {
            uint32_t v[64];
            tmem_ld32(acc + c, v);
            tmem_ld32(acc + c + 32, v + 32);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float f[8];
#pragma unroll
              for (int i8 = 0; i8 < 8; ++i8) f[i8] = none ? 0.f : g * __uint_as_float(v[8 * j + i8]);
              *reinterpret_cast<uint4*>(own_piece(buf, j)) = pack16(f, __nv_bfloat16());
            }
            if (t.dw) {
              flush_rows(buf, reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(p.dw) +
                                                      (static_cast<int64_t>(t.m0) + quarter * 32) * p.d + c0 + c),
                         static_cast<int64_t>(p.d) * 2, valid);
              continue;
            }
            __syncwarp();
#pragma unroll
            for (int it8 = 0; it8 < 8; ++it8) {
              const int r = it8 * 4 + lane / 8, q = lane & 7;
              const int to = __shfl_sync(0xffffffffu, token, r);
              if (r < valid)
                st_v4(static_cast<__nv_bfloat16*>(p.dx) + static_cast<int64_t>(to) * p.d + c0 + c + 8 * q,
                      *reinterpret_cast<const uint4*>(buf + r * 32 + 4 * (q ^ (r & 7))));
            }
            __syncwarp();
          }
          release();
          continue;
        }
        // fp32: 32 columns at a time through shared memory, eight lanes a row
        for (int c = 0; c < lim; c += 32) {
          uint32_t v[32];
          tmem_ld32(acc + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float f[4];
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
              f[i4] = none ? 0.f : (parts ? 1.f : g) * __uint_as_float(v[4 * j + i4]);
            *reinterpret_cast<uint4*>(own_piece(buf, j)) = pack16(f, 0.f);
          }
          __syncwarp();
          const int64_t at = (static_cast<int64_t>(t.m0) + quarter * 32) * p.d + c0 + c;   // (dw, parts)
#pragma unroll
          for (int it8 = 0; it8 < 8; ++it8) {
            const int r = it8 * 4 + lane / 8, q = lane & 7;
            const int to = __shfl_sync(0xffffffffu, token, r);
            if (r >= valid) continue;
            float4 f = *reinterpret_cast<const float4*>(buf + r * 32 + 4 * (q ^ (r & 7)));
            const int64_t mine = at + static_cast<int64_t>(r) * p.d + 4 * q;
            if (parts) {
              *reinterpret_cast<float4*>(p.part + static_cast<int64_t>(t.split) * p.piece * p.d + mine) = f;
            } else if (!t.dw) {
              *reinterpret_cast<float4*>(static_cast<float*>(p.dx) + static_cast<int64_t>(to) * p.d + c0 + c + 4 * q) = f;
            } else {
              if (!p.first) {
                const float4 o = *reinterpret_cast<const float4*>(sum + mine);
                f.x += o.x; f.y += o.y; f.z += o.z; f.w += o.w;
              }
              if (to_sum) *reinterpret_cast<float4*>(sum + mine) = f;
              else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.dw) + mine) =
                    make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
            }
          }
          __syncwarp();
        }
        release();
      }
    }
    if (!ok) {
      if (lane == 0) latch_error(p.dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  if (PAIR) cluster_sync(); else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tbase, kTmemCols);
    else tmem_dealloc(tbase, kTmemCols);
  }
}

template <int MODE, bool PAIR, bool TWO>
int launch_one(const LaunchCtx& ctx, const CUtensorMap& ma, const CUtensorMap& ma2,
               const CUtensorMap& mb, const CUtensorMap& mb2, const GemmArgs& g) {
  auto kern = head_gemm_kernel<MODE, PAIR, TWO>;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = ctx.stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = PAIR ? attr : attr + 1;
  cfg.numAttrs = PAIR ? 2 : 1;
  struct Fit { cudaError_t err; int n_pairs; };
  static PerDevice<Fit> fits;
  const Fit& fit = fits.get(ctx.device, [&](Fit& f) {
    f.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (f.err == cudaSuccess && MODE != HEAD_GRADS) {
      // the split of the registers adds up to a launch with this many: another count
      // (of another compiler) would leave warps waiting for theirs
      cudaFuncAttributes fa;
      f.err = cudaFuncGetAttributes(&fa, kern);
      if (f.err == cudaSuccess && fa.numRegs != kLaunchRegs) f.err = cudaErrorLaunchOutOfResources;
    }
    if (PAIR && f.err == cudaSuccess) {
      cfg.gridDim = dim3(2 * (ctx.num_sms / 2));
      f.err = cudaOccupancyMaxActiveClusters(&f.n_pairs, kern, &cfg);
    }
  });
  if (fit.err != cudaSuccess || (PAIR && fit.n_pairs < 1)) return OCCULT_ERR_CUDA;
  cfg.gridDim = dim3(PAIR ? 2 * fit.n_pairs : ctx.num_sms);
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, ma, ma2, mb, mb2, g));
}

GemmArgs base_args(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0) {
  GemmArgs g{};
  g.cnt = reinterpret_cast<const HeadCounts*>(a.ws + p.o_cnt);
  g.T = p.T; g.row0 = row0; g.piece = p.piece; g.V = p.V; g.d = p.d;
  g.E = p.E; g.ldp = p.piece; g.ld = p.ld;
  g.idx = reinterpret_cast<const int32_t*>(a.ws + p.o_idx);
  g.ent = reinterpret_cast<const int32_t*>(a.ws + p.o_ent);
  g.zt = reinterpret_cast<float*>(a.ws + p.o_zt);
  g.pm = reinterpret_cast<float*>(a.ws + p.o_m);
  g.ps = reinterpret_cast<float*>(a.ws + p.o_s);
  g.ps2 = reinterpret_cast<float*>(a.ws + p.o_s2);
  g.pk = reinterpret_cast<float*>(a.ws + p.o_mk);
  g.kept = reinterpret_cast<uint16_t*>(a.ws + p.o_kept);
  g.inv_tau = 1.f / p.tau; g.q_inv = 1.f / p.q_step;
  g.part = reinterpret_cast<float*>(a.ws + p.o_part);
  g.dloss = a.dloss; g.coef = p.coef; g.coef_kd = p.coef_kd; g.coef_z = p.coef_z; g.tau = p.tau;
  g.dev_err = ctx.dev_err;
  return g;
}
// Stages of single CTAs: A's rows and `b_rows` of B (multiples of 8, so that stages start on
// 1024 bytes).
void ring(GemmArgs& g, int b_rows) {
  g.stage_bytes = kABytes + b_rows * BK * 2;
  g.stages = std::min(kMaxStages, kRingBytes / g.stage_bytes);
}
// rows of the compact copy of x
int64_t copy_rows(const HeadPlan& p) {
  return (static_cast<int64_t>(std::max(1, p.T)) + kHeadRowAlign - 1) / kHeadRowAlign * kHeadRowAlign;
}
// Two row tiles or more go to CTA pairs.
bool paired(const HeadPlan& p) { return std::min(p.piece, p.T) > BM; }

}  // namespace

int launch_head_logits_bf16(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0) {
  const bool pair = paired(p);
  CUtensorMap mx, mc, mw;
  int rc = tensor_map_bf16(&mx, a.x, p.T, p.d, BK, BM);
  if (!rc) rc = tensor_map_bf16(&mc, a.ws + p.o_xc, copy_rows(p), p.d, BK, BM);
  if (!rc) rc = tensor_map_bf16(&mw, a.w, p.V, p.d, BK, pair ? p.bn / 2 : p.bn);
  if (rc) return rc;
  GemmArgs g = base_args(ctx, p, a, row0);
  g.bn = p.bn;
  g.n_tiles = p.n_tiles;
  // Products to a sum in TMEM: 512 in pairs (with 256 the epilogue has to keep up with twice as
  // many: 4096 tokens x 2048 x 50304 took 520 us for 475), 256 in single CTAs, which wait for
  // the weights anyway, and whose few tokens' losses do not average the truncation out (with
  // 128 the accumulators' way to registers and back is what they wait for: 11 x 3008 x 3951
  // took 25 us)
  g.seg = pair ? 8 : 4;
  ring(g, p.bn);
#define OCCULT_HEAD_LOGITS(MODE)                                                           \
  (pair ? (p.two ? launch_one<MODE, true, true>(ctx, mx, mc, mw, mw, g)                    \
                 : launch_one<MODE, true, false>(ctx, mx, mc, mw, mw, g))                  \
        : (p.two ? launch_one<MODE, false, true>(ctx, mx, mc, mw, mw, g)                   \
                 : launch_one<MODE, false, false>(ctx, mx, mc, mw, mw, g)))
  return p.step ? OCCULT_HEAD_LOGITS(HEAD_KEEP) : OCCULT_HEAD_LOGITS(HEAD_STATS);
#undef OCCULT_HEAD_LOGITS
}

int launch_head_grads_bf16(const LaunchCtx& ctx, const HeadPlan& p, const HeadArgs& a, int row0,
                           bool first, bool last) {
  CUtensorMap mz, mw, mx, mc;
  int rc = tensor_map_bf16(&mz, a.ws + p.o_kept, p.piece, p.ld, 64, 64);
  if (!rc) rc = tensor_map_bf16(&mw, a.w, p.V, p.d, 64, 64);
  if (!rc) rc = tensor_map_bf16(&mx, a.x, p.T, p.d, 64, 64);
  if (!rc) rc = tensor_map_bf16(&mc, a.ws + p.o_xc, copy_rows(p), p.d, 64, 64);
  if (rc) return rc;
  GemmArgs g = base_args(ctx, p, a, row0);
  g.bn = p.d <= 128 ? 128 : BN;
  g.n_tiles = (p.d + g.bn - 1) / g.bn;
  g.splits = head_splits(p, a);
  g.seg = 1 << 30;
  g.dx = a.dx;
  g.dw = a.dw;
  g.acc = reinterpret_cast<float*>(a.ws + p.o_acc);
  g.out_bf16 = p.grad_dtype == OCCULT_BF16;
  g.first = first;
  g.last = last;
  return launch_one<HEAD_GRADS, true, false>(ctx, mz, mx, mw, mc, g);
}

}  // namespace occult
