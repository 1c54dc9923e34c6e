// The router's balance loss: per-expert counts, expert, device and z terms over
// groups of tokens, and the gradient with respect to the logits.
//
// Everything is a softmax of each token's row, so both directions are bound by the
// logits they read (and the gradients they write); at the sizes of a router both
// often sit in L2 and what counts is latency.  The loss of a small batch is one launch
// of a cluster that adds its CTAs' sums up over shared memory, else it is two: tiles of
// tokens leave partial sums and counts, then one CTA a group adds them up.  Logits,
// sums and gradients are fp32 throughout, counts are integers.
//
// Measured on one GB300, loss + gradient (added to what is there): 32768 tokens, 64
// experts, top-8 9.9 + 3.7 us (the first launch 3.6 us, bound by two steps of loads;
// the second by its chain of sums in one CTA); 131072 tokens, 256 experts, masked, 32
// sequences 35 + 56 us = 3.9 and 7.2 TB/s (the logits twice, the gradient in and out);
// 256 tokens, 8 experts 4.0 + 1.7 us.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kTileThreads = 512;
constexpr int kOneThreads = 1024;
constexpr int kOneSteps = 2, kClusterSteps = 4;    // steps of a CTA
constexpr int kSumThreads = 1024;
constexpr int kSumWarps = kSumThreads / 32;
static_assert(kSumWarps <= 32 && kSumThreads >= OCCULT_MAX_EXPERTS,
              "a lane a warp's word, a thread an expert");
constexpr int kGradThreads = 256;
// Tiles of a batch: two CTAs an SM where the groups have their own second passes, one
// where a single CTA adds all of them up (11.2 us at 304 tiles, 10.3 at 152 for the loss
// of 32768 tokens and 64 experts in one group; 36 against 63 us with 32 groups of 4096)
// and the first pass is not long: 2^20 lanes of tokens (131072 tokens of 33 experts 16 us
// at 304, 19 at 152, of 256 experts 38 and 49; half of that, 65536 of 64, 12.4 either way).
constexpr int kMaxTiles = 304, kMaxTilesOne = 152;
constexpr int64_t kManyLanes = 1 << 20;
constexpr int kMinTile = 64;     // tokens

// Workspace, in words: probability sums and counts [tiles][Ne], then for every tile
// its sum of lse^2 and its tokens, then {expert, device, sum lse^2} of every group
// and the counter of finished groups.
struct Tiles {
  int per_group, len;
  int64_t n;
};
__host__ __device__ inline Tiles tiles_of(int T, int L, int G, int lp) {
  const int tokens = T < L ? (T > 0 ? T : 1) : L;
  // as many tiles as keep every SM busy, at least kMinTile tokens each
  int per = G == 1 && static_cast<int64_t>(T) * lp < kManyLanes ? kMaxTilesOne : kMaxTiles / G;
  const int most = (tokens + kMinTile - 1) / kMinTile;
  per = per < 1 ? 1 : (per > most ? most : per);
  Tiles t;
  t.len = (tokens + per - 1) / per;
  t.per_group = (tokens + t.len - 1) / t.len;
  t.n = static_cast<int64_t>(t.per_group) * G;
  return t;
}
struct Work {
  float* p_sum;
  int* count;
  float* sq;
  int* n;
  float* terms;
  unsigned* done;
};
__host__ __device__ inline Work work_of(float* ws, int64_t tiles, int Ne, int G) {
  Work w;
  w.p_sum = ws;
  w.count = reinterpret_cast<int*>(ws + tiles * Ne);
  w.sq = ws + 2 * tiles * Ne;
  w.n = reinterpret_cast<int*>(w.sq + tiles);
  w.terms = w.sq + 2 * tiles;
  w.done = reinterpret_cast<unsigned*>(w.terms + 3 * static_cast<int64_t>(G));
  return w;
}

// One token's row over LP lanes: lane s holds experts 4 (h LP + s) + i, h < 2, i < 4,
// so that a row is read as consecutive 16-byte words (`vec`: rows are whole ones), or
// experts j LP + s, j < 8, consecutive words (131072 x 255, loss + gradient: 39 + 64 us;
// with the other order 54 + 73).
template <int LP>
__device__ __forceinline__ int expert_of(int sub, int j, bool vec) {
  return vec ? 4 * ((j >> 2) * LP + sub) + (j & 3) : j * LP + sub;
}
template <int LP>
__device__ __forceinline__ void load_row(const float* row, int Ne, bool vec, int sub, float pad,
                                         float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 q = make_float4(pad, pad, pad, pad);
      if (4 * (h * LP + sub) < Ne)
        q = *reinterpret_cast<const float4*>(row + 4 * (h * LP + sub));
      v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = j * LP + sub < Ne ? row[j * LP + sub] : pad;
  }
}
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 pair(const float (&v)[8], int i) { return make_float2(v[i], v[i + 1]); }
__device__ __forceinline__ void put(float (&v)[8], int i, float2 x) { v[i] = x.x; v[i + 1] = x.y; }
__device__ __forceinline__ float minus_inf() { return -__int_as_float(0x7f800000); }

// v = exp(z - max), *inv = 1 / their sum; returns log sum exp.  The exponentials are
// powers of two of (z - max) log2 e: that product's rounding makes a probability 2^-m
// of the largest m 2^-24 of itself less exact than expf would, which costs sums and
// gradients nothing, at half of the instructions.
template <int LP>
__device__ __forceinline__ float softmax_row(float (&v)[8], float* inv) {
  constexpr float kLog2e = 1.4426950408889634f;
  float mx = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float2 z2 = two(0.f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 y = __fmul2_rn(__fadd2_rn(pair(v, i), two(-mx)), two(kLog2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i + 1]) : "f"(y.y));
    z2 = __fadd2_rn(z2, pair(v, i));
  }
  float z = z2.x + z2.y;
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  *inv = __fdividef(1.f, z);  // z is about 1 .. 256
  return mx + __logf(z);      // z is 1 .. 256: within 3 * 2^-21, and the sum's rounding
}

// What a tile, a group or a batch of one CTA adds up to, in shared memory.
struct Sums {
  float p[OCCULT_MAX_EXPERTS];  // sum of probabilities
  int c[OCCULT_MAX_EXPERTS];    // slots
  float sq;                     // sum of lse^2
  int n;                        // tokens
};

// The sums of tokens [t0, t1) by a CTA of THREADS, in a fixed order.
template <int LP, int THREADS>
struct TileScratch {
  float p[THREADS / 32][LP * 8];
  float sq[THREADS / 32];
  int n[THREADS / 32];
};
template <int LP, int THREADS>
__device__ __forceinline__ void sum_tile(const BalanceArgs& a, int64_t t0, int64_t t1,
                                         TileScratch<LP, THREADS>& x, Sums& out) {
  constexpr int kWarps = THREADS / 32;
  constexpr int kTok = 32 / LP;            // tokens of a row of lanes
  constexpr int kRows = 1;                 // of a step (2: registers spill, 35.6 -> 42.1 us)
  constexpr int kStep = kWarps * kTok * kRows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LP;
  const bool vec = a.Ne % 4 == 0;
  for (int e = threadIdx.x; e < a.Ne; e += THREADS) out.c[e] = 0;
  __syncthreads();
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  float sq = 0.f;
  int n = 0;
  // the next step's rows, masks and ids are on their way while this one's are summed
  // (lanes past the end run along on the first row; what a masked row gives is dropped)
  float next[kRows][8];
  bool next_on[kRows];
  int next_id[kRows][2];
  auto fetch = [&](int64_t b) {
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int64_t t = b + q * (kWarps * kTok) + lane / LP;
      const bool in = t < t1;
      load_row<LP>(a.logits + (in ? t : t0) * a.Ne, a.Ne, vec, sub, minus_inf(), next[q]);
      next_on[q] = in && (!a.mask || a.mask[t]);
#pragma unroll
      for (int r = 0; r < 2; ++r)
        next_id[q][r] = in && sub + r * LP < a.k ? a.ids[t * a.k + sub + r * LP] : -1;
    }
  };
  int64_t b = t0 + warp * kTok;
  if (b < t1) fetch(b);
  for (; b < t1; b += kStep) {
    float v[kRows][8], inv[kRows], lse[kRows];
    bool on[kRows];
    int id[kRows][2];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[q][i] = next[q][i];
      on[q] = next_on[q];
      id[q][0] = next_id[q][0];
      id[q][1] = next_id[q][1];
    }
    if (b + kStep < t1) fetch(b + kStep);
#pragma unroll
    for (int q = 0; q < kRows; ++q) lse[q] = softmax_row<LP>(v[q], &inv[q]);
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if (!on[q]) continue;
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        put(acc, i, __ffma2_rn(pair(v[q], i), two(inv[q]), pair(acc, i)));
      if (sub == 0) { sq = fmaf(lse[q], lse[q], sq); ++n; }
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (static_cast<unsigned>(id[q][r]) < static_cast<unsigned>(a.Ne))
          atomicAdd(&out.c[id[q][r]], 1);
    }
    __syncwarp();
  }
#pragma unroll
  for (int o = 16; o >= LP; o >>= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    sq += __shfl_xor_sync(0xffffffffu, sq, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane < LP)
#pragma unroll
    for (int i = 0; i < 8; ++i) x.p[warp][expert_of<LP>(lane, i, vec)] = acc[i];
  if (lane == 0) { x.sq[warp] = sq; x.n[warp] = n; }
  __syncthreads();
  for (int e = threadIdx.x; e < a.Ne; e += THREADS) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += x.p[i][e];
    out.p[e] = s;
  }
  if (warp == kWarps - 1) {  // (no expert's warp: 256 of them are eight warps' threads)
    float s = lane < kWarps ? x.sq[lane] : 0.f;
    const int m = __reduce_add_sync(0xffffffffu, lane < kWarps ? x.n[lane] : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) { out.sq = s; out.n = m; }
  }
  __syncthreads();
}

// A group's counts, gradient weights and loss terms from its sums (`s.p` is
// overwritten): 1 / A and the CTA's threads given; terms by its first thread.
struct GroupScratch {
  float f[OCCULT_MAX_EXPERTS];
  float fd[OCCULT_MAX_VDEV], sd[OCCULT_MAX_VDEV];
  int dev[OCCULT_MAX_EXPERTS];  // expert_to_vdev, filled by the caller
};
__device__ __forceinline__ void finish_group(const BalanceArgs& a, int64_t g, Sums& s,
                                             GroupScratch& x, float inv_a, float (&terms)[3]) {
  const int tid = threadIdx.x;
  const float inv_g = 1.f / static_cast<float>(s.n > 0 ? s.n : 1);
  const float scale = static_cast<float>(a.Ne) / static_cast<float>(a.k) * inv_g;
  for (int e = tid; e < a.Ne; e += blockDim.x) {
    a.counts[g * a.Ne + e] = s.c[e];
    x.f[e] = static_cast<float>(s.c[e]) * scale;
    s.p[e] *= inv_g;
  }
  __syncthreads();
  // a warp a device
  for (int d = tid >> 5; d < a.Nd; d += blockDim.x / 32) {
    float f = 0.f, S = 0.f, m = 0.f;
    for (int e = tid & 31; e < a.Ne; e += 32)
      if (x.dev[e] == d) { f += x.f[e]; S += s.p[e]; m += 1.f; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      f += __shfl_xor_sync(0xffffffffu, f, o);
      S += __shfl_xor_sync(0xffffffffu, S, o);
      m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if ((tid & 31) == 0) { x.fd[d] = m > 0.f ? f / m : 0.f; x.sd[d] = S; }
  }
  __syncthreads();
  for (int e = tid; e < a.Ne; e += blockDim.x) {
    const int d = x.dev[e];
    const float fd = static_cast<unsigned>(d) < static_cast<unsigned>(a.Nd) ? x.fd[d] : 0.f;
    a.grad_w[g * a.Ne + e] = (a.coef * x.f[e] + a.coef_dev * fd) * inv_g * inv_a;
  }
  if (tid < 32) {
    float expert = 0.f, device = tid < a.Nd ? x.fd[tid] * x.sd[tid] : 0.f;
    for (int e = tid; e < a.Ne; e += 32) expert += x.f[e] * s.p[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      expert += __shfl_xor_sync(0xffffffffu, expert, o);
      device += __shfl_xor_sync(0xffffffffu, device, o);
    }
    terms[0] = expert;
    terms[1] = device;
    terms[2] = s.sq;
  }
}
__device__ __forceinline__ void write_loss(const BalanceArgs& a, const float (&terms)[3], float inv_a,
                                           float inv_n) {
  const float expert = terms[0] * inv_a, device = terms[1] * inv_a, z = terms[2] * inv_n;
  a.loss[0] = a.coef * expert + a.coef_dev * device + a.coef_z * z;
  a.loss[1] = expert;
  a.loss[2] = device;
  a.loss[3] = z;
  a.grad_w[static_cast<size_t>(a.G) * a.Ne] = 2.f * a.coef_z * inv_n;
}

// A word of another CTA's shared memory, at the offset of `p` in this CTA's.
__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(smem_addr_in_rank(p, rank)));
  return v;
}

// A batch of one group and not too many tokens in one launch: the grid is one cluster
// (or one CTA), whose CTAs each sum a tile and whose first then reads the others' sums.
template <int LP>
__global__ void __launch_bounds__(kOneThreads, 1) balance_cluster_kernel(BalanceArgs a) {
  __shared__ TileScratch<LP, kOneThreads> s_tile;
  __shared__ Sums s_sums;
  __shared__ GroupScratch s_group;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, rank = blockIdx.x, ctas = gridDim.x;
  for (int e = threadIdx.x; e < a.Ne; e += kOneThreads) s_group.dev[e] = a.e2v[e];
  const int64_t len = (static_cast<int64_t>(a.T) + ctas - 1) / ctas, t0 = rank * len;
  sum_tile<LP, kOneThreads>(a, t0, min(static_cast<int64_t>(a.T), t0 + len), s_tile, s_sums);
  if (ctas > 1) {
    cluster_sync();
    float p = 0.f, sq = 0.f;
    int c = 0, n = 0;
    if (rank == 0) {
      if (static_cast<int>(threadIdx.x) < a.Ne) {
#pragma unroll 16
        for (int r = 0; r < ctas; ++r) {
          p += __uint_as_float(ld_cluster(&s_sums.p[threadIdx.x], r));
          c += static_cast<int>(ld_cluster(&s_sums.c[threadIdx.x], r));
        }
      }
      if (lane < ctas) {
        sq = __uint_as_float(ld_cluster(&s_sums.sq, lane));
        n = static_cast<int>(ld_cluster(&s_sums.n, lane));
      }
    }
    cluster_sync();  // all of it is read: the CTAs may end, the first may overwrite
    if (rank != 0) return;
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (static_cast<int>(threadIdx.x) < a.Ne) {
      s_sums.p[threadIdx.x] = p;
      s_sums.c[threadIdx.x] = c;
    }
    if (threadIdx.x == 0) { s_sums.sq = sq; s_sums.n = n; }
    __syncthreads();
  }
  float terms[3];
  finish_group(a, 0, s_sums, s_group, 1.f, terms);
  if (threadIdx.x == 0)
    write_loss(a, terms, 1.f, 1.f / static_cast<float>(s_sums.n > 0 ? s_sums.n : 1));
}

template <int LP>
int launch_cluster(const LaunchCtx& ctx, const BalanceArgs& a, int ctas) {
  void (*kernel)(BalanceArgs) = balance_cluster_kernel<LP>;
  if (ctas == 1) return cuda_status(launch_pdl(kernel, 1, kOneThreads, 0, ctx.stream, a));
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return OCCULT_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = ctas;
  cfg.blockDim = kOneThreads;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

// Pass 1: CTA x of group y takes one tile of the group's tokens.  131072 x 256: 27 us,
// near both bounds (5.0 TB/s and two thirds of the issue slots, at 155 instructions a token
// and warp); a token a warp with scalar loads and expf took 55 us.
template <int LP>
__global__ void __launch_bounds__(kTileThreads, 2)
balance_tiles_kernel(BalanceArgs a, Tiles tiles) {
  __shared__ TileScratch<LP, kTileThreads> s_tile;
  __shared__ Sums s_sums;
  pdl_wait();
  pdl_trigger();
  const Work w = work_of(a.ws, tiles.n, a.Ne, a.G);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *w.done = 0;
  for (int g = blockIdx.y; g < a.G; g += gridDim.y) {
    const int64_t g0 = static_cast<int64_t>(g) * a.L;
    const int64_t g1 = min(static_cast<int64_t>(a.T), g0 + a.L);
    const int64_t t0 = g0 + static_cast<int64_t>(blockIdx.x) * tiles.len;
    sum_tile<LP, kTileThreads>(a, t0, min(g1, t0 + tiles.len), s_tile, s_sums);
    const int64_t tile = static_cast<int64_t>(g) * tiles.per_group + blockIdx.x;
    for (int e = threadIdx.x; e < a.Ne; e += kTileThreads) {
      w.p_sum[tile * a.Ne + e] = s_sums.p[e];
      w.count[tile * a.Ne + e] = s_sums.c[e];
    }
    if (threadIdx.x == 0) { w.sq[tile] = s_sums.sq; w.n[tile] = s_sums.n; }
    __syncthreads();
  }
}

// Pass 2, one CTA a group: the group's sums over its tiles, its counts, the
// gradient's weights and its loss terms; the last CTA to finish adds those up.
__global__ void __launch_bounds__(kSumThreads) balance_groups_kernel(BalanceArgs a, Tiles tiles) {
  __shared__ float s_part[kSumThreads];
  __shared__ int s_cpart[kSumThreads];
  __shared__ Sums s_sums;
  __shared__ GroupScratch s_group;
  __shared__ long long s_tok[kSumWarps];
  __shared__ float s_sq[kSumWarps];
  __shared__ float s_terms[kSumWarps][3];
  __shared__ int s_n[kSumWarps];
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  for (int e = tid; e < a.Ne; e += kSumThreads) s_group.dev[e] = a.e2v[e];
  const Work w = work_of(a.ws, tiles.n, a.Ne, a.G);
  int cols = 32;  // a power of two of at least Ne threads a slice of the tiles
  while (cols < a.Ne) cols *= 2;
  const int col = tid % cols, slice = tid / cols, slices = kSumThreads / cols;
  float inv_a = 1.f, inv_n = 1.f;
  long long tok = 0;
  for (int g = blockIdx.x; g < a.G; g += gridDim.x) {
    const int64_t tile0 = static_cast<int64_t>(g) * tiles.per_group;
    float s = 0.f, sq = 0.f;
    int c = 0, n = 0;
    if (col < a.Ne) {
#pragma unroll 10
      for (int i = slice; i < tiles.per_group; i += slices) {
        s += w.p_sum[(tile0 + i) * a.Ne + col];
        c += w.count[(tile0 + i) * a.Ne + col];
      }
    }
    for (int i = tid; i < tiles.per_group; i += kSumThreads) {
      sq += w.sq[tile0 + i];
      n += w.n[tile0 + i];
    }
    if (g == static_cast<int>(blockIdx.x)) {
      // once: tokens, and groups that have any, over the whole batch (a group's tiles by
      // one thread when they are few, by a warp when many); both are below 2^31
      if (a.G == 1) {
        tok = n;  // (summed below)
      } else {
        const int wide = tiles.per_group > 16 ? 32 : 1, part = tid % wide;
        for (int k = tid / wide; k < a.G; k += kSumThreads / wide) {
          int m = 0;
#pragma unroll 4
          for (int i = part; i < tiles.per_group; i += wide)
            m += w.n[static_cast<int64_t>(k) * tiles.per_group + i];
          if (wide == 32) m = __reduce_add_sync(0xffffffffu, m);
          if (part == 0) tok += m + (static_cast<long long>(m > 0) << 32);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tok += __shfl_xor_sync(0xffffffffu, tok, o);
      if (lane == 0) s_tok[warp] = tok;
    }
    s_part[tid] = s;
    s_cpart[tid] = c;
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) { s_sq[warp] = sq; s_n[warp] = n; }
    __syncthreads();
    if (tid < a.Ne) {
      for (int i = 1; i < slices; ++i) {
        s += s_part[i * cols + tid];
        c += s_cpart[i * cols + tid];
      }
      s_sums.p[tid] = s;
      s_sums.c[tid] = c;
    }
    // the last warp adds up the scalars
    if (warp == kSumWarps - 1) {
      const bool have = lane < kSumWarps;
      sq = have ? s_sq[lane] : 0.f;
      n = __reduce_add_sync(0xffffffffu, have ? s_n[lane] : 0);
      tok = have ? s_tok[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        tok += __shfl_xor_sync(0xffffffffu, tok, o);
      }
      if (lane == 0) { s_sums.sq = sq; s_sums.n = n; }
      if (have) s_tok[lane] = lane == 0 ? tok : 0;  // (added up again for the next group)
    }
    __syncthreads();
    tok = s_tok[0];
    const int N = static_cast<int>(tok & 0xffffffffll);
    const int A = a.G == 1 ? 1 : static_cast<int>(tok >> 32);
    inv_a = 1.f / static_cast<float>(A > 0 ? A : 1);
    inv_n = 1.f / static_cast<float>(N > 0 ? N : 1);
    float terms[3];
    finish_group(a, g, s_sums, s_group, inv_a, terms);
    if (tid == 0) {
      if (a.G == 1) write_loss(a, terms, inv_a, inv_n);
#pragma unroll
      for (int i = 0; i < 3; ++i) w.terms[3 * static_cast<int64_t>(g) + i] = terms[i];
    }
    __syncthreads();
  }
  if (a.G == 1) return;
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(w.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float v[3] = {0.f, 0.f, 0.f};
  for (int g = tid; g < a.G; g += kSumThreads)
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += __ldcg(&w.terms[3 * static_cast<int64_t>(g) + i]);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (lane == 0) s_terms[warp][i] = v[i];
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      v[i] = 0.f;
      for (int k = 0; k < kSumWarps; ++k) v[i] += s_terms[k][i];
    }
    write_loss(a, v, inv_a, inv_n);
  }
}

// dz = dloss (p (w - w . p) + w_z lse p), LP lanes a token as in the first pass.  131072
// x 256 added to a gradient: 56 us = 7.2 TB/s, bound by memory (85 us with the gradient
// read after the softmax and a 64-bit division a token).  Four CTAs an SM: three (the
// registers it would take) 65 us, five (spills) 63 us.
template <int LP, bool VEC>
__global__ void __launch_bounds__(kGradThreads, 4) balance_grad_kernel(BalanceArgs a) {
  constexpr int kTok = 32 / LP;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, sub = lane % LP;
  const float up = a.dloss ? *a.dloss : 1.f;
  const float wz = a.grad_w[static_cast<size_t>(a.G) * a.Ne];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kGradThreads / 32) * kTok;
  int64_t b = (static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5)) * kTok;
  // the next step's logits, and what the gradient is added to, are on their way while
  // this one's are worked on
  float next[8], next_old[8];
  bool next_on = false;
  auto fetch = [&](int64_t b) {
    const int64_t t = b + lane / LP;
    const bool in = t < a.T;
    load_row<LP>(a.logits + (in ? t : b) * a.Ne, a.Ne, VEC, sub, minus_inf(), next);
    if (a.accumulate) load_row<LP>(a.dlogits + (in ? t : b) * a.Ne, a.Ne, VEC, sub, 0.f, next_old);
    next_on = in && (!a.mask || a.mask[t]);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) next_old[i] = 0.f;
  if (b < a.T) fetch(b);
  for (; b < a.T; b += step) {
    const int64_t t = b + lane / LP;
    const bool in = t < a.T, on = next_on;
    float v[8], old[8], w[8], inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) { v[i] = next[i]; old[i] = next_old[i]; }
    if (b + step < a.T) fetch(b + step);
    // (weights of a group's row: L1)
    const unsigned g = a.G == 1 ? 0u
                                : static_cast<unsigned>(in ? t : b) / static_cast<unsigned>(a.L);
    load_row<LP>(a.grad_w + static_cast<size_t>(g) * a.Ne, a.Ne, VEC, sub, 0.f, w);
    const float lse = softmax_row<LP>(v, &inv);
    float2 dot2 = two(0.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      put(v, i, __fmul2_rn(pair(v, i), two(inv)));
      dot2 = __ffma2_rn(pair(v, i), pair(w, i), dot2);
    }
    float dot = dot2.x + dot2.y;
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (!in || (!on && a.accumulate)) continue;
    const float shift = wz * lse - dot;
    float* out = a.dlogits + t * a.Ne;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 dz = __ffma2_rn(__fmul2_rn(pair(v, i), two(up)),
                                   __fadd2_rn(pair(w, i), two(shift)), pair(old, i));
      put(v, i, on ? dz : two(0.f));
    }
    if (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (4 * (h * LP + sub) < a.Ne)
          *reinterpret_cast<float4*>(out + 4 * (h * LP + sub)) =
              make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * LP + sub < a.Ne) out[i * LP + sub] = v[i];
    }
  }
}

// Lanes a token: eight of its experts and two of its slots each.  Loss + gradient, us with
// eight lanes at least and so: 131072 tokens of 8 experts 16.4 + 9.7 and 8.8 + 2.6, of 24
// experts 16.5 + 9.8 and 12.1 + 6.5, 256 of 8 experts 4.8 + 1.8 and 4.0 + 1.6.
int lanes_of(int Ne, int k) {
  int lp = 1;
  while (lp < 32 && (8 * lp < Ne || 2 * lp < k)) lp *= 2;
  return lp;
}
template <typename F>
int with_lanes(int lp, F f) {
  return lp == 1    ? f(std::integral_constant<int, 1>{})
         : lp == 2  ? f(std::integral_constant<int, 2>{})
         : lp == 4  ? f(std::integral_constant<int, 4>{})
         : lp == 8  ? f(std::integral_constant<int, 8>{})
         : lp == 16 ? f(std::integral_constant<int, 16>{})
                    : f(std::integral_constant<int, 32>{});
}

}  // namespace

int balance_groups(int T, int group_len, int* L) {
  *L = group_len > 0 ? group_len : (T > 0 ? T : 1);
  const int G = static_cast<int>((static_cast<int64_t>(T) + *L - 1) / *L);
  return G > 0 ? G : 1;
}

size_t balance_ws_bytes(const occult_desc_t& ds, int group_len) {
  int L;
  const int G = balance_groups(ds.T, group_len, &L);
  const Tiles t = tiles_of(ds.T, L, G, lanes_of(ds.n_experts, ds.top_k));
  return (static_cast<size_t>(t.n) * (2 * ds.n_experts + 2) + 3 * static_cast<size_t>(G) + 1) *
         sizeof(float);
}

int launch_balance_loss(const LaunchCtx& ctx, const BalanceArgs& a) {
  const int lp = lanes_of(a.Ne, a.k);
  // One launch for a batch of one group: by one CTA for two steps of all its warps (1024 /
  // lp tokens each), by a cluster of 16 for four of each (where the device has a place for
  // one: a partition of few SMs has not), two launches beyond that.
  // 64 experts, us by one CTA, the cluster, two launches: 4.8, 5.4, 6.1 for 256 tokens,
  // -, 6.7, 7.1 for 4096, -, 8.4, 8.4 for 8192, -, 11.3, 9.1 for 16384.
  const int64_t steps = (static_cast<int64_t>(a.T) * lp + kOneThreads - 1) / kOneThreads;
  const int one_launch = ctx.clusters ? kClusterSteps * kClusterCtas : kOneSteps;
  if (a.G == 1 && steps <= one_launch) {
    const int ctas = steps <= kOneSteps ? 1 : kClusterCtas;
    return with_lanes(lp, [&](auto n) { return launch_cluster<decltype(n)::value>(ctx, a, ctas); });
  }
  const Tiles tiles = tiles_of(a.T, a.L, a.G, lp);
  const dim3 grid(tiles.per_group, a.G < 65535 ? a.G : 65535);
  const int rc = with_lanes(lp, [&](auto n) {
    return cuda_status(launch_pdl(balance_tiles_kernel<decltype(n)::value>, grid, kTileThreads, 0,
                                  ctx.stream, a, tiles));
  });
  if (rc) return rc;
  return cuda_status(launch_pdl(balance_groups_kernel, a.G < ctx.num_sms ? a.G : ctx.num_sms,
                                kSumThreads, 0, ctx.stream, a, tiles));
}

int launch_balance_grad(const LaunchCtx& ctx, const BalanceArgs& a) {
  if (a.T == 0) return OCCULT_OK;
  const int lp = lanes_of(a.Ne, 1), tok = 32 / lp * (kGradThreads / 32);
  const int64_t need = (static_cast<int64_t>(a.T) + tok - 1) / tok;
  const int grid = static_cast<int>(need < ctx.num_sms * 16 ? need : ctx.num_sms * 16);
  // 16-byte words where rows are whole ones and the weights begin at one (those of one
  // layer of several, G Ne + 1 words apart, need not)
  const bool vec = a.Ne % 4 == 0 && reinterpret_cast<uintptr_t>(a.grad_w) % 16 == 0;
  return with_lanes(lp, [&](auto n) {
    constexpr int LP = decltype(n)::value;
    return cuda_status(launch_pdl(vec ? balance_grad_kernel<LP, true> : balance_grad_kernel<LP, false>,
                                  grid, kGradThreads, 0, ctx.stream, a));
  });
}

}  // namespace occult
