// The router's balance loss: per-expert counts, expert, device and z terms over
// groups of tokens, and the gradient with respect to the logits.
//
// Everything is a softmax of each token's row, so both directions are bound by the
// logits they read (and the gradients they write); at the sizes of a router both
// often sit in L2 and what counts is latency.  The loss is two launches: tiles of
// tokens leave partial sums and counts, then one CTA a group adds them up.
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kTileThreads = 512;
constexpr int kTileWarps = kTileThreads / 32;
constexpr int kSumThreads = 1024;
constexpr int kGradThreads = 256;
constexpr int kMaxTiles = 304;   // of a batch that is not cut into more groups
constexpr int kMinTile = 64;     // tokens

// Workspace, in words: probability sums and counts [tiles][Ne], then for every tile
// its sum of lse^2 and its tokens, then {expert, device, sum lse^2} of every group
// and the counter of finished groups.
struct Tiles {
  int per_group, len;
  int64_t n;
};
__host__ __device__ inline Tiles tiles_of(int T, int L, int G) {
  const int tokens = T < L ? (T > 0 ? T : 1) : L;
  // as many tiles as keep every SM busy, at least kMinTile tokens each
  int per = kMaxTiles / G;
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

// The softmax of one token by LP lanes, lane s of them holding experts 8s .. 8s+7:
// p gets exp(z - max) / sum; returns log sum exp.  `vec`: rows are whole float4s.
template <int LP>
__device__ __forceinline__ float softmax8(const float* row, int Ne, bool vec, int sub,
                                          float (&p)[8]) {
  const float NEG = -__int_as_float(0x7f800000);
  const int e0 = sub * 8;
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 v = make_float4(NEG, NEG, NEG, NEG);
      if (e0 + 4 * h < Ne) v = *reinterpret_cast<const float4*>(row + e0 + 4 * h);
      p[4 * h] = v.x; p[4 * h + 1] = v.y; p[4 * h + 2] = v.z; p[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = e0 + i < Ne ? row[e0 + i] : NEG;
  }
  float mx = p[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, p[i]);
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = e0 + i < Ne ? expf(p[i] - mx) : 0.f;
    z += p[i];
  }
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float inv = 1.f / z;
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] *= inv;
  return mx + logf(z);
}

// Pass 1: CTA x of group y takes one tile of the group's tokens.
template <int LP>
__global__ void __launch_bounds__(kTileThreads, 2)
balance_tiles_kernel(BalanceArgs a, Tiles tiles) {
  constexpr int kTok = 32 / LP;  // tokens of a warp's step
  __shared__ float s_p[kTileWarps][LP * 8];
  __shared__ int s_c[LP * 8];
  __shared__ float s_sq[kTileWarps];
  __shared__ int s_n[kTileWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LP;
  const bool vec = a.Ne % 4 == 0;
  const Work w = work_of(a.ws, tiles.n, a.Ne, a.G);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *w.done = 0;
  for (int e = threadIdx.x; e < LP * 8; e += kTileThreads) s_c[e] = 0;
  __syncthreads();
  for (int g = blockIdx.y; g < a.G; g += gridDim.y) {
    const int64_t g0 = static_cast<int64_t>(g) * a.L;
    const int64_t g1 = min(static_cast<int64_t>(a.T), g0 + a.L);
    const int64_t t0 = g0 + static_cast<int64_t>(blockIdx.x) * tiles.len;
    const int64_t t1 = min(g1, t0 + tiles.len);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    float sq = 0.f;
    int n = 0;
#pragma unroll 2
    for (int64_t b = t0 + warp * kTok; b < t1; b += kTileWarps * kTok) {
      const int64_t t = b + lane / LP;
      const bool on = t < t1 && (!a.mask || a.mask[t]);
      float p[8];
      // (lanes of a token that takes no part run along on the tile's first row)
      const float lse = softmax8<LP>(a.logits + (on ? t : t0) * a.Ne, a.Ne, vec, sub, p);
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += p[i];
      if (sub == 0) { sq += lse * lse; ++n; }
      for (int j = sub; j < a.k; j += LP) {
        const int e = a.ids[t * a.k + j];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.Ne)) atomicAdd(&s_c[e], 1);
      }
    }
    __syncwarp();
    // the tokens of a step, then the warps, in a fixed order
#pragma unroll
    for (int o = 16; o >= LP; o >>= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (lane < LP)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_p[warp][lane * 8 + i] = acc[i];
    if (lane == 0) { s_sq[warp] = sq; s_n[warp] = n; }
    __syncthreads();
    const int64_t tile = static_cast<int64_t>(g) * tiles.per_group + blockIdx.x;
    for (int e = threadIdx.x; e < a.Ne; e += kTileThreads) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kTileWarps; ++i) s += s_p[i][e];
      w.p_sum[tile * a.Ne + e] = s;
      w.count[tile * a.Ne + e] = s_c[e];
      s_c[e] = 0;
    }
    if (threadIdx.x == 0) {
      float s = 0.f;
      int m = 0;
      for (int i = 0; i < kTileWarps; ++i) { s += s_sq[i]; m += s_n[i]; }
      w.sq[tile] = s;
      w.n[tile] = m;
    }
    __syncthreads();
  }
}

// Sums over the CTA (kSumThreads); every thread gets them.
__device__ __forceinline__ float cta_sum(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ long long cta_sum(long long v, long long* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Pass 2, one CTA a group: the group's sums over its tiles, its counts, the
// gradient's weights and its loss terms; the last CTA to finish adds those up.
__global__ void __launch_bounds__(kSumThreads) balance_groups_kernel(BalanceArgs a, Tiles tiles) {
  __shared__ float s_part[kSumThreads];
  __shared__ int s_cpart[kSumThreads];
  __shared__ float s_f[OCCULT_MAX_EXPERTS], s_S[OCCULT_MAX_EXPERTS];
  __shared__ float s_fd[OCCULT_MAX_VDEV], s_sd[OCCULT_MAX_VDEV];
  __shared__ int s_dev[OCCULT_MAX_EXPERTS];
  __shared__ float s_redf[32];
  __shared__ long long s_redl[32];
  __shared__ bool s_last;
  const int tid = threadIdx.x;
  for (int e = tid; e < a.Ne; e += kSumThreads) s_dev[e] = a.e2v[e];
  pdl_wait();
  pdl_trigger();
  const Work w = work_of(a.ws, tiles.n, a.Ne, a.G);
  // tokens, and groups that have any, over the whole batch
  long long N = 0, A = 0;
  for (int g = tid; g < a.G; g += kSumThreads) {
    long long n = 0;
    for (int i = 0; i < tiles.per_group; ++i)
      n += w.n[static_cast<int64_t>(g) * tiles.per_group + i];
    N += n;
    A += n > 0;
  }
  N = cta_sum(N, s_redl);
  A = cta_sum(A, s_redl);
  const float inv_a = 1.f / static_cast<float>(A > 0 ? A : 1);
  const float inv_n = 1.f / static_cast<float>(N > 0 ? N : 1);
  int cols = 32;  // a power of two of at least Ne threads a slice of the tiles
  while (cols < a.Ne) cols *= 2;
  const int col = tid % cols, slice = tid / cols, slices = kSumThreads / cols;
  for (int g = blockIdx.x; g < a.G; g += gridDim.x) {
    const int64_t tile0 = static_cast<int64_t>(g) * tiles.per_group;
    float s = 0.f;
    int c = 0;
    if (col < a.Ne) {
#pragma unroll 4
      for (int i = slice; i < tiles.per_group; i += slices) {
        s += w.p_sum[(tile0 + i) * a.Ne + col];
        c += w.count[(tile0 + i) * a.Ne + col];
      }
    }
    float sq = 0.f;
    long long n = 0;
    for (int i = tid; i < tiles.per_group; i += kSumThreads) {
      sq += w.sq[tile0 + i];
      n += w.n[tile0 + i];
    }
    s_part[tid] = s;
    s_cpart[tid] = c;
    n = cta_sum(n, s_redl);
    sq = cta_sum(sq, s_redf);
    const float inv_g = 1.f / static_cast<float>(n > 0 ? n : 1);
    if (tid < a.Ne) {
      for (int i = 1; i < slices; ++i) {
        s += s_part[i * cols + tid];
        c += s_cpart[i * cols + tid];
      }
      a.counts[static_cast<size_t>(g) * a.Ne + tid] = c;
      s_f[tid] = static_cast<float>(c) * (static_cast<float>(a.Ne) / static_cast<float>(a.k)) * inv_g;
      s_S[tid] = s * inv_g;
    }
    __syncthreads();
    // a warp a device
    for (int d = tid >> 5; d < a.Nd; d += kSumThreads / 32) {
      float f = 0.f, S = 0.f, m = 0.f;
      for (int e = tid & 31; e < a.Ne; e += 32)
        if (s_dev[e] == d) { f += s_f[e]; S += s_S[e]; m += 1.f; }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        f += __shfl_xor_sync(0xffffffffu, f, o);
        S += __shfl_xor_sync(0xffffffffu, S, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
      }
      if ((tid & 31) == 0) { s_fd[d] = m > 0.f ? f / m : 0.f; s_sd[d] = S; }
    }
    __syncthreads();
    if (tid < a.Ne) {
      const int d = s_dev[tid];
      const float fd = static_cast<unsigned>(d) < static_cast<unsigned>(a.Nd) ? s_fd[d] : 0.f;
      a.grad_w[static_cast<size_t>(g) * a.Ne + tid] =
          (a.coef * s_f[tid] + a.coef_dev * fd) * inv_g * inv_a;
    }
    const float expert = cta_sum(tid < a.Ne ? s_f[tid] * s_S[tid] : 0.f, s_redf);
    const float device = cta_sum(tid < a.Nd ? s_fd[tid] * s_sd[tid] : 0.f, s_redf);
    if (tid == 0) {
      w.terms[3 * static_cast<int64_t>(g)] = expert;
      w.terms[3 * static_cast<int64_t>(g) + 1] = device;
      w.terms[3 * static_cast<int64_t>(g) + 2] = sq;
    }
    __syncthreads();
  }
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
  for (int i = 0; i < 3; ++i) v[i] = cta_sum(v[i], s_redf);
  if (tid == 0) {
    const float expert = v[0] * inv_a, device = v[1] * inv_a, sq = v[2] * inv_n;
    a.loss[0] = a.coef * expert + a.coef_dev * device + a.coef_z * sq;
    a.loss[1] = expert;
    a.loss[2] = device;
    a.loss[3] = sq;
    a.grad_w[static_cast<size_t>(a.G) * a.Ne] = 2.f * a.coef_z * inv_n;
  }
}

// dz = dloss (p (w - w . p) + w_z lse p), LP lanes a token as in the first pass.
template <int LP>
__global__ void __launch_bounds__(kGradThreads) balance_grad_kernel(BalanceArgs a) {
  constexpr int kTok = 32 / LP;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, sub = lane % LP, e0 = sub * 8;
  const bool vec = a.Ne % 4 == 0;
  const float up = a.dloss ? *a.dloss : 1.f;
  const float wz = a.grad_w[static_cast<size_t>(a.G) * a.Ne];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kGradThreads / 32) * kTok;
  for (int64_t b = (static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5)) * kTok;
       b < a.T; b += step) {
    const int64_t t = b + lane / LP;
    const bool in = t < a.T, on = in && (!a.mask || a.mask[t]);
    const int64_t row = (in ? t : b) * a.Ne;
    float p[8], w[8];
    const float lse = softmax8<LP>(a.logits + row, a.Ne, vec, sub, p);
    const float* gw = a.grad_w + ((in ? t : b) / a.L) * a.Ne;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = e0 + i < a.Ne ? gw[e0 + i] : 0.f;
      dot += p[i] * w[i];
    }
#pragma unroll
    for (int o = LP / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float shift = wz * lse - dot;
    float* out = a.dlogits + row;
    if (!in || (!on && a.accumulate)) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = on ? up * (p[i] * (w[i] + shift)) : 0.f;
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (e0 + 4 * h >= a.Ne) continue;
        float4 v = make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
        float4* q = reinterpret_cast<float4*>(out + e0 + 4 * h);
        if (a.accumulate) {
          const float4 o = *q;
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        *q = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < a.Ne) out[e0 + i] = a.accumulate ? out[e0 + i] + p[i] : p[i];
    }
  }
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
  const Tiles t = tiles_of(ds.T, L, G);
  return (static_cast<size_t>(t.n) * (2 * ds.n_experts + 2) + 3 * static_cast<size_t>(G) + 1) *
         sizeof(float);
}

int launch_balance_loss(const LaunchCtx& ctx, const BalanceArgs& a) {
  const Tiles tiles = tiles_of(a.T, a.L, a.G);
  const dim3 grid(tiles.per_group, a.G < 65535 ? a.G : 65535);
  const int rc = cuda_status(
      a.Ne <= 64    ? launch_pdl(balance_tiles_kernel<8>, grid, kTileThreads, 0, ctx.stream, a, tiles)
      : a.Ne <= 128 ? launch_pdl(balance_tiles_kernel<16>, grid, kTileThreads, 0, ctx.stream, a, tiles)
                    : launch_pdl(balance_tiles_kernel<32>, grid, kTileThreads, 0, ctx.stream, a, tiles));
  if (rc) return rc;
  return cuda_status(launch_pdl(balance_groups_kernel, a.G < ctx.num_sms ? a.G : ctx.num_sms,
                                kSumThreads, 0, ctx.stream, a, tiles));
}

int launch_balance_grad(const LaunchCtx& ctx, const BalanceArgs& a) {
  if (a.T == 0) return OCCULT_OK;
  const int tok = (a.Ne <= 64 ? 4 : a.Ne <= 128 ? 2 : 1) * (kGradThreads / 32);
  const int64_t need = (static_cast<int64_t>(a.T) + tok - 1) / tok;
  const int grid = static_cast<int>(need < ctx.num_sms * 16 ? need : ctx.num_sms * 16);
  return cuda_status(
      a.Ne <= 64    ? launch_pdl(balance_grad_kernel<8>, grid, kGradThreads, 0, ctx.stream, a)
      : a.Ne <= 128 ? launch_pdl(balance_grad_kernel<16>, grid, kGradThreads, 0, ctx.stream, a)
                    : launch_pdl(balance_grad_kernel<32>, grid, kGradThreads, 0, ctx.stream, a));
}

}  // namespace occult
