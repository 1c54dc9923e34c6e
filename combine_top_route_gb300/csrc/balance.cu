// The router's balance loss: per-expert counts, expert, device and z terms over
// groups of tokens, and the gradient with respect to the logits.
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kBalWarps = 8;
constexpr int kBalThreads = kBalWarps * 32;
constexpr int kBalTile = 64;  // tokens of a CTA of the first pass

// Workspace: per tile Ne probability sums, {sum lse^2}, then Ne counts, {tokens}.
__host__ __device__ inline size_t tile_words(int Ne) { return 2 * static_cast<size_t>(Ne + 1); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// softmax of one token's row: lane l holds experts l, l+32, ...; returns log sum exp
template <int PL>
__device__ __forceinline__ float softmax_row(const float* row, int Ne, float (&p)[PL]) {
  const int lane = threadIdx.x & 31;
  const float NEG = -__int_as_float(0x7f800000);
  float mx = NEG;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    p[i] = lane + 32 * i < Ne ? row[lane + 32 * i] : NEG;
    mx = fmaxf(mx, p[i]);
  }
  mx = warp_max(mx);
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    p[i] = lane + 32 * i < Ne ? expf(p[i] - mx) : 0.f;
    z += p[i];
  }
  z = warp_sum(z);
#pragma unroll
  for (int i = 0; i < PL; ++i) p[i] = p[i] / z;
  return mx + logf(z);
}

// Pass 1, one CTA a tile of one group (grid.x tiles, grid.y groups).
template <int PL>
__global__ void __launch_bounds__(kBalThreads)
balance_tiles_kernel(BalanceArgs a) {
  __shared__ float s_p[kBalWarps][PL * 32];
  __shared__ int s_c[PL * 32];
  __shared__ float s_sq[kBalWarps];
  __shared__ int s_n[kBalWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < PL * 32; e += kBalThreads) s_c[e] = 0;
  __syncthreads();
  for (int g = blockIdx.y; g < a.G; g += gridDim.y) {
    const int64_t t0 = static_cast<int64_t>(g) * a.L + static_cast<int64_t>(blockIdx.x) * kBalTile;
    const int64_t end_g = min(static_cast<int64_t>(a.T), static_cast<int64_t>(g + 1) * a.L);
    const int64_t t1 = min(t0 + kBalTile, end_g);
    float acc[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) acc[i] = 0.f;
    float sq = 0.f;
    int n = 0;
    for (int64_t t = t0 + warp; t < t1; t += kBalWarps) {
      if (a.mask && !a.mask[t]) continue;
      float p[PL];
      const float lse = softmax_row<PL>(a.logits + t * a.Ne, a.Ne, p);
#pragma unroll
      for (int i = 0; i < PL; ++i) acc[i] += p[i];
      sq += lse * lse;
      ++n;
      if (lane < a.k) {
        const int e = a.ids[t * a.k + lane];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.Ne)) atomicAdd(&s_c[e], 1);
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) s_p[warp][lane + 32 * i] = acc[i];
    if (lane == 0) { s_sq[warp] = sq; s_n[warp] = n; }
    __syncthreads();
    float* out = a.ws + (static_cast<size_t>(g) * gridDim.x + blockIdx.x) * tile_words(a.Ne);
    int* outc = reinterpret_cast<int*>(out + a.Ne + 1);
    for (int e = threadIdx.x; e <= a.Ne; e += kBalThreads) {
      float s = 0.f;
      int c = 0;
      for (int w = 0; w < kBalWarps; ++w) {
        s += e < a.Ne ? s_p[w][e] : s_sq[w];
        if (e == a.Ne) c += s_n[w];
      }
      if (e < a.Ne) { c = s_c[e]; s_c[e] = 0; }
      out[e] = s;
      outc[e] = c;
    }
    __syncthreads();
  }
}

// Pass 2, one CTA a group: its sums, its part of the loss terms and the gradient's
// weights without the factor 1/A; the scalars over all groups go to pass 3.
__global__ void __launch_bounds__(kBalThreads) balance_groups_kernel(BalanceArgs a, int tiles) {
  __shared__ float s_f[OCCULT_MAX_EXPERTS], s_S[OCCULT_MAX_EXPERTS];
  __shared__ float s_fd[OCCULT_MAX_VDEV], s_sd[OCCULT_MAX_VDEV];
  __shared__ int s_n;
  pdl_wait();
  pdl_trigger();
  const size_t words = tile_words(a.Ne);
  for (int g = blockIdx.x; g < a.G; g += gridDim.x) {
    const float* base = a.ws + static_cast<size_t>(g) * tiles * words;
    float sq = 0.f;
    for (int e = threadIdx.x; e <= a.Ne; e += kBalThreads) {
      float s = 0.f;
      int c = 0;
      for (int i = 0; i < tiles; ++i) {
        s += base[i * words + e];
        c += reinterpret_cast<const int*>(base + i * words + a.Ne + 1)[e];
      }
      if (e < a.Ne) {
        a.counts[static_cast<size_t>(g) * a.Ne + e] = c;
        s_S[e] = s;
        s_f[e] = static_cast<float>(c);
      } else {
        s_n = c;
        sq = s;
        a.group_n[g] = c;
        a.group_terms[3 * g + 2] = sq;
      }
    }
    __syncthreads();
    const float N = static_cast<float>(max(s_n, 1));
    const float scale = static_cast<float>(a.Ne) / (static_cast<float>(a.k) * N);
    for (int e = threadIdx.x; e < a.Ne; e += kBalThreads) { s_f[e] *= scale; s_S[e] /= N; }
    __syncthreads();
    if (threadIdx.x < a.Nd) {
      float f = 0.f, S = 0.f;
      int n = 0;
      for (int e = 0; e < a.Ne; ++e)
        if (a.e2v[e] == static_cast<int>(threadIdx.x)) { f += s_f[e]; S += s_S[e]; ++n; }
      s_fd[threadIdx.x] = n ? f / n : 0.f;
      s_sd[threadIdx.x] = S;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.Ne; e += kBalThreads) {
      const int d = a.e2v[e];
      const float fd = static_cast<unsigned>(d) < static_cast<unsigned>(a.Nd) ? s_fd[d] : 0.f;
      a.grad_w[static_cast<size_t>(g) * a.Ne + e] = (a.coef * s_f[e] + a.coef_dev * fd) / N;
    }
    if (threadIdx.x == 0) {
      float b = 0.f, v = 0.f;
      for (int e = 0; e < a.Ne; ++e) b += s_f[e] * s_S[e];
      for (int d = 0; d < a.Nd; ++d) v += s_fd[d] * s_sd[d];
      a.group_terms[3 * g] = b;
      a.group_terms[3 * g + 1] = v;
    }
    __syncthreads();
  }
}

// Pass 3: the scalars, and the factor 1/A of the weights.
__global__ void __launch_bounds__(kBalThreads) balance_finish_kernel(BalanceArgs a) {
  __shared__ float s_inv;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    int A = 0;
    long long N = 0;
    float b = 0.f, v = 0.f, q = 0.f;
    for (int g = 0; g < a.G; ++g) {
      A += a.group_n[g] > 0;
      N += a.group_n[g];
      b += a.group_terms[3 * g];
      v += a.group_terms[3 * g + 1];
      q += a.group_terms[3 * g + 2];
    }
    const float inv = 1.f / static_cast<float>(max(A, 1));
    const float inv_n = 1.f / static_cast<float>(N > 0 ? N : 1);
    b *= inv; v *= inv; q *= inv_n;
    s_inv = inv;
    if (blockIdx.x == 0) {
      a.loss[0] = a.coef * b + a.coef_dev * v + a.coef_z * q;
      a.loss[1] = b;
      a.loss[2] = v;
      a.loss[3] = q;
      a.grad_w[static_cast<size_t>(a.G) * a.Ne] = 2.f * a.coef_z * inv_n;
    }
  }
  __syncthreads();
  const size_t n = static_cast<size_t>(a.G) * a.Ne;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kBalThreads + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * kBalThreads)
    a.grad_w[i] *= s_inv;
}

template <int PL>
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(BalanceArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const float up = a.dloss ? *a.dloss : 1.f;
  const float wz = a.grad_w[static_cast<size_t>(a.G) * a.Ne];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kBalWarps + (threadIdx.x >> 5); t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kBalWarps) {
    float* out = a.dlogits + t * a.Ne;
    if (a.mask && !a.mask[t]) {
      if (!a.accumulate)
        for (int e = lane; e < a.Ne; e += 32) out[e] = 0.f;
      continue;
    }
    float p[PL], w[PL];
    const float lse = softmax_row<PL>(a.logits + t * a.Ne, a.Ne, p);
    const float* gw = a.grad_w + (t / a.L) * a.Ne;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      w[i] = lane + 32 * i < a.Ne ? gw[lane + 32 * i] : 0.f;
      dot += p[i] * w[i];
    }
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.Ne) {
        const float dz = up * (p[i] * (w[i] - dot) + wz * lse * p[i]);
        out[e] = a.accumulate ? out[e] + dz : dz;
      }
    }
  }
}

}  // namespace

int balance_groups(int T, int group_len, int* L) {
  *L = group_len > 0 ? group_len : (T > 0 ? T : 1);
  const int G = static_cast<int>((static_cast<int64_t>(T) + *L - 1) / *L);
  return G > 0 ? G : 1;
}

static int balance_tiles(int T, int L) {
  const int len = T < L ? T : L;
  return len > 0 ? (len + kBalTile - 1) / kBalTile : 1;
}

size_t balance_ws_bytes(const occult_desc_t& ds, int group_len) {
  int L;
  const size_t G = balance_groups(ds.T, group_len, &L);
  return (G * balance_tiles(ds.T, L) * tile_words(ds.n_experts) + 4 * G) * sizeof(float);
}

#define OCCULT_BAL_BY_NE(call)              \
  (a.Ne <= 32 ? call(1) : a.Ne <= 64 ? call(2) : a.Ne <= 128 ? call(4) : call(8))

int launch_balance_loss(const LaunchCtx& ctx, BalanceArgs a) {
  const int tiles = balance_tiles(a.T, a.L);
  a.group_terms = a.ws + static_cast<size_t>(a.G) * tiles * tile_words(a.Ne);
  a.group_n = reinterpret_cast<int*>(a.group_terms + 3 * static_cast<size_t>(a.G));
  const dim3 grid(tiles, a.G < 65535 ? a.G : 65535);
#define OCCULT_BAL_TILES(PL) \
  launch_pdl(balance_tiles_kernel<PL>, grid, kBalThreads, 0, ctx.stream, a)
  int rc = cuda_status(OCCULT_BAL_BY_NE(OCCULT_BAL_TILES));
#undef OCCULT_BAL_TILES
  if (rc) return rc;
  rc = cuda_status(launch_pdl(balance_groups_kernel, a.G < 4096 ? a.G : 4096, kBalThreads, 0,
                              ctx.stream, a, tiles));
  if (rc) return rc;
  const int64_t n = static_cast<int64_t>(a.G) * a.Ne;
  const int64_t blocks = (n + kBalThreads - 1) / kBalThreads;
  return cuda_status(launch_pdl(balance_finish_kernel,
                                static_cast<int>(blocks < ctx.num_sms ? blocks : ctx.num_sms),
                                kBalThreads, 0, ctx.stream, a));
}

int launch_balance_grad(const LaunchCtx& ctx, const BalanceArgs& a) {
  if (a.T == 0) return OCCULT_OK;
  const int64_t need = (static_cast<int64_t>(a.T) + kBalWarps - 1) / kBalWarps;
  const int grid = static_cast<int>(need < ctx.num_sms * 16 ? need : ctx.num_sms * 16);
#define OCCULT_BAL_GRAD(PL) \
  launch_pdl(balance_grad_kernel<PL>, grid, kBalThreads, 0, ctx.stream, a)
  return cuda_status(OCCULT_BAL_BY_NE(OCCULT_BAL_GRAD));
#undef OCCULT_BAL_GRAD
}

}  // namespace occult
