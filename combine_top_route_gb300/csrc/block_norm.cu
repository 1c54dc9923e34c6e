// The norms around a block: RMS norm of its output, gate and residual sum, RMS
// norm before the next block (forward), and the gradients (backward).
//
// With one row's sums known everything is elementwise, so both directions are
// bound by the bytes they move: with bf16 rows and an fp32 block output the
// forward moves 10 bytes an element, the backward 16.  Sums, means and the column
// sums over the tokens are fp32; only what is stored is rounded to the tensors'
// types, x from the fp32 r'.
//
// Measured on one GB300 (norms on both sides, channel gates, bf16 stream; a copy
// reaches 6.76 TB/s): T=32768, d=2048 forward 101 us = 6.6 TB/s, backward 161 us =
// 6.7 TB/s; T=1 2.4 us, T=512 2.8 us (forward: a launch and a row's latency).
#include "common.cuh"
#include "kernels.h"

namespace occult {

namespace {

constexpr int kWideThreads = 1024;  // of the backward of rows too wide for a ring

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float4 mul4(const float4& a, const float4& b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 scale4(const float4& a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float4 fma4(const float4& a, float b, const float4& c) {
  return make_float4(fmaf(a.x, b, c.x), fmaf(a.y, b, c.y), fmaf(a.z, b, c.z), fmaf(a.w, b, c.w));
}

// The same as packed operations of two columns, which take half the issue slots (the
// backward 165 -> 161 us at T=32768, d=2048, 178 -> 160 us at 11000 x 5632; the forward,
// which waits for memory alone, gained nothing and keeps the plain ones).
__device__ __forceinline__ float2 lo2(const float4& a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ float2 hi2(const float4& a) { return make_float2(a.z, a.w); }
__device__ __forceinline__ float4 join(const float2& a, const float2& b) {
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float4 pmul4(const float4& a, const float4& b) {
  return join(__fmul2_rn(lo2(a), lo2(b)), __fmul2_rn(hi2(a), hi2(b)));
}
__device__ __forceinline__ float4 pscale4(const float4& a, float b) {
  return join(__fmul2_rn(lo2(a), two(b)), __fmul2_rn(hi2(a), two(b)));
}
__device__ __forceinline__ float4 pfma4(const float4& a, const float4& b, const float4& c) {
  return join(__ffma2_rn(lo2(a), lo2(b), lo2(c)), __ffma2_rn(hi2(a), hi2(b), hi2(c)));
}
__device__ __forceinline__ float4 pfma4(const float4& a, float b, const float4& c) {
  return pfma4(a, make_float4(b, b, b, b), c);
}
__device__ __forceinline__ float2 pdot(const float4& a, const float4& b, const float2& s) {
  return __ffma2_rn(hi2(a), hi2(b), __ffma2_rn(lo2(a), lo2(b), s));
}

// Sums of N values over the CTA, in a fixed order; every thread gets them.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*s_red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s_red[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < kWideThreads / 32; ++w) v[i] += s_red[w][i];
  }
}

// Backward of rows too wide for a ring (fp32 streams above 12800 columns) or not whole
// 16 bytes, one CTA a row, read twice (the second time from L2): 4096 x 16384 with a bf16
// stream took 398 us = 2.7 TB/s this way (325 us through the ring), bound by the latency
// of its two passes with one CTA an SM.  D is linear in mean(w_pre dx n), so
// one round of sums gives every mean: with g = w_pre dx, D0 = dr_out + rstd_pre g and
// q = gate w_post m,
//   s0 = sum g n,  s1 = sum q D0,  s2 = sum q n
//   c1 = s0 / d,   sum q D = s1 - c1 rstd_pre s2.
// The column sums stay with the threads that own the columns, in shared memory,
// and go to one row of partial sums a CTA.
template <typename R, typename L>
__global__ void __launch_bounds__(kWideThreads) norm_bwd_kernel(NormArgs a, float* part) {
  extern __shared__ float s_cols[];  // [2][d]: sum dx n, sum (gate) D m
  __shared__ float s_red[kWideThreads / 32][3];
  pdl_wait();
  pdl_trigger();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  const bool use_y = w_post || a.gate_kind != OCCULT_GATE_NONE;
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL, token = a.gate_kind == OCCULT_GATE_TOKEN;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  for (int c = threadIdx.x * 4; c < a.d; c += kWideThreads * 4) {
    st4(s_cols + c, zero);
    st4(s_cols + a.d + c, zero);
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = static_cast<size_t>(t) * a.d;
    const float rp = w_post ? a.rstd_post[t] : 1.f;
    const float rq = w_pre ? a.rstd_pre[t] : 0.f;
    const float tok = token ? a.gate[t] : 1.f;
    float s[3] = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x * 4; c < a.d; c += kWideThreads * 4) {
      const float4 up = a.dr_out ? ld4(static_cast<const R*>(a.dr_out) + base + c) : zero;
      float4 g = zero, n = zero, q = zero;
      if (w_pre) {
        g = mul4(ld4(a.dx + base + c), ld4(w_pre + c));
        n = scale4(ld4(static_cast<const R*>(a.r) + base + c), rq);
      }
      if (use_y) {
        q = scale4(ld4(a.y + base + c), rp);
        if (w_post) q = mul4(q, ld4(w_post + c));
        if (chan) q = mul4(q, ld4(a.gate + c));
      }
      s[0] += dot4(g, n);
      s[1] += dot4(q, fma4(g, rq, up));
      s[2] += dot4(q, n);
    }
    block_sum<3>(s, s_red);
    const float c1 = s[0] / a.d;
    const float qd = s[1] - c1 * rq * s[2];  // sum q D without the token's gate
    if (token && threadIdx.x == 0) a.dgate[t] = qd;
    const float c2 = tok * qd / a.d;         // mean(u m)
    for (int c = threadIdx.x * 4; c < a.d; c += kWideThreads * 4) {
      float4 D = a.dr_out ? ld4(static_cast<const R*>(a.dr_out) + base + c) : zero;
      if (w_pre) {
        const float4 dx = ld4(a.dx + base + c);
        const float4 n = scale4(ld4(static_cast<const R*>(a.r) + base + c), rq);
        D = fma4(fma4(n, -c1, mul4(dx, ld4(w_pre + c))), rq, D);
        st4(s_cols + c, add4(ld4(s_cols + c), mul4(dx, n)));
      }
      st4(static_cast<R*>(a.dr) + base + c, scale4(D, a.y ? a.res_scale : 1.f));
      if (!a.y) continue;
      float4 u = scale4(D, tok);
      float4 m = zero;
      if (use_y) {
        m = scale4(ld4(a.y + base + c), rp);
        st4(s_cols + a.d + c, add4(ld4(s_cols + a.d + c), mul4(chan ? D : u, m)));
      }
      u = mul4(u, chan ? ld4(a.gate + c) : one);
      if (w_post) u = scale4(fma4(m, -c2, mul4(u, ld4(w_post + c))), rp);
      st4(static_cast<L*>(a.dy) + base + c, u);
    }
  }
  __syncthreads();  // the copy below goes over both sums in one stride
  float* row = part + static_cast<size_t>(blockIdx.x) * 2 * a.d;
  for (int c = threadIdx.x * 4; c < 2 * a.d; c += kWideThreads * 4) st4(row + c, ld4(s_cols + c));
}

// ---- rows held by groups of warps ------------------------------------------------
// A group of G warps takes a row at a time; a thread owns the U units of four
// columns 4 (u 32 G + j), j its place in the group, of every row it sees.  The
// groups of a CTA (8 / G, at least one) work apart from each other.
template <int G>
struct Group {
  static constexpr int kGroups = G > 8 ? 1 : 8 / G;
  static constexpr int kThreads = 32 * G * kGroups;
  __device__ static int index() { return threadIdx.x / (32 * G); }
  __device__ static int place() { return threadIdx.x % (32 * G); }
  __device__ static void sync() {
    if (G == 1) __syncwarp();
    else if (kGroups == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" :: "r"(index() + 1), "n"(32 * G) : "memory");
  }
};

// Sums of three values (or, not `all`, of the first) over a group in a fixed order;
// every thread gets them.  The caller alternates between two s_red buffers, so that
// one sync a sum is enough.
template <int G>
__device__ __forceinline__ float4 group_sum(float4 v, bool all, float4* s_red) {
  if (all) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    }
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
  }
  if (G == 1) return v;
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  Group<G>::sync();
  const float4* mine = s_red + Group<G>::index() * G;
  v = mine[0];
#pragma unroll
  for (int w = 1; w < G; ++w) v = add4(v, mine[w]);
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum1(float v, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 1) return v;
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  Group<G>::sync();
  const float* mine = s_red + Group<G>::index() * G;
  v = mine[0];
#pragma unroll
  for (int w = 1; w < G; ++w) v += mine[w];
  return v;
}

// Forward of few rows (or of rows the ring does not take): the row stays in registers
// from its loads to its stores.  2.4 us a call for one token of d=2048, 3.4 us for 607;
// bound by the launch and three dependent steps (loads, two sums).  4096 x 16384: 123 us
// = 5.5 TB/s.
template <typename R, typename L, int G, int U>
__global__ void __launch_bounds__(Group<G>::kThreads) norm_fwd_rows_kernel(NormArgs a) {
  __shared__ float s_red[2][Group<G>::kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  const int place = Group<G>::place();
  int flip = 0;
  const float inv_d = 1.f / a.d;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t t = blockIdx.x * Group<G>::kGroups + Group<G>::index(); t < a.T;
       t += gridDim.x * Group<G>::kGroups) {
    const size_t base = static_cast<size_t>(t) * a.d;
    const R* r_in = static_cast<const R*>(a.r) + base;
    float4 r[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      y[u] = a.y && c < a.d ? ld4(a.y + base + c) : zero;
      r[u] = c < a.d ? ld4(r_in + c) : zero;
    }
    if (a.y) {
      float scale = a.gate_kind == OCCULT_GATE_TOKEN ? a.gate[t] : 1.f;
      if (w_post) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) s += dot4(y[u], y[u]);
        const float rp = rsqrtf(group_sum1<G>(s, s_red[flip]) * inv_d + a.eps);
        flip ^= 1;
        if (place == 0 && a.rstd_post_out) a.rstd_post_out[t] = rp;
        scale *= rp;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = 4 * (u * 32 * G + place);
        if (c >= a.d) continue;
        float4 b = scale4(y[u], scale);
        if (w_post) b = mul4(b, ld4(w_post + c));
        if (a.gate_kind == OCCULT_GATE_CHANNEL) b = mul4(b, ld4(a.gate + c));
        r[u] = fma4(r[u], a.res_scale, b);
        st4(static_cast<R*>(a.r_out) + base + c, r[u]);
      }
    }
    if (!w_pre) continue;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) s += dot4(r[u], r[u]);
    const float rq = rsqrtf(group_sum1<G>(s, s_red[flip]) * inv_d + a.eps);
    flip ^= 1;
    if (place == 0 && a.rstd_pre_out) a.rstd_pre_out[t] = rq;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c < a.d)
        st4(static_cast<L*>(a.x) + base + c, mul4(scale4(r[u], rq), ld4(w_pre + c)));
    }
  }
}

// Contiguous bytes (a multiple of 16) from global to shared memory, complete_tx on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

constexpr int kMaxStages = 3;  // rows of a ring

// One scalar for every row of a group: each warp holds those of 32 rows in its lanes and
// has the next 32 on their way (a load at each row would cost its latency there).
struct RowScalars {
  const float* p;
  int64_t first, step;
  int T;
  float now, next;
  __device__ RowScalars(const float* p, float none, int first, int step, int T)
      : p(p), first(first), step(step), T(T), now(none), next(none) {
    if (p) { load(now, 0); load(next, 32); }
  }
  __device__ void load(float& v, int k) {
    const int64_t t = first + (k + static_cast<int>(threadIdx.x & 31)) * step;
    if (t < T) v = p[t];
  }
  // the scalar of the group's k-th row; k = 0, 1, 2, ... in order
  __device__ float at(int k) {
    if (!p) return now;
    if ((k & 31) == 0 && k > 0) {
      now = next;
      load(next, k + 32);
    }
    return __shfl_sync(0xffffffffu, now, k & 31);
  }
};

// Bytes of one row in the forward's ring: y, then r.
template <typename R>
__host__ __device__ __forceinline__ int fwd_row_bytes(int d) {
  return (d * static_cast<int>(sizeof(float) + sizeof(R)) + 127) & ~127;
}

// Forward of many rows: a group's rows come through a ring of shared memory that bulk
// copies fill ahead of the arithmetic, so that the rows on their way take no registers
// and the two syncs of a row cost no bandwidth.  T=32768, d=2048: 101 us = 6.6 TB/s (rows
// in registers, a warp a row: 129 us; a CTA a row, read twice: 198 us).  Eight warps a
// row of 2048 with two units a thread beat four with four (113 us) and two with eight
// (130 us).
template <typename R, typename L, int G, int U, int CTAS>
__global__ void __launch_bounds__(Group<G>::kThreads, CTAS)
norm_fwd_ring_kernel(NormArgs a, int stages, int* dev_err) {
  extern __shared__ __align__(128) unsigned char s_ring[];
  __shared__ uint64_t s_full[Group<G>::kGroups][kMaxStages];
  __shared__ float s_red[2][Group<G>::kThreads / 32];
  __shared__ int s_abort;
  const int group = Group<G>::index(), place = Group<G>::place();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL;
  const int d = a.d, row_bytes = fwd_row_bytes<R>(d);
  unsigned char* ring = s_ring + static_cast<size_t>(group) * stages * row_bytes;
  if (place < stages) mbar_init(&s_full[group][place], 1);
  if (threadIdx.x == 0) s_abort = 0;
  mbar_fence_init();
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const uint32_t tx = d * (a.y ? 4 + sizeof(R) : sizeof(R));
  auto fill = [&](int stage, int t) {  // by the group's first thread
    unsigned char* p = ring + stage * row_bytes;
    uint64_t* bar = &s_full[group][stage];
    const size_t base = static_cast<size_t>(t) * d;
    mbar_arrive_expect_tx(bar, tx);
    if (a.y) bulk_load(p, a.y + base, d * 4, bar);
    bulk_load(p + d * 4, static_cast<const R*>(a.r) + base, d * sizeof(R), bar);
  };
  const int step = gridDim.x * Group<G>::kGroups;
  const int first = blockIdx.x * Group<G>::kGroups + group;
  if (place == 0)
    for (int i = 0; i < stages; ++i)
      if (static_cast<int64_t>(first) + static_cast<int64_t>(i) * step < a.T)
        fill(i, first + i * step);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 wq[U], wp[U];  // w_post times a channel gate; w_pre
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = 4 * (u * 32 * G + place);
    wp[u] = w_pre && c < d ? ld4(w_pre + c) : zero;
    wq[u] = make_float4(1.f, 1.f, 1.f, 1.f);
    if (c < d) {
      if (w_post) wq[u] = ld4(w_post + c);
      if (chan) wq[u] = mul4(wq[u], ld4(a.gate + c));
    }
  }
  const float inv_d = 1.f / d;
  int stage = 0, flip = 0;
  uint32_t parity = 0;
  RowScalars gate(a.gate_kind == OCCULT_GATE_TOKEN ? a.gate : nullptr, 1.f, first, step, a.T);
  int k = 0;
  for (int64_t t = first; t < a.T; t += step, ++k) {
    float scale = gate.at(k);
    if (!mbar_wait(&s_full[group][stage], parity, &s_abort)) {
      // gave up: the error is latched, the remaining rows run through without copies
      latch_error(dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
      s_abort = 1;
    }
    const float* s_y = reinterpret_cast<const float*>(ring + stage * row_bytes);
    const R* s_r = reinterpret_cast<const R*>(s_y + d);
    float4 r[U], y[U];
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      y[u] = a.y && c < d ? ld4(s_y + c) : zero;
      r[u] = c < d ? ld4(s_r + c) : zero;
      s += dot4(y[u], y[u]);
    }
    // this sync also says that the group has read the row: its place is refilled
    s = group_sum1<G>(s, s_red[flip]);
    flip ^= 1;
    if (G == 1) __syncwarp();
    if (place == 0 && !*const_cast<volatile int*>(&s_abort) &&
        t + static_cast<int64_t>(stages) * step < a.T)
      fill(stage, static_cast<int>(t + static_cast<int64_t>(stages) * step));
    if (++stage == stages) { stage = 0; parity ^= 1; }
    const size_t base = static_cast<size_t>(t) * d;
    if (a.y) {
      if (w_post) {
        const float rp = rsqrtf(s * inv_d + a.eps);
        if (place == 0 && a.rstd_post_out) a.rstd_post_out[t] = rp;
        scale *= rp;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = 4 * (u * 32 * G + place);
        r[u] = fma4(r[u], a.res_scale, mul4(scale4(y[u], scale), wq[u]));
        if (c < d) st4(static_cast<R*>(a.r_out) + base + c, r[u]);
      }
    }
    if (!w_pre) continue;
    s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) s += dot4(r[u], r[u]);
    const float rq = rsqrtf(group_sum1<G>(s, s_red[flip]) * inv_d + a.eps);
    flip ^= 1;
    if (place == 0 && a.rstd_pre_out) a.rstd_pre_out[t] = rq;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c < d) st4(static_cast<L*>(a.x) + base + c, mul4(scale4(r[u], rq), wp[u]));
    }
  }
  if (s_abort && place == 0) {  // copies may still be in flight: give them the limit again
    volatile int none = 0;
    for (int i = 0; i < stages; ++i)
      mbar_wait(&s_full[group][i], i < stage ? parity ^ 1 : parity, &none);
  }
}

// Column `col` of the two sums over all tokens, [dx n | D m], to what they are: dw_pre,
// dw_post and a channel gate's gradient.
template <typename L>
__device__ __forceinline__ void write_column(const NormArgs& a, int col, float s) {
  if (col < a.d) {
    if (a.dw_pre) a.dw_pre[col] = s;
    return;
  }
  const int j = col - a.d;
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL;
  if (a.dw_post) a.dw_post[j] = chan ? s * a.gate[j] : s;
  if (chan) a.dgate[j] = a.w_post ? s * to_f32(static_cast<const L*>(a.w_post)[j]) : s;
}
// A float of another CTA's shared memory, at the offset of `p` in this CTA's.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(smem_addr_in_rank(p, rank)));
  return v;
}

// Bytes of one row in the backward's ring: dx, y, then dr_out and r'.
template <typename R>
__host__ __device__ __forceinline__ int bwd_row_bytes(int d) {
  return (2 * d * static_cast<int>(sizeof(float)) + 2 * d * static_cast<int>(sizeof(R)) + 127) &
         ~127;
}

// Backward.  The rows of a group come through a ring of `stages` rows in shared
// memory, filled by bulk copies that run ahead of the arithmetic.  Up to two units a
// thread stay in registers from their sums to their stores, more are read from shared
// memory a second time.  The one sync of a row's sums also says which rows all of the
// group are done with, so that their places can be refilled.  The column sums stay in
// the registers of the threads that own the columns, over all the rows of the group.
// T=32768, d=2048: 161 us = 6.7 TB/s, a row at a time 312 us; 131 us without a norm after
// the block (12 bytes an element, 90 % of a copy: the sync and the sums of a row).  Two
// units a thread read twice instead of kept: 192 us; four units kept: registers spill,
// 267 against 160 us at d=5632.
template <typename R, typename L, int G, int U, int CTAS>
__global__ void __launch_bounds__(Group<G>::kThreads, CTAS)
norm_bwd_rows_kernel(NormArgs a, bool sums, float* part, int stages, int* dev_err) {
  extern __shared__ __align__(128) unsigned char s_ring[];
  __shared__ uint64_t s_full[Group<G>::kGroups][kMaxStages];
  __shared__ float4 s_red[2][Group<G>::kThreads / 32];
  __shared__ int s_abort;
  constexpr bool kKeep = U <= 2;
  constexpr int KEEP = kKeep ? U : 1;
  const int group = Group<G>::index(), place = Group<G>::place();
  const L* w_post = static_cast<const L*>(a.w_post);
  const L* w_pre = static_cast<const L*>(a.w_pre);
  const bool chan = a.gate_kind == OCCULT_GATE_CHANNEL, token = a.gate_kind == OCCULT_GATE_TOKEN;
  const bool use_y = w_post || a.gate_kind != OCCULT_GATE_NONE;
  const int d = a.d, row_bytes = bwd_row_bytes<R>(d);
  unsigned char* ring = s_ring + static_cast<size_t>(group) * stages * row_bytes;
  if (place < stages) mbar_init(&s_full[group][place], 1);
  if (threadIdx.x == 0) s_abort = 0;
  mbar_fence_init();
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const uint32_t tx = (w_pre ? d * (4 + sizeof(R)) : 0) + (use_y ? d * 4 : 0) +
                      (a.dr_out ? d * sizeof(R) : 0);
  auto fill = [&](int stage, int t) {  // by the group's first thread
    unsigned char* p = ring + stage * row_bytes;
    uint64_t* bar = &s_full[group][stage];
    const size_t base = static_cast<size_t>(t) * d;
    mbar_arrive_expect_tx(bar, tx);
    if (w_pre) {
      bulk_load(p, a.dx + base, d * 4, bar);
      bulk_load(p + d * (8 + sizeof(R)), static_cast<const R*>(a.r) + base, d * sizeof(R), bar);
    }
    if (use_y) bulk_load(p + d * 4, a.y + base, d * 4, bar);
    if (a.dr_out)
      bulk_load(p + d * 8, static_cast<const R*>(a.dr_out) + base, d * sizeof(R), bar);
  };
  const int step = gridDim.x * Group<G>::kGroups;
  const int first = blockIdx.x * Group<G>::kGroups + group;
  if (place == 0)
    for (int i = 0; i < stages; ++i)
      if (static_cast<int64_t>(first) + static_cast<int64_t>(i) * step < a.T)
        fill(i, first + i * step);

  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // w_pre, and w_post times a channel gate: held, or (32 warps have no registers for
  // them) read where they are used
  constexpr bool kHold = G <= 16;
  auto load_wp = [&](int c) { return w_pre && c < d ? ld4(w_pre + c) : zero; };
  auto load_wq = [&](int c) {
    float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
    if (c < d) {
      if (w_post) w = ld4(w_post + c);
      if (chan) w = mul4(w, ld4(a.gate + c));
    }
    return w;
  };
  float4 held_p[kHold ? U : 1], held_q[kHold ? U : 1];
  float4 sum_pre[U], sum_post[U];      // sum dx n; sum D m (of a token gate: gate D m)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = 4 * (u * 32 * G + place);
    if (kHold) { held_p[u] = load_wp(c); held_q[u] = load_wq(c); }
    sum_pre[u] = sum_post[u] = zero;
  }
  const float inv_d = 1.f / d;
  const float out_scale = a.y ? a.res_scale : 1.f;
  int stage = 0, flip = 0;
  uint32_t parity = 0;
  RowScalars post(w_post ? a.rstd_post : nullptr, 1.f, first, step, a.T);
  RowScalars pre(w_pre ? a.rstd_pre : nullptr, 0.f, first, step, a.T);
  RowScalars gate(token ? a.gate : nullptr, 1.f, first, step, a.T);
  int k = 0;
  for (int64_t t = first; t < a.T; t += step, ++k) {
    const float rp = post.at(k), rq = pre.at(k), tok = gate.at(k);
    if (!mbar_wait(&s_full[group][stage], parity, &s_abort)) {
      // gave up: the error is latched, the remaining rows run through without copies
      latch_error(dev_err, OCCULT_ERR_DEVICE_TIMEOUT);
      s_abort = 1;
    }
    const unsigned char* p = ring + stage * row_bytes;
    const float* s_dx = reinterpret_cast<const float*>(p);
    const float* s_y = s_dx + d;
    const R* s_up = reinterpret_cast<const R*>(s_y + d);
    const R* s_r = s_up + d;
    // with D0 = dr_out + rstd_pre w_pre dx:  sum w_pre dx n,  sum wq m D0,  sum wq m n
    // (rows read twice: of r' and y, the factors follow).  A factor of a row meets the
    // row's values or their sums before it meets itself: products of factors alone leave
    // fp32's range (rows of 1e13, zero rows at a small eps) where n, m and means do not.
    float2 sx = two(0.f), sy = two(0.f), sz = two(0.f);
    float4 k_dx[KEEP], k_n[KEEP], k_m[KEEP], k_D[KEEP];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c >= d) continue;
      float4 dx = zero, r = zero, y = zero, D = a.dr_out ? ld4(s_up + c) : zero;
      if (w_pre) {
        dx = ld4(s_dx + c);
        r = ld4(s_r + c);
        if (kKeep) r = pscale4(r, rq);  // n
        const float4 g = pmul4(dx, kHold ? held_p[kHold ? u : 0] : load_wp(c));
        D = pfma4(g, rq, D);
        sx = pdot(g, r, sx);
      }
      if (use_y) {
        y = ld4(s_y + c);
        if (kKeep) y = pscale4(y, rp);  // m
        const float4 q = pmul4(y, kHold ? held_q[kHold ? u : 0] : load_wq(c));
        sy = pdot(q, D, sy);
        sz = pdot(q, r, sz);
      }
      if (kKeep) { k_dx[u % KEEP] = dx; k_n[u % KEEP] = r; k_m[u % KEEP] = y; k_D[u % KEEP] = D; }
    }
    float4 sum = make_float4(sx.x + sx.y, sy.x + sy.y, sz.x + sz.y, 0.f);
    sum = group_sum<G>(sum, use_y, s_red[flip]);
    flip ^= 1;
    if (G == 1) __syncwarp();
    // past that sync all of the group are done with this row, where it is kept in
    // registers, and with the one before in any case: its place is refilled
    const bool filler = place == 0 && !*const_cast<volatile int*>(&s_abort);
    if (kKeep) {
      if (filler && t + static_cast<int64_t>(stages) * step < a.T)
        fill(stage, static_cast<int>(t + static_cast<int64_t>(stages) * step));
    } else if (filler && stages > 1 && t != first &&
               t + static_cast<int64_t>(stages - 1) * step < a.T) {
      fill(stage == 0 ? stages - 1 : stage - 1,
           static_cast<int>(t + static_cast<int64_t>(stages - 1) * step));
    }
    // mean(w_pre dx n); sum wq m D and its mean
    const float fr = kKeep ? 1.f : rq, fy = kKeep ? 1.f : rp;
    const float k1 = -rq * (fr * sum.x * inv_d);
    const float qd = fy * fmaf(k1, fr * sum.z, sum.y);
    if (token && place == 0) a.dgate[t] = qd;
    const float k2 = -rp * (qd * inv_d);
    const float ru = rp * tok;
    const size_t base = static_cast<size_t>(t) * d;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c >= d) continue;
      float4 D = kKeep ? k_D[u % KEEP] : a.dr_out ? ld4(s_up + c) : zero;
      if (w_pre) {
        const float4 dx = kKeep ? k_dx[u % KEEP] : ld4(s_dx + c);
        if (!kKeep) D = pfma4(pmul4(dx, kHold ? held_p[kHold ? u : 0] : load_wp(c)), rq, D);
        const float4 n = kKeep ? k_n[u % KEEP] : pscale4(ld4(s_r + c), rq);
        D = pfma4(n, k1, D);
        sum_pre[u] = pfma4(dx, n, sum_pre[u]);
      }
      st4(static_cast<R*>(a.dr) + base + c, pscale4(D, out_scale));
      if (!a.y) continue;
      float4 o = pscale4(pmul4(D, kHold ? held_q[kHold ? u : 0] : load_wq(c)), ru);
      if (use_y) {
        float4 m = kKeep ? k_m[u % KEEP] : pscale4(ld4(s_y + c), ru);  // times the gate
        if (kKeep && token) m = pscale4(m, tok);
        sum_post[u] = pfma4(D, m, sum_post[u]);
        if (w_post) o = pfma4(m, k2, o);
      }
      st4(static_cast<L*>(a.dy) + base + c, o);
    }
    if (!kKeep && stages == 1) {  // one place: it is refilled when all are done with this row
      Group<G>::sync();
      if (filler && t + static_cast<int64_t>(step) < a.T) fill(0, static_cast<int>(t + step));
    }
    if (++stage == stages) { stage = 0; parity ^= 1; }
  }
  if (s_abort && place == 0) {  // copies may still be in flight: give them the limit again
    volatile int none = 0;
    for (int i = 0; i < stages; ++i)
      mbar_wait(&s_full[group][i], i < stage ? parity ^ 1 : parity, &none);
  }
  if (!sums) return;
  // the groups' sums, then this CTA's: a row of partial sums, or, where the grid is one
  // cluster (part NULL), shared memory that every CTA reads its share of the columns from
  float* s_sum = reinterpret_cast<float*>(s_ring);
  float* row = part ? part + static_cast<size_t>(blockIdx.x) * 2 * d : s_sum;
  if (Group<G>::kGroups > 1 || !part) {
    __syncthreads();  // every group is done with the ring
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c >= d) continue;
      st4(s_sum + (2 * group) * d + c, sum_pre[u]);
      st4(s_sum + (2 * group + 1) * d + c, sum_post[u]);
    }
    __syncthreads();
    if (Group<G>::kGroups > 1) {
      for (int c = threadIdx.x * 4; c < 2 * d; c += Group<G>::kThreads * 4) {
        float4 v = ld4(s_sum + c);
        for (int g = 1; g < Group<G>::kGroups; ++g) v = add4(v, ld4(s_sum + 2 * g * d + c));
        st4(row + c, v);
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = 4 * (u * 32 * G + place);
      if (c >= d) continue;
      st4(row + c, sum_pre[u]);
      st4(row + d + c, sum_post[u]);
    }
  }
  if (part) return;
  cluster_sync();
  for (int c = blockIdx.x * Group<G>::kThreads + threadIdx.x; c < 2 * d;
       c += gridDim.x * Group<G>::kThreads) {
    float v = 0.f;
#pragma unroll 8
    for (int r = 0; r < static_cast<int>(gridDim.x); ++r) v += ld_cluster(s_sum + c, r);
    write_column<L>(a, c, v);
  }
  cluster_sync();  // no CTA ends while its sums are read
}

// Adds the CTAs' partial rows and turns the second sum into dw_post and a channel
// gate's gradient: a CTA takes 32 columns, each of its warps every 32nd row, so that
// the loads of some 300 rows are all on their way at once.
constexpr int kColWarps = 32;
template <typename L>
__global__ void __launch_bounds__(kColWarps * 32)
norm_bwd_cols_kernel(NormArgs a, const float* __restrict__ part, int n_part) {
  __shared__ float s_sum[kColWarps][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * a.d) {
#pragma unroll 10
    for (int p = warp; p < n_part; p += kColWarps) s += part[static_cast<size_t>(p) * 2 * a.d + c];
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  // warp w adds column w of the 32
  s = s_sum[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane != 0 || col >= 2 * a.d) return;
  write_column<L>(a, col, s);
}

template <typename K>
int allow_smem(K kernel, size_t bytes) {
  if (bytes <= 40 * 1024) return OCCULT_OK;  // 48 KB less the static arrays
  return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(bytes)));
}

template <typename R, typename L, int G, int U>
int fwd_rows(const LaunchCtx& ctx, const NormArgs& a) {
  const int need = (a.T + Group<G>::kGroups - 1) / Group<G>::kGroups;
  const int cap = ctx.num_sms * 8;
  return cuda_status(launch_pdl(norm_fwd_rows_kernel<R, L, G, U>, need < cap ? need : cap,
                                Group<G>::kThreads, 0, ctx.stream, a));
}

// Rows of a ring of `bytes` each (all groups of a CTA): three, two with an fp32 stream.
// Reads that run further ahead of the stores slow both: T=30011, d=2048, norms on both
// sides, us with two, three, four rows: forward 102, 93, 92 (bf16 stream) and 130, 147,
// 149 (fp32); backward 155, 152, 153 and 199, 220, 222.
// So do three rows of the forward that are more than 100 KB an SM together (two and three:
// 104 and 114 us at 29127 x 2304, 105 and 116 at 8192 x 8192; at 11915 x 5632, 99 KB, 107
// and 101).
constexpr int kRingBytes = 200 * 1024;   // of shared memory an SM, over its CTAs
constexpr int kAheadBytes = 100 * 1024;  // of them for three rows of the forward
template <typename R>
inline int ring_stages(int bytes, int ctas) {
  const int fit = kRingBytes / ctas / bytes, n = sizeof(R) == 4 ? 2 : 3;
  return n < fit ? n : fit;
}

template <typename R, typename L, int G, int U, int CTAS>
int fwd_ring(const LaunchCtx& ctx, const NormArgs& a) {
  const int row = fwd_row_bytes<R>(a.d) * Group<G>::kGroups;
  int stages = ring_stages<R>(row, CTAS);
  if (stages > 2 && stages * row * CTAS > kAheadBytes) stages = 2;
  const size_t smem = static_cast<size_t>(stages) * row;
  const int rc = allow_smem(norm_fwd_ring_kernel<R, L, G, U, CTAS>, smem);
  if (rc) return rc;
  const int need = (a.T + Group<G>::kGroups - 1) / Group<G>::kGroups;
  const int cap = ctx.num_sms * CTAS;
  return cuda_status(launch_pdl(norm_fwd_ring_kernel<R, L, G, U, CTAS>, need < cap ? need : cap,
                                Group<G>::kThreads, smem, ctx.stream, a, stages, ctx.dev_err));
}

template <typename R, typename L>
int fwd(const LaunchCtx& ctx, const NormArgs& a) {
  const int d = a.d;
  // Many rows come through the ring (its copies move whole 16 bytes and it holds rows
  // of up to 8192 columns); few rows have as many warps each as give a thread two
  // loads of each tensor, and no ring to set up.  (608 rows of 2048 take 3.5 us either
  // way.)  Warps a row and CTAs an SM by width: two units a thread with most of the
  // threads at work, and groups enough to hide one row's latency behind the others'
  // copies, but no more than that (their streams take the memory's rows from each other).
  // The steps end at the widths that were measured; one between them runs on the next
  // step's warps, some of them idle (2880 on 16 warps, 30 % idle, 0.74 of its floor where
  // 2816 on 11 and 4096 on 16 reach 0.93 and 0.96; 3584, 12 % idle, 0.88).
  // With only powers of two warps a row, us before and now: 32768 x 320 27 and 20, x 768 50
  // and 42, x 1408 95 and 73, 31775 x 2112 174 and 105, 23831 x 2816 135 and 105; with an
  // fp32 stream x 768 and x 320 gain nothing, x 1408 109 and 101, x 2112 175 and 141, and
  // 16384 x 4096 takes 146 us with one CTA an SM, 163 with two.
  if (a.T >= 4 * ctx.num_sms && d * sizeof(R) % 16 == 0 && d <= 8192) {
    constexpr bool kF32 = sizeof(R) == 4;
    if (d <= 128) return fwd_ring<R, L, 1, 1, 4>(ctx, a);
    if (d <= 256) return fwd_ring<R, L, 1, 2, 4>(ctx, a);
    if (d <= 384 && !kF32) return fwd_ring<R, L, 1, 3, 3>(ctx, a);
    if (d <= 512) return fwd_ring<R, L, 2, 2, 3>(ctx, a);
    if (d <= 768) return fwd_ring<R, L, 3, 2, 3>(ctx, a);
    if (d <= 1024) return fwd_ring<R, L, 4, 2, 2>(ctx, a);
    if (d <= 1536) return fwd_ring<R, L, 6, 2, 3>(ctx, a);
    if (d <= 2048) return fwd_ring<R, L, 8, 2, 2>(ctx, a);
    if (d <= 2304) return fwd_ring<R, L, 9, 2, kF32 ? 2 : 3>(ctx, a);
    if (d <= 2816) return fwd_ring<R, L, kF32 ? 16 : 11, 2, 2>(ctx, a);
    if (d <= 4096) return fwd_ring<R, L, 16, 2, kF32 ? 1 : 2>(ctx, a);
    if (d <= 6144) return fwd_ring<R, L, 16, 3, 1>(ctx, a);
    return fwd_ring<R, L, 16, 4, 1>(ctx, a);
  }
  if (d <= 256) return fwd_rows<R, L, 1, 2>(ctx, a);
  if (d <= 512) return fwd_rows<R, L, 2, 2>(ctx, a);
  if (d <= 1024) return fwd_rows<R, L, 4, 2>(ctx, a);
  if (d <= 2048) return fwd_rows<R, L, 8, 2>(ctx, a);
  if (d <= 4096) return fwd_rows<R, L, 16, 2>(ctx, a);
  if (d <= 8192) return fwd_rows<R, L, 16, 4>(ctx, a);
  return fwd_rows<R, L, 16, 8>(ctx, a);
}

// Few rows in one launch: a cluster whose CTAs add their column sums up over shared
// memory, for one row a group, three of narrow ones.  On the GPU that is no faster than
// two launches (us: 128 x 64 4.0 and 4.5, 257 x 64 5.4 and 4.7, 16 x 2048 5.1 and 4.9; two
// rows a group of 2048 6.1 and 5.0), but the host has one launch (2 us) less, which is
// what bounds calls of this size.
constexpr int cluster_rows(int G) { return G == 1 ? 3 : 1; }

template <typename R, typename L, int G, int U, int CTAS>
int bwd_rows(const LaunchCtx& ctx, const NormArgs& a, bool sums, float* part, int* n_part) {
  void (*kernel)(NormArgs, bool, float*, int, int*) = norm_bwd_rows_kernel<R, L, G, U, CTAS>;
  const int row = bwd_row_bytes<R>(a.d) * Group<G>::kGroups;
  const int stages = ring_stages<R>(row, CTAS);
  size_t smem = static_cast<size_t>(stages) * row;
  const size_t all = 2 * static_cast<size_t>(a.d) * Group<G>::kGroups * sizeof(float);
  smem = smem > all ? smem : all;
  int rc = allow_smem(kernel, smem);
  if (rc) return rc;
  const int need = (a.T + Group<G>::kGroups - 1) / Group<G>::kGroups;
  *n_part = 0;
  if (sums && ctx.clusters && need <= kClusterCtas * cluster_rows(G)) {
    rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (rc) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = kClusterCtas;
    cfg.blockDim = Group<G>::kThreads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a, sums, static_cast<float*>(nullptr),
                                          stages, ctx.dev_err));
  }
  const int cap = ctx.num_sms * CTAS < kNormMaxParts ? ctx.num_sms * CTAS : kNormMaxParts;
  *n_part = need < cap ? need : cap;
  return cuda_status(launch_pdl(kernel, *n_part, Group<G>::kThreads, smem, ctx.stream, a, sums, part,
                                stages, ctx.dev_err));
}

template <typename R, typename L>
int bwd_any(const LaunchCtx& ctx, const NormArgs& a, float* part, int* grid) {
  const size_t smem = 2 * static_cast<size_t>(a.d) * sizeof(float);
  const int rc = allow_smem(norm_bwd_kernel<R, L>, smem);
  if (rc) return rc;
  *grid = a.T < ctx.num_sms ? a.T : ctx.num_sms;  // (a CTA's column sums fill most of an SM)
  return cuda_status(launch_pdl(norm_bwd_kernel<R, L>, *grid, kWideThreads, smem, ctx.stream, a,
                                part));
}

template <typename R, typename L>
int bwd(const LaunchCtx& ctx, const NormArgs& a, float* part) {
  const int d = a.d;
  const bool sums = a.dw_pre || a.dw_post || a.gate_kind == OCCULT_GATE_CHANNEL;
  constexpr bool kF32 = sizeof(R) == 4;
  int n_part = 0, rc;  // rows of partial sums that are left to add up
  // bulk copies move whole 16 bytes; the ring holds a row of up to 16384 columns (12800
  // with an fp32 stream).  Above 2048 columns three or four units a thread (16 warps of
  // two units, one CTA an SM: 210 against 175 us at 16384 x 4096); one, three or six warps
  // a row up to 384, 768, 1536 and 2304 columns, where the next power of two would leave a
  // quarter to a half of the threads without work (wider ones keep theirs, and 2880 and
  // 6144 columns of bf16 reach 0.82 and 0.69 of their floors).  Powers of two and so, us: 32768
  // x 320 45 -> 40, x 768 84 -> 71, x 1408 149 -> 130, 31775 x 2112 204 -> 179; with an fp32
  // stream 259 -> 225 at 2112, the others the same, but x 320, which keeps two warps.
  if (d * sizeof(R) % 16 != 0 || bwd_row_bytes<R>(d) > kRingBytes)
    rc = bwd_any<R, L>(ctx, a, part, &n_part);
  else if (d <= 128) rc = bwd_rows<R, L, 1, 1, 3>(ctx, a, sums, part, &n_part);
  else if (d <= 256) rc = bwd_rows<R, L, 1, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 384 && !kF32) rc = bwd_rows<R, L, 1, 3, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 512) rc = bwd_rows<R, L, 2, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 768) rc = bwd_rows<R, L, 3, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 1024) rc = bwd_rows<R, L, 4, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 1536) rc = bwd_rows<R, L, 6, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 2048) rc = bwd_rows<R, L, 8, 2, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 2304) rc = bwd_rows<R, L, 6, 3, kF32 ? 3 : 2>(ctx, a, sums, part, &n_part);
  else if (d <= 4096) rc = bwd_rows<R, L, 8, 4, 2>(ctx, a, sums, part, &n_part);
  else if (d <= 6144) rc = bwd_rows<R, L, 16, 3, 1>(ctx, a, sums, part, &n_part);
  else if (d <= 8192) rc = bwd_rows<R, L, 16, 4, 1>(ctx, a, sums, part, &n_part);
  else rc = bwd_rows<R, L, 32, 4, 1>(ctx, a, sums, part, &n_part);
  if (rc || !sums || n_part == 0) return rc;
  return cuda_status(launch_pdl(norm_bwd_cols_kernel<L>, (2 * d + 31) / 32, kColWarps * 32, 0,
                                ctx.stream, a, part, n_part));
}

}  // namespace

int norm_bwd_parts(int T) { return T < kNormMaxParts ? T : kNormMaxParts; }

size_t block_norm_bwd_ws_bytes(const occult_desc_t& ds) {
  return static_cast<size_t>(norm_bwd_parts(ds.T)) * 2 * ds.d * sizeof(float);
}

int launch_block_norm(const LaunchCtx& ctx, const NormArgs& a, int res_dtype, int dtype) {
  if (res_dtype == OCCULT_BF16)
    return dtype == OCCULT_BF16 ? fwd<__nv_bfloat16, __nv_bfloat16>(ctx, a)
                                : fwd<__nv_bfloat16, float>(ctx, a);
  return dtype == OCCULT_BF16 ? fwd<float, __nv_bfloat16>(ctx, a) : fwd<float, float>(ctx, a);
}

int launch_block_norm_bwd(const LaunchCtx& ctx, const NormArgs& a, int res_dtype, int dtype,
                          void* ws) {
  float* part = static_cast<float*>(ws);
  if (res_dtype == OCCULT_BF16)
    return dtype == OCCULT_BF16 ? bwd<__nv_bfloat16, __nv_bfloat16>(ctx, a, part)
                                : bwd<__nv_bfloat16, float>(ctx, a, part);
  return dtype == OCCULT_BF16 ? bwd<float, __nv_bfloat16>(ctx, a, part)
                              : bwd<float, float>(ctx, a, part);
}

}  // namespace occult
