// Group norm with an activation over channels-last features, and its backward pass.
//
// A thread owns V adjacent channels (16 bytes) and walks pixels, so a wave reads whole pixel rows whatever the group
// width is (a group's channels alone are a short strip of each row). Sums are therefore kept per channel and joined
// to groups afterwards.
//
// Where a workgroup's registers hold all pixels of an image over a set of whole groups, one launch reads each feature
// once (k_gn_small, k_gn_small_back: the small maps, whose time is launches). Otherwise:
//   k_gn_stats     per (image, chunk of pixels, channel): mean and sum of squared deviations
//   k_gn_finish    per (image, group): mean and rstd from the chunks' channel statistics
//   k_gn_apply     y = act((x - mean) rstd gamma + beta)
//   k_gn_sums      per (image, chunk, channel): sum dz and sum dz xh
//   k_gn_sums_join per (image, channel): the chunks added; per (image, group): the two means dx needs
//   k_gn_dx        dx, and (its first workgroups) dgamma and dbeta from the images' sums
// Every join adds in a fixed order, so results repeat bit for bit.
#include <type_traits>

#include "feature_common.hpp"

namespace gsr {
namespace {

constexpr int kThreads = 256;

struct GnShape {
  uint32_t images, pixels, channels, groups, cpg;  // cpg: channels per group
  uint32_t cols;                                   // threads across the channels of a workgroup's block
  uint32_t rows;                                   // threads across pixels (kThreads / cols)
  uint32_t chunk, chunks;                          // pixels per chunk
  float eps;
};

// Statistics as the caller keeps them, aligned as float.
struct GnStats {
  float mean, rstd;
};

// 1 / (1 + exp(-z)) with the hardware exponential and reciprocal, each within 1 ulp of its own result (an overflowing
// exponential gives 0).
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == GSR_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == GSR_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays
  return z;
}

// act'(z)
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == GSR_ACT_SILU) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  if constexpr (ACT == GSR_ACT_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);
  return 1.0f;
}

constexpr int kJoinThreads = 1024;  // one workgroup joins the chunks of an (image, group): most loads in flight

// Sum over the workgroup, in a fixed order; every thread gets it. `s` holds kJoinThreads / 64 floats.
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kJoinThreads / 64; ++k) sum += s[k];
  return sum;
}

// Adds two running values of every thread over the threads of its channel column (the rows), leaving the totals in
// row 0. s_a, s_b: [kThreads * V].
template <int V>
__device__ __forceinline__ void add_rows(const GnShape& g, uint32_t col, uint32_t row, bool live, float* a, float* b,
                                         float (*s)[V * 2]) {
  for (uint32_t half = 1u << (31 - __clz(max(1u, g.rows - 1) | 1)); half > 0; half >>= 1) {
    __syncthreads();
    if (live && row >= half && row < 2 * half) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[row * g.cols + col][i] = a[i];
        s[row * g.cols + col][V + i] = b[i];
      }
    }
    __syncthreads();
    if (live && row < half && row + half < g.rows) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] += s[(row + half) * g.cols + col][i];
        b[i] += s[(row + half) * g.cols + col][V + i];
      }
    }
  }
}

// a + b = sum + rest, exactly.
__device__ __forceinline__ void two_sum(float a, float b, float* sum, float* rest) {
  const float s = a + b, t = s - a;
  *rest = (a - (s - t)) + (b - t);
  *sum = s;
}

// Means and squared deviations per channel of one chunk of pixels. A thread takes four pixels at a time: M2 of the four
// about their own mean, then joined to what came before, M2 += M2_4 + (mean_4 - mean)^2 n 4 / (n + 4). No large square is
// cancelled anywhere, so neither a far mean nor an outlier, wherever it stands, costs more than the roundings of the
// sum of positive terms. The differences are taken from the thread's first value (exact for values near each other);
// the means come from the values' own sum, its roundings carried along.
// 2 x 800 x 800 x 64 bfloat16 (164 MB) 39 us, 4.2 TB/s, the vector units busy 62 % (36 us with sums of squares about the
// first value, which an outlier there spoils); 4 x 100 x 100 x 320 float32 (51 MB) 13.4 us. About
// 2,048 chunks over the images: eight workgroups a compute unit, and few enough partial sums that their join is short.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gn_stats(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                       float2* __restrict__ part) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float s[kThreads][V * 2];
  const uint32_t col = threadIdx.x % g.cols, row = threadIdx.x / g.cols;
  const uint32_t c0 = (blockIdx.z * g.cols + col) * V;
  const int n_c = int(g.channels) - int(c0);
  const bool live = row < g.rows && n_c > 0;
  const uint32_t p0 = blockIdx.x * g.chunk, p1 = min(g.pixels, p0 + g.chunk);
  const T* base = x + int64_t(blockIdx.y) * xi + c0;
  // shift: the first value; from_shift: sum of x - shift; sum + rest: sum of x
  float shift[V], from_shift[V], sum[V], rest[V], m2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) shift[i] = from_shift[i] = sum[i] = rest[i] = m2[i] = 0.0f;
  uint32_t n = 0;
  if (live && p0 + row < p1) {
    load_f32<V>(base + int64_t(p0 + row) * xp, n_c, shift);
    uint32_t p = p0 + row;
    for (; p + 3 * g.rows < p1; p += 4 * g.rows) {
      float f[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) load_f32<V>(base + int64_t(p + k * g.rows) * xp, n_c, f[k]);
      const float inv = n ? __builtin_amdgcn_rcpf(float(n)) : 0.0f;
      const float weight = float(4 * n) * __builtin_amdgcn_rcpf(float(n + 4));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float e[4], low;
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = f[k][i] - shift[i];
        const float four = (e[0] + e[1]) + (e[2] + e[3]), mean = 0.25f * four;
        const float d = fmaf(-from_shift[i], inv, mean);
        float q = d * d * weight;
#pragma unroll
        for (int k = 0; k < 4; ++k) q = fmaf(e[k] - mean, e[k] - mean, q);
        m2[i] += q;
        from_shift[i] += four;
        two_sum(sum[i], (f[0][i] + f[1][i]) + (f[2][i] + f[3][i]), &sum[i], &low);
        rest[i] += low;
      }
      n += 4;
    }
    for (; p < p1; p += g.rows) {
      float f[V];
      load_f32<V>(base + int64_t(p) * xp, n_c, f);
      const float inv = n ? __builtin_amdgcn_rcpf(float(n)) : 0.0f;
      const float weight = float(n) * __builtin_amdgcn_rcpf(float(n + 1));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float low;
        const float e = f[i] - shift[i], d = fmaf(-from_shift[i], inv, e);
        m2[i] = fmaf(d * weight, d, m2[i]);
        from_shift[i] += e;
        two_sum(sum[i], f[i], &sum[i], &low);
        rest[i] += low;
      }
      ++n;
    }
  }
  // (n, mean, M2) of the column: the mean first, then every thread's M2 about it
  float mean[V], part_mean[V], zero[V];
  const float share = float(n) / float(p1 - p0);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    part_mean[i] = (rest[i] - rest[i] == 0.0f ? sum[i] + rest[i] : sum[i]) / float(max(1u, n));  // infinite: no rest
    if (!(m2[i] - m2[i] == 0.0f)) m2[i] = m2[i] - m2[i];  // infinities and NaN carry on as NaN
    mean[i] = n ? part_mean[i] * share : 0.0f;
    zero[i] = 0.0f;
  }
  add_rows<V>(g, col, row, live, mean, zero, s);
  __syncthreads();
  if (live && row == 0)
#pragma unroll
    for (int i = 0; i < V; ++i) s[col][i] = mean[i];
  __syncthreads();
  if (live && n) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = part_mean[i] - s[col][i];
      m2[i] = fmaf(float(n) * d, d, m2[i]);
    }
  }
  add_rows<V>(g, col, row, live, m2, zero, s);
  if (live && row == 0) {
    float2* out = part + (int64_t(blockIdx.y) * g.chunks + blockIdx.x) * g.channels + c0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n_c) out[i] = make_float2(mean[i], m2[i]);
  }
}

// f(chunk, channel within the group, entry) over the chunks and channels of one (image, group), eight loads in flight.
// Threads take (channel, part of the chunks), so that a wave reads along channels.
template <typename F>
__device__ __forceinline__ void for_parts(const GnShape& g, uint32_t img, uint32_t grp,
                                          const float2* __restrict__ part, F f) {
  const uint32_t width = min(g.cpg, uint32_t(kJoinThreads)), lanes = kJoinThreads / width;
  const uint32_t tc = threadIdx.x % width, tk = threadIdx.x / width;
  if (tk >= lanes) return;
  for (uint32_t c = tc; c < g.cpg; c += width) {
    const float2* base = part + int64_t(img) * g.chunks * g.channels + grp * g.cpg + c;
    for (uint32_t k0 = tk; k0 < g.chunks; k0 += 8 * lanes) {
      float2 v[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
        if (k0 + i * lanes < g.chunks) v[i] = base[int64_t(k0 + i * lanes) * g.channels];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
        if (k0 + i * lanes < g.chunks) f(k0 + i * lanes, c, v[i]);
    }
  }
}

// Mean and rstd of one (image, group) from its chunks' channel statistics: the weighted mean of the means, then
// M2 = sum M2_i + n_i (mean_i - mean)^2.
// Bound by latency (one pass for the means, one for the deviations, over at most a megabyte): 6 us at either size above.
__global__ __launch_bounds__(kJoinThreads) void k_gn_finish(GnShape g, const float2* __restrict__ part,
                                                        GnStats* __restrict__ stats) {
  __shared__ float s[kJoinThreads / 64];
  const uint32_t grp = blockIdx.x, img = blockIdx.y;
  const float last = float(g.pixels - (g.chunks - 1) * g.chunk), full = float(g.chunk);
  const float total = float(g.pixels) * float(g.cpg);
  const float w_full = full / total, w_last = last / total;
  float m = 0.0f;
  for_parts(g, img, grp, part,
            [&](uint32_t k, uint32_t, float2 v) { m = fmaf(k + 1 == g.chunks ? w_last : w_full, v.x, m); });
  const float mean = block_sum(m, s);
  float q = 0.0f;
  for_parts(g, img, grp, part, [&](uint32_t k, uint32_t, float2 v) {
    const float d = v.x - mean;
    q += fmaf((k + 1 == g.chunks ? last : full) * d, d, v.y);
  });
  const float var = block_sum(q, s) / total;
  if (threadIdx.x == 0) stats[uint64_t(img) * g.groups + grp] = GnStats{mean, 1.0f / sqrtf(var + g.eps)};
}

// The channel constants a thread keeps for its V channels of one image.
template <int V>
struct Channel {
  float mean[V], rstd[V], gamma[V], beta[V];
  __device__ __forceinline__ void load(const GnShape& g, uint32_t img, uint32_t c0, int n_c, const GnStats* stats,
                                       const float* gm, const float* bt) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t c = i < n_c ? c0 + i : g.channels - 1;
      const GnStats st = stats[uint64_t(img) * g.groups + c / g.cpg];
      mean[i] = st.mean;
      rstd[i] = st.rstd;
      gamma[i] = gm ? gm[c] : 1.0f;
      beta[i] = bt ? bt[c] : 0.0f;
    }
  }
};

// The map read again, normalised and written: 2 x 800 x 800 x 64 bfloat16 64 us, 5.1 TB/s of read and write, the rate of
// a copy; 4 x 100 x 100 x 320 float32 18 us. Taking the images in the reverse of k_gn_stats's order, for what the last
// level of cache still holds, changed nothing (108 against 104 us a call).
template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_apply(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                       const float* __restrict__ gamma,
                                                       const float* __restrict__ beta,
                                                       const GnStats* __restrict__ stats, T* y, int64_t yi,
                                                       int64_t yp) {
  constexpr int V = 16 / sizeof(T);
  const uint32_t col = threadIdx.x % g.cols, row = threadIdx.x / g.cols;
  const uint32_t c0 = (blockIdx.z * g.cols + col) * V;
  const int n_c = int(g.channels) - int(c0);
  if (row >= g.rows || n_c <= 0) return;
  Channel<V> ch;
  ch.load(g, blockIdx.y, c0, n_c, stats, gamma, beta);
#pragma unroll
  for (int i = 0; i < V; ++i) ch.rstd[i] *= ch.gamma[i];
  const uint32_t p0 = blockIdx.x * g.chunk, p1 = min(g.pixels, p0 + g.chunk);
  const T* xb = x + int64_t(blockIdx.y) * xi + c0;
  T* yb = y + int64_t(blockIdx.y) * yi + c0;
  constexpr int kAtOnce = 4;  // loads in flight before the first store (y may be x, so the compiler keeps their order)
  uint32_t p = p0 + row;
  for (; p + (kAtOnce - 1) * g.rows < p1; p += kAtOnce * g.rows) {
    float f[kAtOnce][V];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) load_f32<V>(xb + int64_t(p + k * g.rows) * xp, n_c, f[k]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[k][i] = act_value<ACT>(fmaf(f[k][i] - ch.mean[i], ch.rstd[i], ch.beta[i]));
      store_f32<V>(yb + int64_t(p + k * g.rows) * yp, n_c, f[k]);
    }
  }
  for (; p < p1; p += g.rows) {
    float f[V];
    load_f32<V>(xb + int64_t(p) * xp, n_c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = act_value<ACT>(fmaf(f[i] - ch.mean[i], ch.rstd[i], ch.beta[i]));
    store_f32<V>(yb + int64_t(p) * yp, n_c, f);
  }
}

// Bound by memory, x and dy read: 4 x 100 x 100 x 320 float32 (102 MB) 19.5 us, 5.3 TB/s.
template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_sums(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                      const float* __restrict__ gamma,
                                                      const float* __restrict__ beta,
                                                      const GnStats* __restrict__ stats, const T* __restrict__ dy,
                                                      int64_t di, int64_t dp, float2* __restrict__ part) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float s[kThreads][V * 2];
  const uint32_t col = threadIdx.x % g.cols, row = threadIdx.x / g.cols;
  const uint32_t c0 = (blockIdx.z * g.cols + col) * V;
  const int n_c = int(g.channels) - int(c0);
  const bool live = row < g.rows && n_c > 0;
  const uint32_t p0 = blockIdx.x * g.chunk, p1 = min(g.pixels, p0 + g.chunk);
  float a[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
  if (live) {
    Channel<V> ch;
    ch.load(g, blockIdx.y, c0, n_c, stats, gamma, beta);
    const T* xb = x + int64_t(blockIdx.y) * xi + c0;
    const T* db = dy + int64_t(blockIdx.y) * di + c0;
#pragma unroll 2
    for (uint32_t p = p0 + row; p < p1; p += g.rows) {
      float f[V], d[V];
      load_f32<V>(xb + int64_t(p) * xp, n_c, f);
      load_f32<V>(db + int64_t(p) * dp, n_c, d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (f[i] - ch.mean[i]) * ch.rstd[i];
        const float dz = d[i] * act_slope<ACT>(fmaf(xh, ch.gamma[i], ch.beta[i]));
        a[i] += dz;
        b[i] = fmaf(dz, xh, b[i]);
      }
    }
  }
  add_rows<V>(g, col, row, live, a, b, s);
  if (live && row == 0) {
    float2* out = part + (int64_t(blockIdx.y) * g.chunks + blockIdx.x) * g.channels + c0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n_c) out[i] = make_float2(a[i], b[i]);
  }
}

// One workgroup per (image, group); latency, 6 us for 4 images of 32 groups and 480 chunks.
__global__ __launch_bounds__(kJoinThreads) void k_gn_sums_join(GnShape g, const float2* __restrict__ part,
                                                           const float* __restrict__ gamma,
                                                           float2* __restrict__ chan, float2* __restrict__ group) {
  __shared__ float sa[kJoinThreads], sb[kJoinThreads], s[kJoinThreads / 64];
  const uint32_t grp = blockIdx.x, img = blockIdx.y;
  const uint32_t width = min(g.cpg, uint32_t(kJoinThreads)), lanes = kJoinThreads / width;
  const uint32_t tc = threadIdx.x % width, tk = threadIdx.x / width;
  float ga = 0.0f, gb = 0.0f;
  for (uint32_t c0 = 0; c0 < g.cpg; c0 += width) {
    const bool live = c0 + tc < g.cpg;
    const uint32_t c = grp * g.cpg + c0 + tc;
    float a = 0.0f, b = 0.0f;
    if (tk < lanes && live) {
      const float2* base = part + int64_t(img) * g.chunks * g.channels + c;
      for (uint32_t k0 = tk; k0 < g.chunks; k0 += 8 * lanes) {
        float2 v[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
          v[i] = k0 + i * lanes < g.chunks ? base[int64_t(k0 + i * lanes) * g.channels] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
          a += v[i].x;
          b += v[i].y;
        }
      }
    }
    __syncthreads();
    sa[threadIdx.x] = a;
    sb[threadIdx.x] = b;
    __syncthreads();
    // the parts of a channel, halving (a fixed order)
    for (uint32_t half = lanes > 1 ? 1u << (31 - __clz(lanes - 1)) : 0; half > 0; half >>= 1) {
      if (tk < half && tk + half < lanes) {
        sa[threadIdx.x] += sa[threadIdx.x + half * width];
        sb[threadIdx.x] += sb[threadIdx.x + half * width];
      }
      __syncthreads();
    }
    if (tk == 0 && live) {
      a = sa[threadIdx.x];
      b = sb[threadIdx.x];
      chan[int64_t(img) * g.channels + c] = make_float2(a, b);
      const float gm = gamma ? gamma[c] : 1.0f;
      ga = fmaf(a, gm, ga);
      gb = fmaf(b, gm, gb);
    }
  }
  ga = block_sum(ga, s);
  gb = block_sum(gb, s);
  if (threadIdx.x == 0) {
    const float m = float(g.pixels) * float(g.cpg);
    group[uint64_t(img) * g.groups + grp] = make_float2(ga / m, gb / m);
  }
}

// Bound by memory, x and dy read and dx written: 4 x 100 x 100 x 320 float32 (154 MB) 25 us, 6.1 TB/s (part of x and dy is
// still in the last level of cache).
template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_dx(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                    const float* __restrict__ gamma, const float* __restrict__ beta,
                                                    const GnStats* __restrict__ stats, const T* dy, int64_t di,
                                                    int64_t dp, const float2* __restrict__ chan,
                                                    const float2* __restrict__ group, T* dx, int64_t oi, int64_t op,
                                                    float* __restrict__ dgamma, float* __restrict__ dbeta) {
  constexpr int V = 16 / sizeof(T);
  const uint32_t col = threadIdx.x % g.cols, row = threadIdx.x / g.cols;
  const uint32_t c0 = (blockIdx.z * g.cols + col) * V;
  const int n_c = int(g.channels) - int(c0);
  if (row >= g.rows || n_c <= 0) return;
  if (blockIdx.x == 0 && blockIdx.y == 0 && row == 0 && (dgamma || dbeta)) {
    for (int i = 0; i < V && i < n_c; ++i) {
      float a = 0.0f, b = 0.0f;
      for (uint32_t n = 0; n < g.images; ++n) {
        const float2 v = chan[int64_t(n) * g.channels + c0 + i];
        a += v.x;
        b += v.y;
      }
      if (dgamma) dgamma[c0 + i] = b;
      if (dbeta) dbeta[c0 + i] = a;
    }
  }
  if (!dx) return;
  Channel<V> ch;
  ch.load(g, blockIdx.y, c0, n_c, stats, gamma, beta);
  float m1[V], m2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t c = i < n_c ? c0 + i : g.channels - 1;
    const float2 v = group[uint64_t(blockIdx.y) * g.groups + c / g.cpg];
    m1[i] = v.x;
    m2[i] = v.y;
  }
  const uint32_t p0 = blockIdx.x * g.chunk, p1 = min(g.pixels, p0 + g.chunk);
  const T* xb = x + int64_t(blockIdx.y) * xi + c0;
  const T* db = dy + int64_t(blockIdx.y) * di + c0;
  T* ob = dx + int64_t(blockIdx.y) * oi + c0;
  auto gradient = [&](const float* f, float* d) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float xh = (f[i] - ch.mean[i]) * ch.rstd[i];
      const float dz = d[i] * act_slope<ACT>(fmaf(xh, ch.gamma[i], ch.beta[i]));
      d[i] = ch.rstd[i] * (fmaf(dz, ch.gamma[i], -m1[i]) - xh * m2[i]);
    }
  };
  uint32_t p = p0 + row;
  for (; p + g.rows < p1; p += 2 * g.rows) {  // two pixels' loads in flight before the first store
    float f[2][V], d[2][V];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      load_f32<V>(xb + int64_t(p + k * g.rows) * xp, n_c, f[k]);
      load_f32<V>(db + int64_t(p + k * g.rows) * dp, n_c, d[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      gradient(f[k], d[k]);
      store_f32<V>(ob + int64_t(p + k * g.rows) * op, n_c, d[k]);
    }
  }
  if (p < p1) {
    float f[V], d[V];
    load_f32<V>(xb + int64_t(p) * xp, n_c, f);
    load_f32<V>(db + int64_t(p) * dp, n_c, d);
    gradient(f, d);
    store_f32<V>(ob + int64_t(p) * op, n_c, d);
  }
}

// ---- one launch: all pixels of an image over a set of whole groups in a workgroup's registers

constexpr int kSmallThreads = 1024, kHoldForward = 8, kHoldBackward = 4;  // vectors of an input a thread holds

struct GnSet {
  uint32_t groups, channels;  // of a full set; the last may have fewer
  uint32_t cols, rows;        // threads across the set's channels and across pixels
};

// Totals over the workgroup's pixels of every channel (s_chan) from each thread's V values.
// s_part: [kSmallThreads][V], s_sub: [kSmallThreads].
template <int V>
__device__ __forceinline__ void channel_totals(const GnSet& t, bool live, const float* v, float (*s_part)[V],
                                               float* s_sub, float* s_chan) {
  const uint32_t wide = t.cols * V, subs = max(1u, min(8u, kSmallThreads / wide));
  __syncthreads();
  if (live) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_part[threadIdx.x][i] = v[i];
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < subs * wide; e += kSmallThreads) {
    const uint32_t ch = e % wide, sub = e / wide;
    float sum = 0.0f;
    for (uint32_t r = sub; r < t.rows; r += subs) sum += s_part[r * t.cols + ch / V][ch % V];
    if (subs > 1)
      s_sub[e] = sum;
    else
      s_chan[ch] = sum;
  }
  __syncthreads();
  if (subs > 1 && threadIdx.x < wide) {
    float sum = 0.0f;
    for (uint32_t k = 0; k < subs; ++k) sum += s_sub[k * wide + threadIdx.x];
    s_chan[threadIdx.x] = sum;
  }
  __syncthreads();
}

// Sums over each group's channels of s_chan (times gamma, if given): a wave per group.
__device__ __forceinline__ void group_totals(uint32_t groups, uint32_t cpg, const float* s_chan, const float* gamma,
                                             float* s_group) {
  const uint32_t lane = threadIdx.x & 63;
  for (uint32_t g = threadIdx.x >> 6; g < groups; g += kSmallThreads / 64) {
    float sum = 0.0f;
    for (uint32_t c = lane; c < cpg; c += 64) sum = fmaf(s_chan[g * cpg + c], gamma ? gamma[g * cpg + c] : 1.0f, sum);
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
    if (lane == 0) s_group[g] = sum;
  }
  __syncthreads();
}

// Shared memory of a set, at most kSmallThreads channels and as many groups.
template <int V>
struct SmallShared {
  float part[kSmallThreads][V];
  float sub[kSmallThreads], chan[2][kSmallThreads], group[2][kSmallThreads];
};

template <typename T, int V, int kHold>
struct Held {
  Vec<T, V> v[kHold];
  __device__ __forceinline__ void load(const T* base, int64_t stride, uint32_t row, uint32_t rows, uint32_t pixels,
                                       int n) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const uint32_t p = row + k * rows;
      if (p >= pixels) continue;
      if (n >= V) {
        __builtin_memcpy(&v[k], base + int64_t(p) * stride, sizeof v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = i < n ? base[int64_t(p) * stride + i] : T(0.0f);
      }
    }
  }
};

// The whole forward pass in one launch, the features read once into registers: bound by latency, 3 x 17 x 19 x 90 float16
// 9 us for 0.35 MB (its launches through k_gn_stats, k_gn_finish and k_gn_apply would be three of 2.5 to 6 us).
template <typename T, int ACT, int V>
__global__ __launch_bounds__(kSmallThreads) void k_gn_small(GnShape g, GnSet t, const T* x, int64_t xi, int64_t xp,
                                                            const float* __restrict__ gamma,
                                                            const float* __restrict__ beta,
                                                            GnStats* __restrict__ stats, T* y, int64_t yi,
                                                            int64_t yp) {
  constexpr int kHold = kHoldForward;
  __shared__ SmallShared<V> s;
  const uint32_t grp0 = blockIdx.x * t.groups, groups = min(t.groups, g.groups - grp0), c_set = grp0 * g.cpg;
  const uint32_t col = threadIdx.x % t.cols, row = threadIdx.x / t.cols;
  const int n_c = int(groups * g.cpg) - int(col * V);
  const bool live = row < t.rows && n_c > 0;
  Held<T, V, kHold> f;
  if (live) f.load(x + int64_t(blockIdx.y) * xi + c_set + col * V, xp, row, t.rows, g.pixels, n_c);
  float v[V], mean[V], scale[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if (live && row + k * t.rows < g.pixels) v[i] += float(f.v[k][i]);
  }
  const float total = float(g.pixels) * float(g.cpg);
  channel_totals<V>(t, row < t.rows, v, s.part, s.sub, s.chan[0]);
  group_totals(groups, g.cpg, s.chan[0], nullptr, s.group[0]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    mean[i] = i < n_c ? s.group[0][(col * V + i) / g.cpg] / total : 0.0f;
    v[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const float d = live && row + k * t.rows < g.pixels && i < n_c ? float(f.v[k][i]) - mean[i] : 0.0f;
      v[i] = fmaf(d, d, v[i]);
    }
  }
  channel_totals<V>(t, row < t.rows, v, s.part, s.sub, s.chan[0]);
  group_totals(groups, g.cpg, s.chan[0], nullptr, s.group[1]);
  for (uint32_t k = threadIdx.x; k < groups; k += kSmallThreads)
    stats[uint64_t(blockIdx.y) * g.groups + grp0 + k] =
        GnStats{s.group[0][k] / total, 1.0f / sqrtf(s.group[1][k] / total + g.eps)};
  if (!live) return;
  float shift[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t c = c_set + col * V + i;
    scale[i] = i < n_c ? 1.0f / sqrtf(s.group[1][(col * V + i) / g.cpg] / total + g.eps) : 0.0f;
    if (i < n_c && gamma) scale[i] *= gamma[c];
    shift[i] = i < n_c && beta ? beta[c] : 0.0f;
  }
  T* yb = y + int64_t(blockIdx.y) * yi + c_set + col * V;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const uint32_t p = row + k * t.rows;
    if (p >= g.pixels) break;
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = act_value<ACT>(fmaf(float(f.v[k][i]) - mean[i], scale[i], shift[i]));
    store_f32<V>(yb + int64_t(p) * yp, n_c, o);
  }
}

// The backward pass in one launch, x and dy read once into registers; 9 us at the size above.
template <typename T, int ACT, int V>
__global__ __launch_bounds__(kSmallThreads) void k_gn_small_back(
    GnShape g, GnSet t, const T* __restrict__ x, int64_t xi, int64_t xp, const float* __restrict__ gamma,
    const float* __restrict__ beta, const GnStats* __restrict__ stats, const T* dy, int64_t di, int64_t dp, T* dx,
    int64_t oi, int64_t op, float* __restrict__ dgamma, float* __restrict__ dbeta, float2* __restrict__ chan) {
  constexpr int kHold = kHoldBackward;
  __shared__ SmallShared<V> s;
  const uint32_t grp0 = blockIdx.x * t.groups, groups = min(t.groups, g.groups - grp0), c_set = grp0 * g.cpg;
  const uint32_t col = threadIdx.x % t.cols, row = threadIdx.x / t.cols;
  const int n_c = int(groups * g.cpg) - int(col * V);
  const bool live = row < t.rows && n_c > 0;
  Held<T, V, kHold> f, d;
  Channel<V> ch;
  float a[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
  if (live) {
    f.load(x + int64_t(blockIdx.y) * xi + c_set + col * V, xp, row, t.rows, g.pixels, n_c);
    d.load(dy + int64_t(blockIdx.y) * di + c_set + col * V, dp, row, t.rows, g.pixels, n_c);
    ch.load(g, blockIdx.y, c_set + col * V, n_c, stats, gamma, beta);
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      if (row + k * t.rows >= g.pixels) break;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (float(f.v[k][i]) - ch.mean[i]) * ch.rstd[i];
        const float dz = float(d.v[k][i]) * act_slope<ACT>(fmaf(xh, ch.gamma[i], ch.beta[i]));
        a[i] += dz;
        b[i] = fmaf(dz, xh, b[i]);
      }
    }
  }
  channel_totals<V>(t, row < t.rows, a, s.part, s.sub, s.chan[0]);
  channel_totals<V>(t, row < t.rows, b, s.part, s.sub, s.chan[1]);
  group_totals(groups, g.cpg, s.chan[0], gamma ? gamma + c_set : nullptr, s.group[0]);
  group_totals(groups, g.cpg, s.chan[1], gamma ? gamma + c_set : nullptr, s.group[1]);
  const bool alone = g.images == 1;
  for (uint32_t c = threadIdx.x; c < groups * g.cpg; c += kSmallThreads) {
    if (!alone) chan[int64_t(blockIdx.y) * g.channels + c_set + c] = make_float2(s.chan[0][c], s.chan[1][c]);
    if (alone && dbeta) dbeta[c_set + c] = s.chan[0][c];
    if (alone && dgamma) dgamma[c_set + c] = s.chan[1][c];
  }
  if (live && dx) {
    const float inv = 1.0f / (float(g.pixels) * float(g.cpg));
    float m1[V], m2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t k = i < n_c ? (col * V + i) / g.cpg : 0;
      m1[i] = s.group[0][k] * inv;
      m2[i] = s.group[1][k] * inv;
    }
    T* ob = dx + int64_t(blockIdx.y) * oi + c_set + col * V;
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const uint32_t p = row + k * t.rows;
      if (p >= g.pixels) break;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (float(f.v[k][i]) - ch.mean[i]) * ch.rstd[i];
        const float dz = float(d.v[k][i]) * act_slope<ACT>(fmaf(xh, ch.gamma[i], ch.beta[i]));
        o[i] = ch.rstd[i] * (fmaf(dz, ch.gamma[i], -m1[i]) - xh * m2[i]);
      }
      store_f32<V>(ob + int64_t(p) * op, n_c, o);
    }
  }
}

// dgamma and dbeta from the images' channel sums, in order. (A last-workgroup-done counter inside k_gn_small_back saves
// this launch of 3 us, but its fences across the dies cost 15 us.)
__global__ void k_gn_images(uint32_t images, uint32_t channels, const float2* __restrict__ chan,
                            float* __restrict__ dgamma, float* __restrict__ dbeta) {
  const uint32_t c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= channels) return;
  float a = 0.0f, b = 0.0f;
#pragma unroll 8
  for (uint32_t n = 0; n < images; ++n) {
    const float2 v = chan[int64_t(n) * channels + c];
    a += v.x;
    b += v.y;
  }
  if (dbeta) dbeta[c] = a;
  if (dgamma) dgamma[c] = b;
}

// dgamma and dbeta when no pixel is there to sum.
__global__ void k_gn_zero(float* a, float* b, uint32_t n) {
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  if (a) a[i] = 0.0f;
  if (b) b[i] = 0.0f;
}

// The arguments both directions share.
gsr_status check_desc(gsr_ctx* ctx, const gsr_group_norm* d, const char* who) {
  if (!d) return fail(ctx, GSR_EINVAL, "%s: null descriptor", who);
  if (d->dtype > GSR_BF16) return fail(ctx, GSR_EINVAL, "%s: unknown dtype %u", who, d->dtype);
  if (d->activation > GSR_ACT_RELU) return fail(ctx, GSR_EINVAL, "%s: unknown activation %u", who, d->activation);
  if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return fail(ctx, GSR_EINVAL, "%s: eps must be finite and >= 0", who);
  if (d->groups == 0 || d->channels % d->groups)
    return fail(ctx, GSR_EINVAL, "%s: %u channels are not a multiple of %u groups", who, d->channels, d->groups);
  if (uint64_t(d->pixels) * (d->channels / d->groups) >= (uint64_t(1) << 31))
    return fail(ctx, GSR_EOVERFLOW, "%s: pixels * channels / groups >= 2^31", who);
  if (d->images >= (1u << 16)) return fail(ctx, GSR_EOVERFLOW, "%s: images >= 2^16", who);
  if (d->channels >= (1u << 20)) return fail(ctx, GSR_EOVERFLOW, "%s: channels >= 2^20", who);
  return GSR_OK;
}

gsr_status check_out(gsr_ctx* ctx, const gsr_group_norm* d, const int64_t* st, const char* who, const char* name) {
  if (!distinct({{st[0], d->images}, {st[1], d->pixels}}, d->channels))
    return fail(ctx, GSR_EINVAL, "%s: the strides of %s overlap", who, name);
  return GSR_OK;
}

// Threads across channels and pixels, and the pixels of a workgroup: about eight workgroups per compute unit, and at
// least four pixels per thread, so that the joins stay small.
GnShape shape_of(const gsr_group_norm* d) {
  GnShape g{};
  g.images = d->images;
  g.pixels = d->pixels;
  g.channels = d->channels;
  g.groups = d->groups;
  g.cpg = d->channels / d->groups;
  g.eps = d->eps;
  const uint32_t v = d->dtype == GSR_F32 ? 4 : 8;
  g.cols = std::min<uint32_t>((d->channels + v - 1) / v, kThreads);
  g.rows = kThreads / g.cols;
  const uint64_t want = std::max<uint64_t>(1, 2048 / std::max(1u, d->images));
  const uint64_t per = std::max<uint64_t>((d->pixels + want - 1) / want, 4 * g.rows);
  g.chunk = uint32_t((per + g.rows - 1) / g.rows * g.rows);
  g.chunks = uint32_t((uint64_t(d->pixels) + g.chunk - 1) / g.chunk);
  return g;
}

// The set of groups whose pixels a workgroup of the one-launch form holds, `hold` vectors of `*v` elements a thread, or
// false. Up to 1 MB of features, where time is latency, one group a workgroup and two elements a thread: most workgroups,
// shortest chains of work (a 3 x 323 x 90 float16 map: 11 us a launch with 128-byte strips on six workgroups). Above,
// the fewest groups that make a 128-byte strip of a row (64 if those do not fit; narrower strips waste the cache lines
// they touch), if that makes 64 workgroups: a forward pass of 2 x 2,000 x 512 float32 on 64 of them 17 us, by several
// launches 24; a training pass of 4 x 1,024 x 640 bfloat16, whose forward would have 44, 57 us against 49.
bool small_set(const GnShape& g, uint32_t dtype, uint32_t hold, GnSet* t, uint32_t* v) {
  const uint32_t eb = dtype == GSR_F32 ? 4 : 2;
  const bool tiny = uint64_t(g.images) * g.pixels * g.channels * eb <= (1u << 20);
  *v = tiny ? 2 : 16 / eb;
  for (uint32_t n = tiny ? 1 : std::min<uint32_t>(g.groups, (128 / eb + g.cpg - 1) / g.cpg); n >= 1; --n) {
    t->groups = n;
    t->channels = n * g.cpg;
    t->cols = (t->channels + *v - 1) / *v;
    if (t->cols * *v > kSmallThreads) continue;
    if (!tiny && t->channels * eb < 64 && n < g.groups) return false;
    t->rows = kSmallThreads / t->cols;
    const uint64_t sets = (g.groups + n - 1) / n;
    if (uint64_t(t->rows) * hold >= g.pixels) return tiny || sets * g.images >= 64;
  }
  return false;
}

dim3 grid_of(const GnShape& g, uint32_t dtype) {
  const uint32_t v = dtype == GSR_F32 ? 4 : 8;
  const uint32_t vecs = (g.channels + v - 1) / v;
  return dim3(g.chunks, g.images, (vecs + g.cols - 1) / g.cols);
}

// Calls f(element type, activation) with compile-time values.
template <typename F>
void by_kind(const gsr_group_norm* d, F f) {
  auto act = [&](auto t) {
    if (d->activation == GSR_ACT_SILU)
      f(t, std::integral_constant<int, GSR_ACT_SILU>());
    else if (d->activation == GSR_ACT_RELU)
      f(t, std::integral_constant<int, GSR_ACT_RELU>());
    else
      f(t, std::integral_constant<int, GSR_ACT_NONE>());
  };
  if (d->dtype == GSR_F32)
    act(float());
  else if (d->dtype == GSR_F16)
    act(_Float16());
  else
    act(__bf16());
}

}  // namespace
}  // namespace gsr

using namespace gsr;

extern "C" gsr_status gsr_group_norm_forward(gsr_ctx* ctx, void* stream, const gsr_group_norm* d, const void* x,
                                             const float* gamma, const float* beta, void* y, float* stats) {
  static const char* who = "gsr_group_norm_forward";
  if (!ctx) return GSR_EINVAL;
  gsr_status st = check_desc(ctx, d, who);
  if (st) return st;
  if (!d->images || !d->pixels || !d->channels) return GSR_OK;
  if (!x || !y || !stats) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  const size_t eb = elem_bytes(d->dtype);
  if (misaligned(x, eb) || misaligned(y, eb) || misaligned(gamma, 4) || misaligned(beta, 4) || misaligned(stats, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if ((st = check_out(ctx, d, d->y_stride, who, "y"))) return st;
  if ((st = enter(ctx))) return st;
  const GnShape g = shape_of(d);
  GnSet set;
  uint32_t vec;
  if (small_set(g, d->dtype, kHoldForward, &set, &vec)) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    timing_mark(ctx, GSR_STAGE_GROUP_NORM_FORWARD, s, false);
    by_kind(d, [&](auto t, auto a) {
      using T = decltype(t);
      auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((g.groups + set.groups - 1) / set.groups, g.images), dim3(kSmallThreads), 0, s,
                           g, set, static_cast<const T*>(x), d->x_stride[0], d->x_stride[1], gamma, beta,
                           reinterpret_cast<GnStats*>(stats), static_cast<T*>(y), d->y_stride[0], d->y_stride[1]);
      };
      if (vec == 2)
        launch(k_gn_small<T, decltype(a)::value, 2>);
      else
        launch(k_gn_small<T, decltype(a)::value, 16 / int(sizeof(T))>);
    });
    timing_mark(ctx, GSR_STAGE_GROUP_NORM_FORWARD, s, true);
    return check_launch(ctx, who);
  }
  if ((st = grow(ctx, ctx->arena.feat_part, size_t(g.images) * g.chunks * g.channels * sizeof(float2)))) return st;
  float2* part = static_cast<float2*>(ctx->arena.feat_part.ptr);
  GnStats* out = reinterpret_cast<GnStats*>(stats);
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_FORWARD, s, false);
  by_kind(d, [&](auto t, auto a) {
    using T = decltype(t);
    const T* xt = static_cast<const T*>(x);
    hipLaunchKernelGGL((k_gn_stats<T>), grid_of(g, d->dtype), dim3(kThreads), 0, s, g, xt, d->x_stride[0],
                       d->x_stride[1], part);
    hipLaunchKernelGGL(k_gn_finish, dim3(g.groups, g.images), dim3(kJoinThreads), 0, s, g, part, out);
    hipLaunchKernelGGL((k_gn_apply<T, decltype(a)::value>), grid_of(g, d->dtype), dim3(kThreads), 0, s, g, xt, d->x_stride[0],
                       d->x_stride[1], gamma, beta, out, static_cast<T*>(y), d->y_stride[0], d->y_stride[1]);
  });
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_FORWARD, s, true);
  return check_launch(ctx, who);
}

extern "C" gsr_status gsr_group_norm_backward(gsr_ctx* ctx, void* stream, const gsr_group_norm* d, const void* x,
                                              const float* gamma, const float* beta, const float* stats,
                                              const void* dy, void* dx, float* dgamma, float* dbeta) {
  static const char* who = "gsr_group_norm_backward";
  if (!ctx) return GSR_EINVAL;
  gsr_status st = check_desc(ctx, d, who);
  if (st) return st;
  if (!d->channels || (!dx && !dgamma && !dbeta)) return GSR_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (misaligned(dgamma, 4) || misaligned(dbeta, 4) || misaligned(gamma, 4) || misaligned(beta, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!d->images || !d->pixels) {
    if (!dgamma && !dbeta) return GSR_OK;
    if ((st = enter(ctx))) return st;
    hipLaunchKernelGGL(k_gn_zero, dim3((d->channels + 255) / 256), dim3(256), 0, s, dgamma, dbeta, d->channels);
    return check_launch(ctx, who);
  }
  if (!x || !stats || !dy) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  const size_t eb = elem_bytes(d->dtype);
  if (misaligned(x, eb) || misaligned(dy, eb) || misaligned(dx, eb) || misaligned(stats, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (dx && (st = check_out(ctx, d, d->dx_stride, who, "dx"))) return st;
  if ((st = enter(ctx))) return st;
  const GnShape g = shape_of(d);
  GnSet set;
  uint32_t vec;
  const bool small = small_set(g, d->dtype, kHoldBackward, &set, &vec);
  // one launch leaves the sums of several images alone in the scratch
  const size_t n_part = small ? 0 : size_t(g.images) * g.chunks * g.channels;
  const size_t n_chan = small && g.images == 1 ? 0 : size_t(g.images) * g.channels;
  const size_t n_group = small ? 0 : size_t(g.images) * g.groups;
  if ((st = grow(ctx, ctx->arena.feat_part, (n_part + n_chan + n_group) * sizeof(float2)))) return st;
  float2* part = static_cast<float2*>(ctx->arena.feat_part.ptr);
  float2* chan = part + n_part;
  float2* group = chan + n_chan;
  const GnStats* in = reinterpret_cast<const GnStats*>(stats);
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_BACKWARD, s, false);
  if (small) {
    by_kind(d, [&](auto t, auto a) {
      using T = decltype(t);
      auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((g.groups + set.groups - 1) / set.groups, g.images), dim3(kSmallThreads), 0, s,
                           g, set, static_cast<const T*>(x), d->x_stride[0], d->x_stride[1], gamma, beta, in,
                           static_cast<const T*>(dy), d->dy_stride[0], d->dy_stride[1], static_cast<T*>(dx),
                           d->dx_stride[0], d->dx_stride[1], dgamma, dbeta, chan);
      };
      if (vec == 2)
        launch(k_gn_small_back<T, decltype(a)::value, 2>);
      else
        launch(k_gn_small_back<T, decltype(a)::value, 16 / int(sizeof(T))>);
    });
    if (g.images > 1 && (dgamma || dbeta))
      hipLaunchKernelGGL(k_gn_images, dim3((g.channels + 63) / 64), dim3(64), 0, s, g.images, g.channels, chan, dgamma,
                         dbeta);
    timing_mark(ctx, GSR_STAGE_GROUP_NORM_BACKWARD, s, true);
    return check_launch(ctx, who);
  }
  by_kind(d, [&](auto t, auto a) {
    using T = decltype(t);
    const T *xt = static_cast<const T*>(x), *dt = static_cast<const T*>(dy);
    hipLaunchKernelGGL((k_gn_sums<T, decltype(a)::value>), grid_of(g, d->dtype), dim3(kThreads), 0, s, g, xt, d->x_stride[0],
                       d->x_stride[1], gamma, beta, in, dt, d->dy_stride[0], d->dy_stride[1], part);
    hipLaunchKernelGGL(k_gn_sums_join, dim3(g.groups, g.images), dim3(kJoinThreads), 0, s, g, part, gamma, chan, group);
    dim3 grid = grid_of(g, d->dtype);
    if (!dx) grid.x = grid.y = 1;
    hipLaunchKernelGGL((k_gn_dx<T, decltype(a)::value>), grid, dim3(kThreads), 0, s, g, xt, d->x_stride[0], d->x_stride[1], gamma, beta,
                       in, dt, d->dy_stride[0], d->dy_stride[1], chan, group, static_cast<T*>(dx), d->dx_stride[0],
                       d->dx_stride[1], dgamma, dbeta);
  });
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_BACKWARD, s, true);
  return check_launch(ctx, who);
}
