// Group norm with an activation over channels-last features, and its backward pass.
//
// A thread owns V adjacent channels (16 bytes) and walks pixels, so a wave reads whole pixel rows whatever the group
// width is (a group's channels alone are a short strip of each row). Sums are therefore kept per channel and joined
// to groups afterwards:
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

// Sum over the workgroup, in a fixed order; every thread gets it. `s` holds kThreads floats.
__device__ __forceinline__ float block_sum(float v, float* s) {
  const int t = threadIdx.x;
  __syncthreads();
  s[t] = v;
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h >>= 1) {
    if (t < h) s[t] += s[t + h];
    __syncthreads();
  }
  return s[0];
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

// Means and squared deviations per channel of one chunk of pixels. A thread's own first value of a channel is the
// shift of its sums: with d = x - shift, mean = shift + sum d / n and M2 = sum d^2 - (sum d)^2 / n. An outlying shift
// cannot spoil the group's variance, because it is itself one of the values: the rounding is at most n 2^-24 of
// (shift - mean)^2, a part of the sum it is added to.
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
  float shift[V], s1[V], s2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) shift[i] = s1[i] = s2[i] = 0.0f;
  uint32_t n = 0;
  if (live && p0 + row < p1) {
    load_f32<V>(base + int64_t(p0 + row) * xp, n_c, shift);
#pragma unroll 4
    for (uint32_t p = p0 + row; p < p1; p += g.rows) {
      float f[V];
      load_f32<V>(base + int64_t(p) * xp, n_c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = f[i] - shift[i];
        s1[i] += d;
        s2[i] = fmaf(d, d, s2[i]);
      }
      ++n;
    }
  }
  // (n, mean, M2) of the column: the mean first, then every thread's M2 about it
  const float inv = n ? 1.0f / float(n) : 0.0f;
  float m2[V], mean[V], part_mean[V], zero[V];
  const float share = float(n) / float(p1 - p0);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float d = s1[i] * inv;
    part_mean[i] = shift[i] + d;
    m2[i] = n ? fmaxf(fmaf(-s1[i], d, s2[i]), 0.0f) : 0.0f;
    if (!(s2[i] - s2[i] == 0.0f)) m2[i] = s2[i] - s2[i];  // infinities and NaN carry on as NaN
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

// Mean and rstd of one (image, group) from its chunks' channel statistics: the weighted mean of the means, then
// M2 = sum M2_i + n_i (mean_i - mean)^2.
__global__ __launch_bounds__(kThreads) void k_gn_finish(GnShape g, const float2* __restrict__ part,
                                                        float2* __restrict__ stats) {
  __shared__ float s[kThreads];
  const uint32_t grp = blockIdx.x, img = blockIdx.y;
  const float2* base = part + int64_t(img) * g.chunks * g.channels + grp * g.cpg;
  const uint32_t n = g.chunks * g.cpg;
  const float last = float(g.pixels - (g.chunks - 1) * g.chunk);
  const float total = float(g.pixels) * float(g.cpg);
  float m = 0.0f;
  for (uint32_t e = threadIdx.x; e < n; e += kThreads) {
    const uint32_t k = e / g.cpg;
    const float w = k + 1 == g.chunks ? last : float(g.chunk);
    m = fmaf(w / total, base[int64_t(k) * g.channels + (e - k * g.cpg)].x, m);
  }
  const float mean = block_sum(m, s);
  float q = 0.0f;
  for (uint32_t e = threadIdx.x; e < n; e += kThreads) {
    const uint32_t k = e / g.cpg;
    const float w = k + 1 == g.chunks ? last : float(g.chunk);
    const float2 v = base[int64_t(k) * g.channels + (e - k * g.cpg)];
    const float d = v.x - mean;
    q += fmaf(w * d, d, v.y);
  }
  const float var = block_sum(q, s) / total;
  if (threadIdx.x == 0) stats[img * g.groups + grp] = make_float2(mean, 1.0f / sqrtf(var + g.eps));
}

// The channel constants a thread keeps for its V channels of one image.
template <int V>
struct Channel {
  float mean[V], rstd[V], gamma[V], beta[V];
  __device__ __forceinline__ void load(const GnShape& g, uint32_t img, uint32_t c0, int n_c, const float2* stats,
                                       const float* gm, const float* bt) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t c = i < n_c ? c0 + i : g.channels - 1;
      const float2 st = stats[img * g.groups + c / g.cpg];
      mean[i] = st.x;
      rstd[i] = st.y;
      gamma[i] = gm ? gm[c] : 1.0f;
      beta[i] = bt ? bt[c] : 0.0f;
    }
  }
};

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_apply(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                       const float* __restrict__ gamma,
                                                       const float* __restrict__ beta,
                                                       const float2* __restrict__ stats, T* y, int64_t yi,
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
#pragma unroll 4
  for (uint32_t p = p0 + row; p < p1; p += g.rows) {
    float f[V];
    load_f32<V>(xb + int64_t(p) * xp, n_c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = act_value<ACT>(fmaf(f[i] - ch.mean[i], ch.rstd[i], ch.beta[i]));
    store_f32<V>(yb + int64_t(p) * yp, n_c, f);
  }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_sums(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                      const float* __restrict__ gamma,
                                                      const float* __restrict__ beta,
                                                      const float2* __restrict__ stats, const T* __restrict__ dy,
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

// One workgroup per (image, group): threads take (channel, part of the chunks), so that a wave reads along channels.
__global__ __launch_bounds__(kThreads) void k_gn_sums_join(GnShape g, const float2* __restrict__ part,
                                                           const float* __restrict__ gamma,
                                                           float2* __restrict__ chan, float2* __restrict__ group) {
  __shared__ float sa[kThreads], sb[kThreads];
  const uint32_t grp = blockIdx.x, img = blockIdx.y;
  const uint32_t width = min(g.cpg, uint32_t(kThreads)), lanes = kThreads / width;
  const uint32_t tc = threadIdx.x % width, tk = threadIdx.x / width;
  float ga = 0.0f, gb = 0.0f;
  for (uint32_t c0 = 0; c0 < g.cpg; c0 += width) {
    const uint32_t c = grp * g.cpg + c0 + tc;
    float a = 0.0f, b = 0.0f;
    if (tk < lanes && c0 + tc < g.cpg) {
      for (uint32_t k = tk; k < g.chunks; k += lanes) {
        const float2 v = part[(int64_t(img) * g.chunks + k) * g.channels + c];
        a += v.x;
        b += v.y;
      }
    }
    __syncthreads();
    sa[threadIdx.x] = a;
    sb[threadIdx.x] = b;
    __syncthreads();
    if (tk == 0 && c0 + tc < g.cpg) {
      for (uint32_t k = 1; k < lanes; ++k) {
        a += sa[k * width + tc];
        b += sb[k * width + tc];
      }
      chan[int64_t(img) * g.channels + c] = make_float2(a, b);
      const float gm = gamma ? gamma[c] : 1.0f;
      ga = fmaf(a, gm, ga);
      gb = fmaf(b, gm, gb);
    }
  }
  ga = block_sum(ga, sa);
  gb = block_sum(gb, sa);
  if (threadIdx.x == 0) {
    const float m = float(g.pixels) * float(g.cpg);
    group[img * g.groups + grp] = make_float2(ga / m, gb / m);
  }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kThreads) void k_gn_dx(GnShape g, const T* __restrict__ x, int64_t xi, int64_t xp,
                                                    const float* __restrict__ gamma, const float* __restrict__ beta,
                                                    const float2* __restrict__ stats, const T* dy, int64_t di,
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
    const float2 v = group[blockIdx.y * g.groups + c / g.cpg];
    m1[i] = v.x;
    m2[i] = v.y;
  }
  const uint32_t p0 = blockIdx.x * g.chunk, p1 = min(g.pixels, p0 + g.chunk);
  const T* xb = x + int64_t(blockIdx.y) * xi + c0;
  const T* db = dy + int64_t(blockIdx.y) * di + c0;
  T* ob = dx + int64_t(blockIdx.y) * oi + c0;
#pragma unroll 2
  for (uint32_t p = p0 + row; p < p1; p += g.rows) {
    float f[V], d[V];
    load_f32<V>(xb + int64_t(p) * xp, n_c, f);
    load_f32<V>(db + int64_t(p) * dp, n_c, d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float xh = (f[i] - ch.mean[i]) * ch.rstd[i];
      const float dz = d[i] * act_slope<ACT>(fmaf(xh, ch.gamma[i], ch.beta[i]));
      d[i] = ch.rstd[i] * (fmaf(dz, ch.gamma[i], -m1[i]) - xh * m2[i]);
    }
    store_f32<V>(ob + int64_t(p) * op, n_c, d);
  }
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
  if (misaligned(x, eb) || misaligned(y, eb) || misaligned(gamma, 4) || misaligned(beta, 4) || misaligned(stats, 8))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if ((st = check_out(ctx, d, d->y_stride, who, "y"))) return st;
  if ((st = enter(ctx))) return st;
  const GnShape g = shape_of(d);
  if ((st = grow(ctx, ctx->arena.feat_part, size_t(g.images) * g.chunks * g.channels * sizeof(float2)))) return st;
  float2* part = static_cast<float2*>(ctx->arena.feat_part.ptr);
  float2* out = reinterpret_cast<float2*>(stats);
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_FORWARD, s, false);
  by_kind(d, [&](auto t, auto a) {
    using T = decltype(t);
    const T* xt = static_cast<const T*>(x);
    hipLaunchKernelGGL((k_gn_stats<T>), grid_of(g, d->dtype), dim3(kThreads), 0, s, g, xt, d->x_stride[0],
                       d->x_stride[1], part);
    hipLaunchKernelGGL(k_gn_finish, dim3(g.groups, g.images), dim3(kThreads), 0, s, g, part, out);
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
  if (misaligned(x, eb) || misaligned(dy, eb) || misaligned(dx, eb) || misaligned(stats, 8))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (dx && (st = check_out(ctx, d, d->dx_stride, who, "dx"))) return st;
  if ((st = enter(ctx))) return st;
  const GnShape g = shape_of(d);
  const size_t n_part = size_t(g.images) * g.chunks * g.channels, n_chan = size_t(g.images) * g.channels;
  if ((st = grow(ctx, ctx->arena.feat_part, (n_part + n_chan + size_t(g.images) * g.groups) * sizeof(float2))))
    return st;
  float2* part = static_cast<float2*>(ctx->arena.feat_part.ptr);
  float2* chan = part + n_part;
  float2* group = chan + n_chan;
  const float2* in = reinterpret_cast<const float2*>(stats);
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_BACKWARD, s, false);
  by_kind(d, [&](auto t, auto a) {
    using T = decltype(t);
    const T *xt = static_cast<const T*>(x), *dt = static_cast<const T*>(dy);
    hipLaunchKernelGGL((k_gn_sums<T, decltype(a)::value>), grid_of(g, d->dtype), dim3(kThreads), 0, s, g, xt, d->x_stride[0],
                       d->x_stride[1], gamma, beta, in, dt, d->dy_stride[0], d->dy_stride[1], part);
    hipLaunchKernelGGL(k_gn_sums_join, dim3(g.groups, g.images), dim3(kThreads), 0, s, g, part, gamma, chan, group);
    dim3 grid = grid_of(g, d->dtype);
    if (!dx) grid.x = grid.y = 1;
    hipLaunchKernelGGL((k_gn_dx<T, decltype(a)::value>), grid, dim3(kThreads), 0, s, g, xt, d->x_stride[0], d->x_stride[1], gamma, beta,
                       in, dt, d->dy_stride[0], d->dy_stride[1], chan, group, static_cast<T*>(dx), d->dx_stride[0],
                       d->dx_stride[1], dgamma, dbeta);
  });
  timing_mark(ctx, GSR_STAGE_GROUP_NORM_BACKWARD, s, true);
  return check_launch(ctx, who);
}
