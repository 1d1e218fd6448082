// Rotary positions with several axes: each pair of a head's elements is turned by an angle set by the token's position
// on the pair's axis. One read and one write of the features; the sine and cosine of a (token, pair) are shared by all
// heads, so a thread keeps them for its pairs and walks the heads.
//
// The angle p base^(-i / n) is kept in turns: with f = base^(-i / n) / (2 pi) as a sum hi + lo of two floats (rounded
// from a double on the host), p hi splits into its rounded product t and the exact remainder fma(p, hi, -t), so the
// fraction of a turn (t - rint(t)) + (remainder + p lo) carries an error near 2^-25 of a turn at any position up to
// 2^24, where a float angle would be off by p 2^-24 radians.
#include <type_traits>

#include "feature_common.hpp"

namespace gsr {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // wide loads in flight before the first store (x may be out, so the compiler keeps their order)

struct RotaryArgs {
  uint64_t items;  // tokens of all batch entries * units per token
  uint32_t tokens, heads, head_dim, units, pairs, axes, heads_per_thread;
  int64_t x_stride[3], out_stride[3], pos_stride;
  uint8_t axis[GSR_ROTARY_MAX_PAIRS];
  float hi[GSR_ROTARY_MAX_PAIRS], lo[GSR_ROTARY_MAX_PAIRS];
};

__device__ __forceinline__ void turn(const RotaryArgs& a, const float* pos, uint32_t pair, bool back, float* c,
                                     float* s) {
  const float p = pos[a.axis[pair]], hi = a.hi[pair];
  const float t = p * hi;
  const float r = (t - rintf(t)) + fmaf(p, a.lo[pair], fmaf(p, hi, -t));
  float sn, cs;
  sincospif(2.0f * r, &sn, &cs);
  *c = cs;
  *s = back ? -sn : sn;
}

// Interleaved pairs: a unit is V adjacent elements (V / 2 pairs).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_rotary_interleaved(RotaryArgs a, const T* x,
                                                                 const float* __restrict__ positions, T* out,
                                                                 bool back) {
  constexpr int V = 16 / sizeof(T);
  const uint64_t id = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (id >= a.items) return;
  const uint32_t unit = uint32_t(id % a.units);
  const uint64_t tok = id / a.units;
  const uint64_t b = tok / a.tokens, t = tok % a.tokens;
  const float* pos = positions + int64_t(b) * a.pos_stride + int64_t(t) * a.axes;
  const uint32_t e0 = unit * V;
  const int n = int(a.head_dim) - int(e0);
  float c[V / 2], s[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const uint32_t pair = e0 / 2 + i;
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (pair < a.pairs) turn(a, pos, pair, back, &c[i], &s[i]);
  }
  const uint32_t h0 = blockIdx.y * a.heads_per_thread, h1 = min(a.heads, h0 + a.heads_per_thread);
  const T* xp = x + int64_t(b) * a.x_stride[0] + int64_t(t) * a.x_stride[1] + e0;
  T* op = out + int64_t(b) * a.out_stride[0] + int64_t(t) * a.out_stride[1] + e0;
  auto turned = [&](float* f) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float u = f[2 * i], v = f[2 * i + 1];
      if (e0 / 2 + i < a.pairs) {
        f[2 * i] = fmaf(u, c[i], -(v * s[i]));
        f[2 * i + 1] = fmaf(u, s[i], v * c[i]);
      }
    }
  };
  uint32_t h = h0;
  for (; h + kAtOnce <= h1; h += kAtOnce) {
    float f[kAtOnce][V];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) load_f32<V>(xp + int64_t(h + k) * a.x_stride[2], n, f[k]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) turned(f[k]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) store_f32<V>(op + int64_t(h + k) * a.out_stride[2], n, f[k]);
  }
  for (; h < h1; ++h) {
    float f[V];
    load_f32<V>(xp + int64_t(h) * a.x_stride[2], n, f);
    turned(f);
    store_f32<V>(op + int64_t(h) * a.out_stride[2], n, f);
  }
}

// Split halves: a unit is V adjacent pairs, elements (i ..) and (i + pairs ..); the units after them copy V elements
// of the rest each.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_rotary_halves(RotaryArgs a, const T* x,
                                                            const float* __restrict__ positions, T* out, bool back) {
  constexpr int V = 16 / sizeof(T);
  const uint64_t id = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (id >= a.items) return;
  const uint32_t unit = uint32_t(id % a.units);
  const uint64_t tok = id / a.units;
  const uint64_t b = tok / a.tokens, t = tok % a.tokens;
  const float* pos = positions + int64_t(b) * a.pos_stride + int64_t(t) * a.axes;
  const uint32_t turning = (a.pairs + V - 1) / V;
  const uint32_t h0 = blockIdx.y * a.heads_per_thread, h1 = min(a.heads, h0 + a.heads_per_thread);
  const T* xp = x + int64_t(b) * a.x_stride[0] + int64_t(t) * a.x_stride[1];
  T* op = out + int64_t(b) * a.out_stride[0] + int64_t(t) * a.out_stride[1];
  if (unit >= turning) {
    const uint32_t e0 = 2 * a.pairs + (unit - turning) * V;
    const int n = int(a.head_dim) - int(e0);
    for (uint32_t h = h0; h < h1; ++h) {
      float f[V];
      load_f32<V>(xp + int64_t(h) * a.x_stride[2] + e0, n, f);
      store_f32<V>(op + int64_t(h) * a.out_stride[2] + e0, n, f);
    }
    return;
  }
  const uint32_t e0 = unit * V;
  const int n = int(a.pairs) - int(e0);
  float c[V], s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = s[i] = 0.0f;
    if (i < n) turn(a, pos, e0 + i, back, &c[i], &s[i]);
  }
  auto turned = [&](float* u, float* v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float w = fmaf(u[i], c[i], -(v[i] * s[i]));
      v[i] = fmaf(u[i], s[i], v[i] * c[i]);
      u[i] = w;
    }
  };
  constexpr int kPairsAtOnce = kAtOnce / 2;
  uint32_t h = h0;
  for (; h + kPairsAtOnce <= h1; h += kPairsAtOnce) {
    float u[kPairsAtOnce][V], v[kPairsAtOnce][V];
#pragma unroll
    for (int k = 0; k < kPairsAtOnce; ++k) {
      load_f32<V>(xp + int64_t(h + k) * a.x_stride[2] + e0, n, u[k]);
      load_f32<V>(xp + int64_t(h + k) * a.x_stride[2] + e0 + a.pairs, n, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kPairsAtOnce; ++k) turned(u[k], v[k]);
#pragma unroll
    for (int k = 0; k < kPairsAtOnce; ++k) {
      store_f32<V>(op + int64_t(h + k) * a.out_stride[2] + e0, n, u[k]);
      store_f32<V>(op + int64_t(h + k) * a.out_stride[2] + e0 + a.pairs, n, v[k]);
    }
  }
  for (; h < h1; ++h) {
    float u[V], v[V];
    load_f32<V>(xp + int64_t(h) * a.x_stride[2] + e0, n, u);
    load_f32<V>(xp + int64_t(h) * a.x_stride[2] + e0 + a.pairs, n, v);
    turned(u, v);
    store_f32<V>(op + int64_t(h) * a.out_stride[2] + e0, n, u);
    store_f32<V>(op + int64_t(h) * a.out_stride[2] + e0 + a.pairs, n, v);
  }
}

gsr_status rotary(gsr_ctx* ctx, void* stream, const gsr_rotary* d, const void* x, const float* positions, void* out,
                  bool back, const char* who) {
  if (!ctx) return GSR_EINVAL;
  if (!d) return fail(ctx, GSR_EINVAL, "%s: null descriptor", who);
  if (d->dtype > GSR_BF16) return fail(ctx, GSR_EINVAL, "%s: unknown dtype %u", who, d->dtype);
  if (d->layout > GSR_ROTARY_HALVES) return fail(ctx, GSR_EINVAL, "%s: unknown layout %u", who, d->layout);
  if (d->axes < 1 || d->axes > GSR_ROTARY_MAX_AXES)
    return fail(ctx, GSR_EINVAL, "%s: %u axes, 1 to %d are supported", who, d->axes, GSR_ROTARY_MAX_AXES);
  if (!(d->base > 0.0f) || std::isinf(d->base)) return fail(ctx, GSR_EINVAL, "%s: base must be finite and > 0", who);
  uint64_t pairs = 0;
  for (uint32_t a = 0; a < d->axes; ++a) pairs += d->axis_pairs[a];
  if (pairs > d->head_dim / 2 || pairs > GSR_ROTARY_MAX_PAIRS)
    return fail(ctx, GSR_EINVAL, "%s: %llu pairs do not fit a head of %u elements (at most %d pairs)", who,
                (unsigned long long)pairs, d->head_dim, GSR_ROTARY_MAX_PAIRS);
  if (uint64_t(d->batch) * d->tokens >= (uint64_t(1) << 31))
    return fail(ctx, GSR_EOVERFLOW, "%s: batch * tokens >= 2^31", who);
  if (d->heads >= (1u << 16) || d->head_dim >= (1u << 16))
    return fail(ctx, GSR_EOVERFLOW, "%s: heads or head_dim >= 2^16", who);
  if (!d->batch || !d->tokens || !d->heads || !d->head_dim) return GSR_OK;
  if (!x || !positions || !out) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  const size_t eb = elem_bytes(d->dtype);
  if (misaligned(x, eb) || misaligned(out, eb) || misaligned(positions, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!distinct({{d->out_stride[0], d->batch}, {d->out_stride[1], d->tokens}, {d->out_stride[2], d->heads}},
                d->head_dim))
    return fail(ctx, GSR_EINVAL, "%s: the strides of the output overlap", who);
  gsr_status st = enter(ctx);
  if (st) return st;
  RotaryArgs a{};
  a.tokens = d->tokens;
  a.heads = d->heads;
  a.head_dim = d->head_dim;
  a.pairs = uint32_t(pairs);
  a.axes = d->axes;
  for (int i = 0; i < 3; ++i) {
    a.x_stride[i] = d->x_stride[i];
    a.out_stride[i] = d->out_stride[i];
  }
  a.pos_stride = d->position_stride;
  uint32_t at = 0;
  for (uint32_t ax = 0; ax < d->axes; ++ax)
    for (uint32_t i = 0; i < d->axis_pairs[ax]; ++i, ++at) {
      const double f = std::exp2(-std::log2(double(d->base)) * i / d->axis_pairs[ax]) / 6.283185307179586476925;
      a.axis[at] = uint8_t(ax);
      a.hi[at] = float(f);
      a.lo[at] = float(f - double(a.hi[at]));
    }
  const uint32_t v = d->dtype == GSR_F32 ? 4 : 8;
  if (d->layout == GSR_ROTARY_INTERLEAVED)
    a.units = (d->head_dim + v - 1) / v;
  else
    a.units = (a.pairs + v - 1) / v + (d->head_dim - 2 * a.pairs + v - 1) / v;
  a.items = uint64_t(d->batch) * d->tokens * a.units;
  // a thread takes several heads (sharing their sines) once the tokens alone fill the compute units
  a.heads_per_thread = 1;
  while (a.heads_per_thread < d->heads && a.items * (d->heads / (2 * a.heads_per_thread)) >= (1u << 19))
    a.heads_per_thread *= 2;
  const dim3 grid(uint32_t((a.items + kThreads - 1) / kThreads),
                  (d->heads + a.heads_per_thread - 1) / a.heads_per_thread);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto launch = [&](auto t) {
    using T = decltype(t);
    const T* xt = static_cast<const T*>(x);
    if (d->layout == GSR_ROTARY_INTERLEAVED)
      hipLaunchKernelGGL((k_rotary_interleaved<T>), grid, dim3(kThreads), 0, s, a, xt, positions,
                         static_cast<T*>(out), back);
    else
      hipLaunchKernelGGL((k_rotary_halves<T>), grid, dim3(kThreads), 0, s, a, xt, positions, static_cast<T*>(out),
                         back);
  };
  timing_mark(ctx, GSR_STAGE_ROTARY, s, false);
  if (d->dtype == GSR_F32)
    launch(float());
  else if (d->dtype == GSR_F16)
    launch(_Float16());
  else
    launch(__bf16());
  timing_mark(ctx, GSR_STAGE_ROTARY, s, true);
  return check_launch(ctx, who);
}

}  // namespace
}  // namespace gsr

using namespace gsr;

extern "C" gsr_status gsr_rotary_forward(gsr_ctx* ctx, void* stream, const gsr_rotary* d, const void* x,
                                         const float* positions, void* out) {
  return rotary(ctx, stream, d, x, positions, out, false, "gsr_rotary_forward");
}

extern "C" gsr_status gsr_rotary_backward(gsr_ctx* ctx, void* stream, const gsr_rotary* d, const void* dout,
                                          const float* positions, void* dx) {
  return rotary(ctx, stream, d, dout, positions, dx, true, "gsr_rotary_backward");
}
