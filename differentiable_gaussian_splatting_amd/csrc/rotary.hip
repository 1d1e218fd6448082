// Rotary positions with several axes: each pair of a head's elements is turned by an angle set by the token's position
// on the pair's axis. One read and one write of the features. A workgroup takes a few whole tokens: it computes their
// sines and cosines once, in LDS, and streams every head of them past, adjacent threads on adjacent 16 bytes; the first
// loads are in flight while the angles are computed.
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

struct RotaryArgs {
  uint32_t all_tokens;  // of all batch entries
  uint32_t heads, head_dim, pairs, axes;
  uint32_t group;       // tokens of a workgroup
  uint32_t turning;     // units of a head that turn (split halves)
  FastDiv units, head_div, pair_div, token_div;
  int64_t x_stride[3], out_stride[3], pos_stride;
  uint8_t axis[GSR_ROTARY_MAX_PAIRS];
  float hi[GSR_ROTARY_MAX_PAIRS], lo[GSR_ROTARY_MAX_PAIRS];
};

// The cosine and sine of pair `pair` at the token's positions `pos`.
__device__ __forceinline__ float2 turn(const RotaryArgs& a, const float* pos, uint32_t pair, bool back) {
  const float p = pos[a.axis[pair]], hi = a.hi[pair];
  const float t = p * hi;
  const float r = (t - rintf(t)) + fmaf(p, a.lo[pair], fmaf(p, hi, -t));
  float sn, cs;
  sincospif(2.0f * r, &sn, &cs);
  return make_float2(cs, back ? -sn : sn);
}

constexpr uint32_t kAngles = 2048;  // (token, pair) angles a workgroup keeps

// A unit is V adjacent elements: V / 2 interleaved pairs, or with split halves V pairs (two loads, V elements apart by
// the pairs) and, after those, V elements of the rest, which are copied.
// Bound by memory: 4 x 10,000 tokens, 16 heads of 128 bfloat16 (328 MB read and written) 68 us, 4.8 TB/s, a copy's rate
// at that size being 5.1 to 5.3; 2 x 2,501 tokens, 12 heads of 80 float16 with split halves (19 MB) 13 us; one token
// 2.3 us, the shortest a launch takes. 2,048 angles (16 KB of LDS) let eight workgroups share a compute unit.
template <typename T, bool kHalves>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a, const T* x, const float* __restrict__ positions,
                                                     T* out, bool back) {
  constexpr int V = 16 / sizeof(T), kAtOnce = kHalves ? 2 : 4;
  __shared__ float2 s_turn[kAngles];
  const uint64_t first = grid_index() * a.group;
  if (first >= a.all_tokens) return;
  const uint32_t tok0 = uint32_t(first), group = min(a.group, a.all_tokens - tok0);
  const uint32_t items = group * a.heads * a.units.d;
  struct Item {
    const T* from;
    T* to;
    uint32_t token, e0;  // within the group; first element (or pair, of a turning unit of split halves)
    int n;               // elements (pairs) of the unit; <= 0: none
    bool turns;
    float u[V], v[kHalves ? V : 1];
  };
  auto load = [&](uint32_t e, Item& it) {
    it.n = 0;
    if (e >= items) return;
    const uint32_t th = a.units.div(e), unit = e - th * a.units.d;
    it.token = a.head_div.div(th);
    const uint32_t head = th - it.token * a.heads;
    const uint32_t tok = tok0 + it.token, b = a.token_div.div(tok), t = tok - b * a.token_div.d;
    it.turns = !kHalves || unit < a.turning;
    it.e0 = kHalves && !it.turns ? 2 * a.pairs + (unit - a.turning) * V : unit * V;
    it.n = int(kHalves && it.turns ? a.pairs : a.head_dim) - int(it.e0);
    it.from = x + int64_t(b) * a.x_stride[0] + int64_t(t) * a.x_stride[1] + int64_t(head) * a.x_stride[2] + it.e0;
    it.to = out + int64_t(b) * a.out_stride[0] + int64_t(t) * a.out_stride[1] + int64_t(head) * a.out_stride[2] + it.e0;
    load_f32<V>(it.from, it.n, it.u);
    if constexpr (kHalves)
      if (it.turns) load_f32<V>(it.from + a.pairs, it.n, it.v);
  };
  auto finish = [&](Item& it) {
    if (it.n <= 0) return;
    const float2* cs = s_turn + it.token * a.pairs;
    if constexpr (kHalves) {
      if (it.turns) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 r = i < it.n ? cs[it.e0 + i] : make_float2(1.0f, 0.0f);
          const float w = fmaf(it.u[i], r.x, -(it.v[i] * r.y));
          it.v[i] = fmaf(it.u[i], r.y, it.v[i] * r.x);
          it.u[i] = w;
        }
        store_f32<V>(it.to + a.pairs, it.n, it.v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const uint32_t pair = it.e0 / 2 + i;
        if (pair >= a.pairs) break;
        const float2 r = cs[pair];
        const float u = it.u[2 * i], v = it.u[2 * i + 1];
        it.u[2 * i] = fmaf(u, r.x, -(v * r.y));
        it.u[2 * i + 1] = fmaf(u, r.y, v * r.x);
      }
    }
    store_f32<V>(it.to, it.n, it.u);
  };
  Item it[kAtOnce];
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) load(threadIdx.x + k * kThreads, it[k]);
  for (uint32_t e = threadIdx.x; e < group * a.pairs; e += kThreads) {
    const uint32_t token = a.pair_div.div(e), pair = e - token * a.pairs;
    const uint32_t tok = tok0 + token, b = a.token_div.div(tok), t = tok - b * a.token_div.d;
    s_turn[e] = turn(a, positions + int64_t(b) * a.pos_stride + int64_t(t) * a.axes, pair, back);
  }
  __syncthreads();
  for (uint32_t e0 = threadIdx.x; e0 < items; e0 += kAtOnce * kThreads) {
    // all of a batch is loaded before any of it is stored: x may be out, and the compiler keeps their order
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) finish(it[k]);
    if (e0 + kAtOnce * kThreads < items) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) load(e0 + (kAtOnce + k) * kThreads, it[k]);
    }
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
  a.all_tokens = d->batch * d->tokens;
  a.token_div.set(d->tokens);
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
  const bool halves = d->layout == GSR_ROTARY_HALVES;
  a.turning = (a.pairs + v - 1) / v;
  const uint32_t units = halves ? a.turning + (d->head_dim - 2 * a.pairs + v - 1) / v : (d->head_dim + v - 1) / v;
  a.units.set(units);
  a.head_div.set(d->heads);
  a.pair_div.set(std::max(1u, a.pairs));
  // whole tokens of about 2048 units a workgroup, at most kAngles angles; fewer where that leaves compute units idle
  const uint64_t per_token = uint64_t(units) * d->heads;
  uint64_t group = std::max<uint64_t>(1, std::min<uint64_t>(2048 / per_token, kAngles / std::max(1u, a.pairs)));
  group = std::min(group, std::max<uint64_t>(1, a.all_tokens / 1024));
  a.group = uint32_t(group);
  const dim3 grid = grid_rows((uint64_t(a.all_tokens) + group - 1) / group);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto launch = [&](auto t) {
    using T = decltype(t);
    const T* xt = static_cast<const T*>(x);
    if (halves)
      hipLaunchKernelGGL((k_rotary<T, true>), grid, dim3(kThreads), 0, s, a, xt, positions, static_cast<T*>(out), back);
    else
      hipLaunchKernelGGL((k_rotary<T, false>), grid, dim3(kThreads), 0, s, a, xt, positions, static_cast<T*>(out),
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
