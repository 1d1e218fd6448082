// Cross attention, forward: o = softmax(scale q k^T) v in one pass over the keys, with the running maximum and sum of
// the softmax (in base 2: exp(scale s) = 2^(c s), c = scale log2 e).
//
// A workgroup holds 128 rows (query, head of one key head's group: heads that share keys share the tiles), 32 to a
// wave, and streams tiles of keys and values through LDS; the next tile's loads are in flight while a tile is
// multiplied. Scores are computed transposed (keys down, queries across), so that a query's maximum and sum are a
// lane's own registers plus one exchange between the wave's halves. With few rows and many keys, the keys are split
// over workgroups and k_attn_join adds the parts in order.
#include <type_traits>

#include "attention_common.hpp"

namespace gsr {
namespace {

template <typename T, int DP>
constexpr int kKeyTile = sizeof(T) == 2 ? 64 : 32;

template <typename T, int DP, bool kMask>
__global__ __launch_bounds__(kAttnThreads) void k_attn_fwd(AttnArgs a) {
  using L = Tile<T, DP>;
  constexpr int KT = kKeyTile<T, DP>, kBlocks = KT / 32, kLoads = (KT * L::kChunks + kAttnThreads - 1) / kAttnThreads;
  __shared__ __attribute__((aligned(16))) char s_k[KT * L::kRowBytes];
  __shared__ __attribute__((aligned(16))) char s_v[KT * L::kRowBytes];
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, dim = int(a.dim);
  const uint32_t row = w.tile * kAttnRows + (tid >> 6) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const bool active = w.tile * kAttnRows + (tid >> 6) * 32 < a.rows;  // the wave has a row
  uint32_t query = 0, head = 0;
  if (valid) row_of(a, w.kv_head, row, &query, &head);
  Vec<T, 8> qf[DP / 16];
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) qf[kk] = zero_frag<T>();
  if (valid) {
    const T* qr = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + int64_t(query) * a.qs[1] +
                  int64_t(head) * a.qs[2];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) qf[kk] = load_frag(qr, kk, dim);
  }
  const uint8_t* mask = nullptr;
  if constexpr (kMask)
    mask = a.mask + int64_t(w.batch) * a.ms[0] + int64_t(head) * a.ms[1] + int64_t(query) * a.ms[2];
  const uint32_t len = keys_of(a, w.batch), tiles = (len + KT - 1) / KT;
  const uint32_t t0 = uint32_t(uint64_t(tiles) * w.split / a.splits);
  const uint32_t t1 = uint32_t(uint64_t(tiles) * (w.split + 1) / a.splits);
  const T* kb = static_cast<const T*>(a.k) + int64_t(w.batch) * a.ks[0] + int64_t(w.kv_head) * a.ks[2];
  const T* vb = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(w.kv_head) * a.vs[2];

  u32x4 rk[kLoads], rv[kLoads];
  auto fetch = [&](uint32_t t) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kAttnThreads, r = e / L::kChunks, c = e % L::kChunks * L::kPer;
      const uint32_t key = t * KT + r;
      rk[i] = rv[i] = u32x4{0, 0, 0, 0};
      if (key < len && c < dim && r < KT) {
        rk[i] = load_chunk(kb + int64_t(key) * a.ks[1], c, dim);
        rv[i] = load_chunk(vb + int64_t(key) * a.vs[1], c, dim);
      }
    }
  };

  const float c = a.scale * kLog2e;
  f32x16 o[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) o[dt] = f32x16{};
  float m = -INFINITY, m_c = 0.0f, l = 0.0f;  // running maximum of the scores, c times it (0 while there is none), sum
  if (t0 < t1) fetch(t0);
  for (uint32_t t = t0; t < t1; ++t) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kAttnThreads, r = e / L::kChunks;
      if (r < KT) {
        *reinterpret_cast<u32x4*>(s_k + L::at(r, e % L::kChunks)) = rk[i];
        *reinterpret_cast<u32x4*>(s_v + L::at(r, e % L::kChunks)) = rv[i];
      }
      if constexpr (kMask) odd |= any_nonfinite<T>(rv[i]);
    }
    if constexpr (kMask)
      odd = __syncthreads_or(odd);
    else
      __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    if (active) {
      f32x16 s[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        s[b] = f32x16{};
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) s[b] = mma(L::frag(s_k, 32 * b, kk), qf[kk], s[b]);
      }
      uint32_t seen[kBlocks];
      if (kMask || (t + 1) * KT > len) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          seen[b] = 0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t key = t * KT + 32 * b + 8 * g + 4 * h;
            uint32_t bytes = 0x01010101u;
            if constexpr (kMask) {
              bytes = 0;
              if (valid) {
                if (key + 4 <= len) {
                  __builtin_memcpy(&bytes, mask + key, 4);
                } else {
                  for (uint32_t i = 0; i < 4; ++i)
                    if (key + i < len) bytes |= uint32_t(mask[key + i]) << (8 * i);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool vis = key + i < len && ((bytes >> (8 * i)) & 0xffu) != 0;
              seen[b] |= uint32_t(vis) << (4 * g + i);
              s[b][4 * g + i] = vis ? s[b][4 * g + i] : -INFINITY;
            }
          }
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      top = fmaxf(top, other_half(top));
      if (__any(top > m)) {
        const float m_new = fmaxf(m, top), mc_new = m_new == -INFINITY ? 0.0f : m_new * c;
        const float f = m == -INFINITY ? 0.0f : exp2_fast(m_c - mc_new);
        m = m_new;
        m_c = mc_new;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[dt][i] *= f;
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[b][i] = exp2_fast(fmaf(s[b][i], c, kLift<T> - m_c));
          l += s[b][i];
        }
        contract<T, DP>(o, s_v, 32 * b, s[b], kMask && odd, seen[b]);
      }
    }
    __syncthreads();
  }
  if (!valid) return;
  l += other_half(l);
  if (a.splits > 1) {
    const int64_t at = (int64_t(w.batch * a.kv_heads + w.kv_head) * a.splits + w.split) * a.rows + row;
    store_column<float, DP>(a.part + at * dim, o, 1.0f, dim);
    if (h == 0) reinterpret_cast<float2*>(a.part_ml)[at] = make_float2(l == 0.0f ? -INFINITY : m_c, l);
    return;
  }
  T* out = static_cast<T*>(a.out) + int64_t(w.batch) * a.os[0] + int64_t(query) * a.os[1] + int64_t(head) * a.os[2];
  store_column<T, DP>(out, o, l == 0.0f ? 0.0f : 1.0f / l, dim);
  if (a.lse && h == 0)
    a.lse[(int64_t(w.batch) * a.heads + head) * a.queries + query] = l == 0.0f ? -INFINITY : (m_c - kLift<T> + log2f(l)) * kLn2;
}

// Joins the parts of rows whose keys were split: a thread per (row, element).
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void k_attn_join(AttnArgs a) {
  const uint64_t id = uint64_t(blockIdx.x) * kAttnThreads + threadIdx.x;
  const uint64_t rows = uint64_t(a.batch) * a.kv_heads * a.rows;
  if (id >= rows * a.dim) return;
  const uint32_t d = uint32_t(id % a.dim);
  const uint64_t at = id / a.dim, group = at / a.rows;
  const uint32_t row = uint32_t(at % a.rows), kv_head = uint32_t(group % a.kv_heads), b = uint32_t(group / a.kv_heads);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + group * a.splits * a.rows + row;
  const float* part = a.part + (group * a.splits * a.rows + row) * a.dim + d;
  float top = -INFINITY;
  for (uint32_t s = 0; s < a.splits; ++s) top = fmaxf(top, ml[uint64_t(s) * a.rows].x);
  float l = 0.0f, o = 0.0f;
  for (uint32_t s = 0; s < a.splits; ++s) {
    const float2 v = ml[uint64_t(s) * a.rows];
    if (v.x == -INFINITY) continue;
    const float f = exp2_fast(v.x - top);
    l = fmaf(v.y, f, l);
    o = fmaf(part[uint64_t(s) * a.rows * a.dim], f, o);
  }
  uint32_t query, head;
  row_of(a, kv_head, row, &query, &head);
  T* out = static_cast<T*>(a.out) + int64_t(b) * a.os[0] + int64_t(query) * a.os[1] + int64_t(head) * a.os[2];
  out[d] = T(l == 0.0f ? 0.0f : o / l);
  if (a.lse && d == 0)
    a.lse[(int64_t(b) * a.heads + head) * a.queries + query] = l == 0.0f ? -INFINITY : (top - kLift<T> + log2f(l)) * kLn2;
}

}  // namespace

gsr_status attention_args(gsr_ctx* ctx, const gsr_attention* d, const void* q, const void* k, const void* v,
                          const int32_t* kv_lengths, const uint8_t* mask, const void* o, const char* who,
                          AttnArgs* a) {
  if (!d) return fail(ctx, GSR_EINVAL, "%s: null descriptor", who);
  if (d->dtype > GSR_BF16) return fail(ctx, GSR_EINVAL, "%s: unknown dtype %u", who, d->dtype);
  if (d->kv_heads == 0 || d->heads == 0 || d->heads % d->kv_heads)
    return fail(ctx, GSR_EINVAL, "%s: %u heads are not a multiple of %u key heads", who, d->heads, d->kv_heads);
  if (d->head_dim < 1 || d->head_dim > GSR_ATTENTION_MAX_DIM)
    return fail(ctx, GSR_EINVAL, "%s: head_dim %u, 1 to %d are supported", who, d->head_dim, GSR_ATTENTION_MAX_DIM);
  if (!(d->scale > 0.0f) || std::isinf(d->scale))
    return fail(ctx, GSR_EINVAL, "%s: scale must be finite and > 0", who);
  const uint64_t lim = uint64_t(1) << 31;
  if (d->heads >= (1u << 16) || d->batch >= (1u << 24) || uint64_t(d->batch) * d->heads >= lim ||
      uint64_t(d->batch) * d->heads * d->queries >= lim || uint64_t(d->batch) * d->kv_heads * d->keys >= lim)
    return fail(ctx, GSR_EOVERFLOW, "%s: batch * heads * queries or batch * kv_heads * keys >= 2^31", who);
  if (d->batch && d->queries && (!q || !o)) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  if (d->batch && d->keys && (!k || !v)) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  const size_t eb = elem_bytes(d->dtype);
  if (misaligned(q, eb) || misaligned(k, eb) || misaligned(v, eb) || misaligned(o, eb) || misaligned(kv_lengths, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  *a = AttnArgs{};
  a->q = q;
  a->k = k;
  a->v = v;
  a->kv_len = kv_lengths;
  a->mask = mask;
  a->batch = d->batch;
  a->heads = d->heads;
  a->kv_heads = d->kv_heads;
  a->queries = d->queries;
  a->keys = d->keys;
  a->dim = d->head_dim;
  a->scale = d->scale;
  a->share.set(d->heads / d->kv_heads);
  a->rows = d->queries * (d->heads / d->kv_heads);
  for (int i = 0; i < 3; ++i) {
    a->qs[i] = d->q_stride[i];
    a->ks[i] = d->k_stride[i];
    a->vs[i] = d->v_stride[i];
    a->os[i] = d->o_stride[i];
    a->ms[i] = d->mask_stride[i];
    a->dos[i] = d->do_stride[i];
    a->dqs[i] = d->dq_stride[i];
    a->dks[i] = d->dk_stride[i];
    a->dvs[i] = d->dv_stride[i];
  }
  return GSR_OK;
}

}  // namespace gsr

using namespace gsr;

extern "C" gsr_status gsr_cross_attention_forward(gsr_ctx* ctx, void* stream, const gsr_attention* d, const void* q,
                                                  const void* k, const void* v, const int32_t* kv_lengths,
                                                  const uint8_t* mask, void* o, float* lse) {
  static const char* who = "gsr_cross_attention_forward";
  if (!ctx) return GSR_EINVAL;
  AttnArgs a;
  gsr_status st = attention_args(ctx, d, q, k, v, kv_lengths, mask, o, who, &a);
  if (st) return st;
  if (misaligned(lse, 4)) return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!distinct({{d->o_stride[0], d->batch}, {d->o_stride[1], d->queries}, {d->o_stride[2], d->heads}}, d->head_dim))
    return fail(ctx, GSR_EINVAL, "%s: the strides of o overlap", who);
  if (!d->batch || !d->queries) return GSR_OK;
  if ((st = enter(ctx))) return st;
  a.out = o;
  a.lse = lse;
  const uint32_t key_tile = d->dtype == GSR_F32 ? 32 : 64;
  const dim3 grid = attention_grid(&a, (a.rows + kAttnRows - 1) / kAttnRows,
                                   (uint64_t(a.keys) + key_tile - 1) / key_tile, 1024);
  if (a.splits > 1) {
    const size_t parts = size_t(a.batch) * a.kv_heads * a.splits * a.rows;
    if ((st = grow(ctx, ctx->arena.feat_part, parts * (a.dim + 2) * sizeof(float)))) return st;
    a.part_ml = static_cast<float*>(ctx->arena.feat_part.ptr);
    a.part = a.part_ml + parts * 2;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_ATTENTION_FORWARD, s, false);
  attention_by_kind(d->dtype, a.dim, mask != nullptr && a.keys, [&](auto t, auto dp, auto masked) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_attn_fwd<T, decltype(dp)::value, decltype(masked)::value>), grid, dim3(kAttnThreads), 0, s,
                       a);
    if (a.splits > 1) {
      const uint64_t n = uint64_t(a.batch) * a.kv_heads * a.rows * a.dim;
      hipLaunchKernelGGL((k_attn_join<T>), dim3(uint32_t((n + kAttnThreads - 1) / kAttnThreads)), dim3(kAttnThreads),
                         0, s, a);
    }
  });
  timing_mark(ctx, GSR_STAGE_ATTENTION_FORWARD, s, true);
  return check_launch(ctx, who);
}
