// Cross attention, backward, from the forward's o and lse: p = exp(s - lse), ds = scale p (do.v - do.o),
//   dq = ds k,  dk = ds^T q,  dv = p^T do.
//
// Two kernels, each owning what it writes, so that no sum depends on the order of atomics: k_attn_dq streams keys past
// the rows of a workgroup (three products a block, and do.o of its rows, which the second kernel reads), k_attn_dkv
// streams rows past the keys of a workgroup (four products). Recomputing the scores and do.v in both costs seven
// products instead of five. The rows of one key head are the queries of every head that shares it, so the sums of a
// shared key's gradient need no join. Where rows or keys are few, the streamed side is split over workgroups and
// k_attn_add adds the parts in order.
#include <type_traits>

#include "attention_common.hpp"

namespace gsr {
namespace {

// float16 values of ds, whose size follows the loss's scale, are kept in range by a power of two per column of the
// accumulator (a query's dq, a key's dk): set from the first block that has a value, lowered when a later block would
// overflow. Other types need none.
template <typename T, int DP>
struct Ranged {
  float f = 0.0f;  // 0: nothing seen yet
  static constexpr bool kOn = std::is_same_v<T, _Float16>;

  __device__ __forceinline__ void fit(f32x16& ds, f32x16* acc) {
    if constexpr (kOn) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(ds[i]));
      top = fmaxf(top, other_half(top));
      const bool change = f == 0.0f ? top > 0.0f : top * f > 32768.0f;
      if (__any(change)) {
        const float f_new = change ? ldexpf(1.0f, min(max(9 - __builtin_amdgcn_frexp_expf(top), -100), 100)) : f;
        const float ratio = change && f != 0.0f ? f_new / f : 1.0f;
        f = f_new;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[dt][i] *= ratio;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] *= f;
    }
  }
  __device__ __forceinline__ float undo() const { return kOn ? (f == 0.0f ? 0.0f : 1.0f / f) : 1.0f; }
};

template <typename T, int DP, bool kMask>
__global__ __launch_bounds__(kAttnThreads) void k_attn_dq(AttnArgs a) {
  using L = Tile<T, DP>;
  constexpr int KT = 32, kLoads = (KT * L::kChunks + kAttnThreads - 1) / kAttnThreads;
  __shared__ __attribute__((aligned(16))) char s_k[KT * L::kRowBytes];
  __shared__ __attribute__((aligned(16))) char s_v[KT * L::kRowBytes];
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, dim = int(a.dim);
  const uint32_t row = w.tile * kAttnRows + (tid >> 6) * 32 + (lane & 31);
  const bool valid = row < a.rows;
  const bool active = w.tile * kAttnRows + (tid >> 6) * 32 < a.rows;
  uint32_t query = 0, head = 0;
  if (valid) row_of(a, w.kv_head, row, &query, &head);
  Vec<T, 8> qf[DP / 16], df[DP / 16];
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) qf[kk] = df[kk] = zero_frag<T>();
  // a row that saw no key (lse = -inf) has p = 0 everywhere; whatever its gradient holds is not looked at
  float lse2 = INFINITY, delta = 0.0f;
  if (valid) {
    const int64_t at = (int64_t(w.batch) * a.heads + head) * a.queries + query;
    const float lse = a.lse[at];
    if (lse != -INFINITY) {
      lse2 = lse * kLog2e;
      const T* qr = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + int64_t(query) * a.qs[1] +
                    int64_t(head) * a.qs[2];
      const T* dr = static_cast<const T*>(a.dout) + int64_t(w.batch) * a.dos[0] + int64_t(query) * a.dos[1] +
                    int64_t(head) * a.dos[2];
      const T* orow = static_cast<const T*>(a.o) + int64_t(w.batch) * a.os[0] + int64_t(query) * a.os[1] +
                      int64_t(head) * a.os[2];
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        qf[kk] = load_frag(qr, kk, dim);
        df[kk] = load_frag(dr, kk, dim);
        const Vec<T, 8> of = load_frag(orow, kk, dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta = fmaf(float(df[kk][j]), float(of[j]), delta);
      }
    }
  }
  delta += other_half(delta);
  if (valid && h == 0 && w.split == 0) a.delta[(int64_t(w.batch) * a.heads + head) * a.queries + query] = delta;
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

  const float c = a.scale * kLog2e, delta_s = delta * a.scale;
  f32x16 acc[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = f32x16{};
  Ranged<T, DP> range;
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
      if constexpr (kMask) odd |= any_nonfinite<T>(rk[i]);
    }
    if constexpr (kMask)
      odd = __syncthreads_or(odd);
    else
      __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    if (active) {
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) s = mma(L::frag(s_k, 0, kk), qf[kk], s);
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) dp = mma(L::frag(s_v, 0, kk), df[kk], dp);
      uint32_t seen = 0;
      const bool some = kMask || (t + 1) * KT > len;
      if (some) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t key = t * KT + 8 * g + 4 * h;
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
            seen |= uint32_t(vis) << (4 * g + i);
            s[4 * g + i] = vis ? s[4 * g + i] : -INFINITY;
            dp[4 * g + i] = vis ? dp[4 * g + i] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = exp2_fast(fmaf(s[i], c, -lse2)) * fmaf(dp[i], a.scale, -delta_s);
      range.fit(s, acc);
      contract<T, DP>(acc, s_k, 0, s, kMask && odd, seen);
    }
    __syncthreads();
  }
  if (!valid) return;
  if (a.splits > 1) {
    const int64_t at = (int64_t(w.batch * a.kv_heads + w.kv_head) * a.splits + w.split) * a.rows + row;
    store_column<float, DP>(a.part + at * dim, acc, range.undo(), dim);
    return;
  }
  T* out = static_cast<T*>(a.dq) + int64_t(w.batch) * a.dqs[0] + int64_t(query) * a.dqs[1] +
           int64_t(head) * a.dqs[2];
  store_column<T, DP>(out, acc, range.undo(), dim);
}

template <typename T, int DP, bool kMask>
__global__ __launch_bounds__(kAttnThreads) void k_attn_dkv(AttnArgs a) {
  using L = Tile<T, DP>;
  constexpr int QT = 32, kLoads = (QT * L::kChunks + kAttnThreads - 1) / kAttnThreads;
  __shared__ __attribute__((aligned(16))) char s_q[QT * L::kRowBytes];
  __shared__ __attribute__((aligned(16))) char s_d[QT * L::kRowBytes];
  __shared__ __attribute__((aligned(16))) float s_lse[QT];
  __shared__ __attribute__((aligned(16))) float s_delta[QT];
  __shared__ int64_t s_mask[QT];
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, dim = int(a.dim);
  const uint32_t key = w.tile * kAttnRows + (tid >> 6) * 32 + (lane & 31);
  const uint32_t len = keys_of(a, w.batch);
  const bool valid = key < len;
  const bool active = w.tile * kAttnRows + (tid >> 6) * 32 < len;
  Vec<T, 8> kf[DP / 16], vf[DP / 16];
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) kf[kk] = vf[kk] = zero_frag<T>();
  if (valid) {
    const T* kr = static_cast<const T*>(a.k) + int64_t(w.batch) * a.ks[0] + int64_t(key) * a.ks[1] +
                  int64_t(w.kv_head) * a.ks[2];
    const T* vr = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(key) * a.vs[1] +
                  int64_t(w.kv_head) * a.vs[2];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      kf[kk] = load_frag(kr, kk, dim);
      vf[kk] = load_frag(vr, kk, dim);
    }
  }
  const uint32_t tiles = w.tile * kAttnRows < len ? (a.rows + QT - 1) / QT : 0;  // no visible key: nothing to sum
  const uint32_t t0 = uint32_t(uint64_t(tiles) * w.split / a.splits);
  const uint32_t t1 = uint32_t(uint64_t(tiles) * (w.split + 1) / a.splits);
  const T* qb = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0];
  const T* db = static_cast<const T*>(a.dout) + int64_t(w.batch) * a.dos[0];
  const int64_t stat0 = int64_t(w.batch) * a.heads * a.queries;

  // A streamed row that saw no key is taken as zeros, whatever it holds (its lse2 of +inf makes p = 0).
  u32x4 rq[kLoads], rd[kLoads];
  float lse2 = INFINITY, delta = 0.0f;
  int64_t mask_at = 0;
  auto fetch = [&](uint32_t t) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kAttnThreads, r = e / L::kChunks, c = e % L::kChunks * L::kPer;
      const uint32_t row = t * QT + r;
      rq[i] = rd[i] = u32x4{0, 0, 0, 0};
      if (row < a.rows && c < dim && r < QT) {
        uint32_t query, head;
        row_of(a, w.kv_head, row, &query, &head);
        if (a.lse[stat0 + int64_t(head) * a.queries + query] != -INFINITY) {
          rq[i] = load_chunk(qb + int64_t(query) * a.qs[1] + int64_t(head) * a.qs[2], c, dim);
          rd[i] = load_chunk(db + int64_t(query) * a.dos[1] + int64_t(head) * a.dos[2], c, dim);
        }
      }
    }
    if (tid < QT) {
      lse2 = INFINITY;
      delta = 0.0f;
      mask_at = 0;
      const uint32_t row = t * QT + tid;
      if (row < a.rows) {
        uint32_t query, head;
        row_of(a, w.kv_head, row, &query, &head);
        const float lse = a.lse[stat0 + int64_t(head) * a.queries + query];
        if (lse != -INFINITY) {
          lse2 = lse * kLog2e;
          delta = a.delta[stat0 + int64_t(head) * a.queries + query] * a.scale;
        }
        if constexpr (kMask) mask_at = int64_t(head) * a.ms[1] + int64_t(query) * a.ms[2];
      }
    }
  };

  constexpr float kDown = std::is_same_v<T, _Float16> ? 1.0f / 16384.0f : 1.0f;  // undoes kLift
  const float c = a.scale * kLog2e;
  const uint8_t* mask = kMask ? a.mask + int64_t(w.batch) * a.ms[0] + key : nullptr;
  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) dk[dt] = dv[dt] = f32x16{};
  Ranged<T, DP> range;
  if (t0 < t1) fetch(t0);
  for (uint32_t t = t0; t < t1; ++t) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kAttnThreads, r = e / L::kChunks;
      if (r < QT) {
        *reinterpret_cast<u32x4*>(s_q + L::at(r, e % L::kChunks)) = rq[i];
        *reinterpret_cast<u32x4*>(s_d + L::at(r, e % L::kChunks)) = rd[i];
      }
      if constexpr (kMask) odd |= any_nonfinite<T>(rq[i]) || any_nonfinite<T>(rd[i]);
    }
    if (tid < QT) {
      s_lse[tid] = lse2;
      s_delta[tid] = delta;
      if constexpr (kMask) s_mask[tid] = mask_at;
    }
    if constexpr (kMask)
      odd = __syncthreads_or(odd);
    else
      __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    if (active) {
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) s = mma(L::frag(s_q, 0, kk), kf[kk], s);
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) dp = mma(L::frag(s_d, 0, kk), vf[kk], dp);
      uint32_t seen = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const Vec<float, 4> ls = *reinterpret_cast<const Vec<float, 4>*>(s_lse + 8 * g + 4 * h);
        const Vec<float, 4> dl = *reinterpret_cast<const Vec<float, 4>*>(s_delta + 8 * g + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * g + i;
          bool vis = valid;
          if constexpr (kMask) {
            const uint32_t row = t * QT + 8 * g + 4 * h + i;
            if (valid && row < a.rows) vis = mask[s_mask[8 * g + 4 * h + i]] != 0;
            vis = vis && ls[i] != INFINITY;
            seen |= uint32_t(vis) << e;
          }
          const float p = vis ? exp2_fast(fmaf(s[e], c, kLift<T> - ls[i])) : 0.0f;
          s[e] = p;
          dp[e] = vis ? p * (fmaf(dp[e], a.scale, -dl[i]) * kDown) : 0.0f;
        }
      }
      contract<T, DP>(dv, s_d, 0, s, kMask && odd, seen);
      range.fit(dp, dk);
      contract<T, DP>(dk, s_q, 0, dp, kMask && odd, seen);
    }
    __syncthreads();
  }
  if (key >= a.keys) return;
  if (a.splits > 1) {
    const int64_t group = int64_t(w.batch) * a.kv_heads + w.kv_head, all = int64_t(a.batch) * a.kv_heads;
    const int64_t at = (group * a.splits + w.split) * a.keys + key;
    store_column<float, DP>(a.part + at * dim, dk, range.undo(), dim);
    store_column<float, DP>(a.part + (all * a.splits * a.keys + at) * dim, dv, kDown, dim);
    return;
  }
  T* ok = static_cast<T*>(a.dk) + int64_t(w.batch) * a.dks[0] + int64_t(key) * a.dks[1] + int64_t(w.kv_head) * a.dks[2];
  T* ov = static_cast<T*>(a.dv) + int64_t(w.batch) * a.dvs[0] + int64_t(key) * a.dvs[1] + int64_t(w.kv_head) * a.dvs[2];
  store_column<T, DP>(ok, dk, range.undo(), dim);
  store_column<T, DP>(ov, dv, kDown, dim);
}

// Adds the parts of split rows: a thread per (row, element). blockIdx.y = 1 adds dv after dk.
template <typename T, bool kKeys>
__global__ __launch_bounds__(kAttnThreads) void k_attn_add(AttnArgs a) {
  const uint64_t id = uint64_t(blockIdx.x) * kAttnThreads + threadIdx.x;
  const uint32_t per = kKeys ? a.keys : a.rows;
  const uint64_t rows = uint64_t(a.batch) * a.kv_heads * per;
  if (id >= rows * a.dim) return;
  const uint32_t d = uint32_t(id % a.dim);
  const uint64_t at = id / a.dim, group = at / per;
  const uint32_t row = uint32_t(at % per), kv_head = uint32_t(group % a.kv_heads), b = uint32_t(group / a.kv_heads);
  const float* part = a.part + (group * a.splits * per + row) * a.dim + d;
  if (kKeys && blockIdx.y) part += rows * a.splits * a.dim;
  float v = 0.0f;
  for (uint32_t s = 0; s < a.splits; ++s) v += part[uint64_t(s) * per * a.dim];
  if constexpr (kKeys) {
    const int64_t* st = blockIdx.y ? a.dvs : a.dks;
    T* out = static_cast<T*>(blockIdx.y ? a.dv : a.dk);
    out[int64_t(b) * st[0] + int64_t(row) * st[1] + int64_t(kv_head) * st[2] + d] = T(v);
  } else {
    uint32_t query, head;
    row_of(a, kv_head, row, &query, &head);
    static_cast<T*>(a.dq)[int64_t(b) * a.dqs[0] + int64_t(query) * a.dqs[1] + int64_t(head) * a.dqs[2] + d] = T(v);
  }
}

}  // namespace
}  // namespace gsr

using namespace gsr;

extern "C" gsr_status gsr_cross_attention_backward(gsr_ctx* ctx, void* stream, const gsr_attention* d, const void* q,
                                                   const void* k, const void* v, const int32_t* kv_lengths,
                                                   const uint8_t* mask, const void* o, const float* lse,
                                                   const void* dout, void* dq, void* dk, void* dv) {
  static const char* who = "gsr_cross_attention_backward";
  if (!ctx) return GSR_EINVAL;
  AttnArgs a;
  gsr_status st = attention_args(ctx, d, q, k, v, kv_lengths, mask, o, who, &a);
  if (st) return st;
  const size_t eb = elem_bytes(d->dtype);
  const bool has_q = d->batch && d->queries, has_k = d->batch && d->keys;
  if ((has_q && (!lse || !dout || !dq)) || (has_k && (!dk || !dv)))
    return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  if (misaligned(lse, 4) || misaligned(dout, eb) || misaligned(dq, eb) || misaligned(dk, eb) || misaligned(dv, eb))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!distinct({{d->dq_stride[0], d->batch}, {d->dq_stride[1], d->queries}, {d->dq_stride[2], d->heads}},
                d->head_dim))
    return fail(ctx, GSR_EINVAL, "%s: the strides of dq overlap", who);
  if (!distinct({{d->dk_stride[0], d->batch}, {d->dk_stride[1], d->keys}, {d->dk_stride[2], d->kv_heads}},
                d->head_dim) ||
      !distinct({{d->dv_stride[0], d->batch}, {d->dv_stride[1], d->keys}, {d->dv_stride[2], d->kv_heads}},
                d->head_dim))
    return fail(ctx, GSR_EINVAL, "%s: the strides of dk or dv overlap", who);
  if (!has_q && !has_k) return GSR_OK;
  if ((st = enter(ctx))) return st;
  a.o = o;
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  // one scratch buffer: do.o of every row, then the parts of whichever kernel splits (one after the other)
  AttnArgs b = a;
  const dim3 grid_q = attention_grid(&a, (a.rows + kAttnRows - 1) / kAttnRows, (uint64_t(a.keys) + 31) / 32, 512);
  const dim3 grid_k = attention_grid(&b, (b.keys + kAttnRows - 1) / kAttnRows, (uint64_t(b.rows) + 31) / 32, 512);
  const size_t groups = size_t(a.batch) * a.kv_heads, deltas = (groups * a.rows + 3) / 4 * 4;
  size_t parts = 0;
  if (a.splits > 1) parts = groups * a.splits * a.rows * a.dim;
  if (b.splits > 1) parts = std::max(parts, 2 * groups * b.splits * b.keys * b.dim);
  if ((st = grow(ctx, ctx->arena.feat_part, (deltas + parts) * sizeof(float)))) return st;
  a.delta = b.delta = static_cast<float*>(ctx->arena.feat_part.ptr);
  a.part = b.part = a.delta + deltas;
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_ATTENTION_BACKWARD, s, false);
  attention_by_kind(d->dtype, a.dim, mask != nullptr && a.keys, [&](auto t, auto dp, auto masked) {
    using T = decltype(t);
    constexpr int DP = decltype(dp)::value;
    constexpr bool kMask = decltype(masked)::value;
    const dim3 block(kAttnThreads);
    auto blocks = [&](uint64_t n) { return uint32_t((n + kAttnThreads - 1) / kAttnThreads); };
    if (has_q) {
      hipLaunchKernelGGL((k_attn_dq<T, DP, kMask>), grid_q, block, 0, s, a);
      if (a.splits > 1) hipLaunchKernelGGL((k_attn_add<T, false>), dim3(blocks(groups * a.rows * a.dim)), block, 0, s, a);
    }
    if (has_k) {
      hipLaunchKernelGGL((k_attn_dkv<T, DP, kMask>), grid_k, block, 0, s, b);
      if (b.splits > 1)
        hipLaunchKernelGGL((k_attn_add<T, true>), dim3(blocks(groups * b.keys * b.dim), 2), block, 0, s, b);
    }
  });
  timing_mark(ctx, GSR_STAGE_ATTENTION_BACKWARD, s, true);
  return check_launch(ctx, who);
}
