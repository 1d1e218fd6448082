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

// Wide 16-bit heads: a wave's two operands (its rows' q and do, or its keys' k and v), the sums and two blocks of
// scores pass 256 registers, and a wave alone on its SIMD waits out every LDS read. There one of the two operands is kept
// in LDS, the stream goes by 32 rows through two buffers, and two waves share a SIMD. Both kernels of a bfloat16 training
// step of 2,500 x 2,500, 8 heads, with its forward pass: 96 wide 448 -> 342 us (of it 364 by the keys' kernel alone),
// 128 wide 516 -> 484 us by the keys' kernel. The queries' kernel keeps ds to twice the bits and at 128 wide still spills
// (484 -> 824 us), so it stays at one wave there. (Measured while dk rounded its ds once: 354 and 487 us today.)
template <typename T, int DK, bool kMask>
constexpr bool kOneInLds = sizeof(T) == 2 && DK == 96 && !kMask;
template <typename T, int DK, bool kMask>
constexpr bool kOneInLdsKeys = sizeof(T) == 2 && DK > 64 && !kMask;
// Waves that share a SIMD, so that one multiplies while another computes exponentials: two where 256 registers hold a
// wave's operands and sums, or all but a few of them. 16 bits at 64 wide spill 2 to 15 registers of the queries' kernel,
// 96 wide 13 to 24, the keys' kernel at 128 wide 10 to 31, and two waves are faster all the same (training steps of
// 2,500 x 2,500, 8 heads, bfloat16: 237 against 266 us, 353 against 395, 486 against 515); so is float32 at 48 wide
// (1,300 x 1,369: 355 against 361), but not at 64 wide (16 to 35 spilled: 431 against 427, with a mask 550 against 533).
template <typename T, int DK, bool kMask>
constexpr int kWavesPerSimd = DK <= (sizeof(T) == 2 ? 64 : 48) || kOneInLds<T, DK, kMask> ? 2 : 1;
template <typename T, int DK, bool kMask>
constexpr int kWavesPerSimdKeys =
    sizeof(T) == 2 ? (DK <= 64 || kOneInLdsKeys<T, DK, kMask> ? 2 : 1) : (DK <= 32 || (DK <= 48 && !kMask) ? 2 : 1);
// 32-row blocks of a streamed tile: two halve the barriers and give the matrix cores one block's products while the
// other's exponentials are taken.
template <typename T, bool kMask, bool kOne>
constexpr int kStreamBlocks = sizeof(T) == 2 && !kMask && !kOne ? 2 : 1;

// float16 values of ds, whose size follows the loss's scale, are kept in range by a power of two per column of the
// accumulator (a query's dq, a key's dk): set from the first block that has a value, lowered when a later block would
// overflow. Other types need none.
template <typename T, int DK>
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
        for (int dt = 0; dt < Tile<T, DK>::kOut; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[dt][i] *= ratio;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] *= f;
    }
  }
  __device__ __forceinline__ float undo() const { return kOn ? (f == 0.0f ? 0.0f : 1.0f / f) : 1.0f; }
};

// dq of the workgroup's rows. 2 x 2,500 x 2,500, 8 heads, 128 wide, bfloat16: 185 us, 415 TFLOP/s of its three
// products (553 with the second one of ds); 777 x 1,369, 6 heads on 2, 48 wide, masked, float32: 69 us. Bound by LDS
// latency with one wave on a SIMD at 128 wide (the matrix cores busy 24 %), by issue below; float32 by its products,
// which the vector units do not overlap.
template <typename T, int DK, bool kMask>
__global__ __launch_bounds__(kAttnThreads, (kWavesPerSimd<T, DK, kMask>)) void k_attn_dq(AttnArgs a) {
  using L = Tile<T, DK>;
  constexpr bool kOwn = kOneInLds<T, DK, kMask>;
  constexpr int kBlocks = kStreamBlocks<T, kMask, kOwn>, KT = 32 * kBlocks, kTile = KT * L::kRowBytes;
  constexpr int kRing = kOwn ? 2 : 3;  // tiles in LDS: the one multiplied and those on their way
  __shared__ __attribute__((aligned(16))) char s_tile[2 * kRing * kTile];
  __shared__ __attribute__((aligned(16))) char s_own[kOwn ? kAttnRows * L::kRowBytes : 16];
  __shared__ BadBits<T, DK, kMask ? KT : 1> s_bad;
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, dim = int(a.dim), dim_in = int(a.dim_in);
  const uint32_t row0 = w.tile * kAttnRows + (tid >> 6) * 32, row = row0 + (lane & 31);
  const bool valid = row < a.rows;
  uint32_t query = 0, head = 0;
  if (valid) row_of(a, w.kv_head, row, &query, &head);
  const int64_t stat = (int64_t(w.batch) * a.heads + head) * a.queries + query;
  const uint8_t* mask = nullptr;
  if (kMask && valid)
    mask = a.mask + int64_t(w.batch) * a.ms[0] + int64_t(head) * a.ms[1] + int64_t(query) * a.ms[2];
  const uint32_t len = keys_of(a, w.batch), tiles = (len + KT - 1) / KT;
  const uint32_t t0 = uint32_t(uint64_t(tiles) * w.split / a.splits);
  const uint32_t t1 = uint32_t(uint64_t(tiles) * (w.split + 1) / a.splits);
  const T* kb = static_cast<const T*>(a.k) + int64_t(w.batch) * a.ks[0] + int64_t(w.kv_head) * a.ks[2];
  const T* vb = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(w.kv_head) * a.vs[2];
  using Copy = Copier<T, DK, KT>;
  auto start = [&](uint32_t t, char* s) {
    const uint32_t key0 = t * KT;
    Copy::start(s, len - key0, dim_in, [&](int r) { return kb + int64_t(key0 + r) * a.ks[1]; });
    Copy::start(s + kTile, len - key0, dim_in, [&](int r) { return vb + int64_t(key0 + r) * a.vs[1]; });
  };

  if constexpr (kMask) s_bad.clear();
  clear_tiles<T, DK>(s_tile, 2 * kRing * kTile, dim_in);
  if constexpr (kOwn) clear_tiles<T, DK>(s_own, kAttnRows * L::kRowBytes, dim_in);
  __syncthreads();
  if (t0 < t1) start(t0, s_tile);
  if (kRing == 3 && t0 + 1 < t1) start(t0 + 1, s_tile + 2 * kTile);
  if (kOwn && t0 < t1) {
    const T* db = static_cast<const T*>(a.dout) + int64_t(w.batch) * a.dos[0];
    Copier<T, DK, kAttnRows>::start(s_own, a.rows - w.tile * kAttnRows, dim_in, [&](int r) {
      uint32_t t, hd;
      row_of(a, w.kv_head, w.tile * kAttnRows + r, &t, &hd);
      return db + int64_t(t) * a.dos[1] + int64_t(hd) * a.dos[2];
    });
  }
  Vec<T, 8> qf[DK / 16], df[DK / 16];
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk) qf[kk] = df[kk] = zero_frag<T>();
  // a row that saw no key (lse = -inf) has p = 0 everywhere; whatever its gradient holds counts as zeros
  float lse2 = INFINITY, delta = 0.0f;
  if (valid) {
    const float lse = a.lse[stat];
    const T* qr = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + int64_t(query) * a.qs[1] +
                  int64_t(head) * a.qs[2];
    const T* dr = static_cast<const T*>(a.dout) + int64_t(w.batch) * a.dos[0] + int64_t(query) * a.dos[1] +
                  int64_t(head) * a.dos[2];
    const T* orow = static_cast<const T*>(a.o) + int64_t(w.batch) * a.os[0] + int64_t(query) * a.os[1] +
                    int64_t(head) * a.os[2];
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) {
      qf[kk] = load_frag(qr, kk, dim_in);
      df[kk] = load_frag(dr, kk, dim_in);
      const Vec<T, 8> of = load_frag(orow, kk, dim_in);
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = fmaf(float(df[kk][j]), float(of[j]), delta);
    }
    // p carries the rounding of lse: 2^-24 |lse| of a whole row. In float32 that leaves dv at 1.7 times the error of a
    // form that keeps its probabilities where |lse| is 116, at 4 times (1.3e-5) where it is 464, and dk and dv at
    // twice (7e-7) on 10,000 nearly equal keys; dq and dk differ by less.
    if (lse != -INFINITY) {
      lse2 = lse * kLog2e;
    } else {
      delta = 0.0f;
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) qf[kk] = df[kk] = zero_frag<T>();
    }
  }
  delta += other_half(delta);
  if (valid && h == 0 && w.split == 0) a.delta[stat] = delta;
  const float c = a.scale * kLog2e, delta_s = delta * a.scale;
  f32x16 acc[L::kOut];
#pragma unroll
  for (int dt = 0; dt < L::kOut; ++dt) acc[dt] = f32x16{};
  Ranged<T, DK> range;
  uint32_t words[kBlocks][4], seen[kBlocks] = {};  // the mask of the tile that comes next; what this one shows
  auto multiply = [&](uint32_t t, const char* s_k, const char* s_v, bool odd, auto edge) {
    f32x16 s[kBlocks], dp[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      s[b] = dp[b] = f32x16{};
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) s[b] = mma(L::frag(s_k, 32 * b, kk), qf[kk], s[b]);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk)
        dp[b] = mma(L::frag(s_v, 32 * b, kk), kOwn ? L::frag(s_own, (tid >> 6) * 32, kk) : df[kk], dp[b]);
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      auto key_element = [&](int r, int d) { return kb[int64_t(t * KT + r) * a.ks[1] + d]; };
      if constexpr (kMask) {
        if (odd) {
          const T* qr = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + int64_t(keep_here(query)) * a.qs[1] +
                        int64_t(keep_here(head)) * a.qs[2];
          add_products<T, DK, KT>(s[b], seen[b], 32 * b, t - t0, s_bad, key_element, [&](int d) { return qr[d]; });
        }
      }
      if constexpr (kMask || decltype(edge)::value) {
        if constexpr (!kMask) seen[b] = visible<false>(nullptr, t * KT + 32 * b, len);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[b][i] = (seen[b] >> i) & 1 ? s[b][i] : -INFINITY;
          dp[b][i] = (seen[b] >> i) & 1 ? dp[b][i] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[b][i] = exp2_fast(fmaf(s[b][i], c, -lse2)) * fmaf(dp[b][i], a.scale, -delta_s);
      range.fit(s[b], acc);
      // ds is kept to twice the bits: rounded once, it and the o in do.o together leave dq and dk over 1.5 times the
      // error of their own rounding (now 1.0 to 1.2); that costs 4 % of a training step for dq and 5 % for dk
      // (2,500 x 2,500, 8 heads, 128 wide, bfloat16: 484 -> 511 us). p is rounded once: dv stays below 1.48 times.
      contract<T, DK, (sizeof(T) == 2)>(acc, s_k, 32 * b, s[b]);
      if constexpr (kMask) {
        if (odd) add_outputs<T, DK, KT>(acc, s[b], seen[b], 32 * b, t - t0, s_bad, key_element);
      }
    }
  };
  if (kMask && t0 < t1) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) mask_words(mask, t0 * KT + 32 * b, len, words[b]);
  }
  int buf = 0;
  for (uint32_t t = t0; t < t1; ++t) {
    char *s_k = s_tile + buf * 2 * kTile, *s_v = s_k + kTile;
    if (kRing == 3 && t + 1 < t1 && (t + 2) * KT <= len)
      tile_barrier<2 * Copy::kSteps>();
    else
      tile_barrier<0>();
    if constexpr (kMask) {  // before the copies start, so that waiting for these loads does not wait for those
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        seen[b] = visible<true>(words[b], 0, 0);
        mask_words(t + 1 < t1 ? mask : nullptr, (t + 1) * KT + 32 * b, len, words[b]);
      }
    }
    if (t + kRing - 1 < t1) start(t + kRing - 1, s_tile + (buf == 0 ? kRing - 1 : buf - 1) * 2 * kTile);
    bool odd = false;
    if constexpr (kMask)
      odd = tile_make_finite<T, DK, KT>(s_k, t - t0, s_bad, [](int) { return true; });
    if (row0 < a.rows) {
      if ((t + 1) * KT <= len)
        multiply(t, s_k, s_v, odd, std::false_type());
      else
        multiply(t, s_k, s_v, odd, std::true_type());
    }
    buf = buf == kRing - 1 ? 0 : buf + 1;
  }
  if (!valid) return;
  if (a.splits > 1) {
    const int64_t part = (int64_t(w.batch * a.kv_heads + w.kv_head) * a.splits + w.split) * a.rows + row;
    store_column<L::kOut>(a.part + part * dim, acc, range.undo(), dim);
    return;
  }
  T* out = static_cast<T*>(a.dq) + int64_t(w.batch) * a.dqs[0] + int64_t(query) * a.dqs[1] +
           int64_t(head) * a.dqs[2];
  store_column<L::kOut>(out, acc, range.undo(), dim);
}

// dk and dv of the workgroup's keys, at the same sizes: 190 us, 539 TFLOP/s of its four products (674 with the second
// one of ds), the matrix cores busy 30 %; float32 105 us. Bound by LDS: every operand of a streamed tile is read by
// row and once more transposed.
template <typename T, int DK, bool kMask>
__global__ __launch_bounds__(kAttnThreads, (kWavesPerSimdKeys<T, DK, kMask>)) void k_attn_dkv(AttnArgs a) {
  using L = Tile<T, DK>;
  constexpr bool kOwn = kOneInLdsKeys<T, DK, kMask>;
  constexpr int kBlocks = kStreamBlocks<T, kMask, kOwn>, QT = 32 * kBlocks, kTile = QT * L::kRowBytes;
  constexpr int kRing = kOwn ? 2 : 3;  // tiles in LDS: the one multiplied and those on their way
  __shared__ __attribute__((aligned(16))) char s_tile[2 * kRing * kTile];
  __shared__ __attribute__((aligned(16))) char s_own[kOwn ? kAttnRows * L::kRowBytes : 16];
  __shared__ __attribute__((aligned(16))) float s_lse[3][QT];
  __shared__ __attribute__((aligned(16))) float s_delta[3][QT];
  __shared__ int64_t s_mask[3][kMask ? QT : 1];
  __shared__ BadBits<T, DK, kMask ? 2 * QT : 1> s_bad;
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, dim = int(a.dim), dim_in = int(a.dim_in);
  const uint32_t key0 = w.tile * kAttnRows + (tid >> 6) * 32, key = key0 + (lane & 31);
  const uint32_t len = keys_of(a, w.batch);
  const bool valid = key < len;
  const uint32_t tiles = w.tile * kAttnRows < len ? (a.rows + QT - 1) / QT : 0;  // no visible key: nothing to sum
  const uint32_t t0 = uint32_t(uint64_t(tiles) * w.split / a.splits);
  const uint32_t t1 = uint32_t(uint64_t(tiles) * (w.split + 1) / a.splits);
  // with one query head to a key head, the rows are the queries, a constant stride apart
  const bool plain = a.share.d == 1;
  const int64_t stat0 = int64_t(w.batch) * a.heads * a.queries;
  const T* qb = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + (plain ? int64_t(w.kv_head) * a.qs[2] : 0);
  const T* db = static_cast<const T*>(a.dout) + int64_t(w.batch) * a.dos[0] +
                (plain ? int64_t(w.kv_head) * a.dos[2] : 0);
  using Copy = Copier<T, DK, QT>;
  float lse = -INFINITY, delta = 0.0f;  // of row tid of the newest tile (the first QT threads)
  int64_t mask_at = 0;
  auto start = [&](uint32_t t, char* s) {
    const uint32_t row0 = t * QT;
    if (tid < QT) {
      lse = -INFINITY;
      delta = 0.0f;
      if (row0 + tid < a.rows) {
        uint32_t query, head;
        row_of(a, w.kv_head, row0 + tid, &query, &head);
        const int64_t at = stat0 + int64_t(head) * a.queries + query;
        lse = a.lse[at];
        delta = a.delta[at];
        if constexpr (kMask) mask_at = int64_t(head) * a.ms[1] + int64_t(query) * a.ms[2];
      }
    }
    // past the last row, q's is repeated, not made zeros: a key's infinity times 0 would be NaN, and its score has to be
    // what p = 0 leaves alone (do is zeros there)
    if (plain) {
      Copy::start(s, QT, dim_in, [&](int r) { return qb + int64_t(min(row0 + r, a.rows - 1)) * a.qs[1]; });
      Copy::start(s + kTile, a.rows - row0, dim_in,
                  [&](int r) { return db + int64_t(row0 + r) * a.dos[1]; });
    } else {
      auto row_at = [&](const T* base, const int64_t* st, int r) {
        uint32_t query, head;
        row_of(a, w.kv_head, row0 + r, &query, &head);
        return base + int64_t(query) * st[1] + int64_t(head) * st[2];
      };
      Copy::start(s, QT, dim_in, [&](int r) { return row_at(qb, a.qs, min(row0 + r, a.rows - 1) - row0); });
      Copy::start(s + kTile, a.rows - row0, dim_in, [&](int r) { return row_at(db, a.dos, r); });
    }
  };

  constexpr float kDown = std::is_same_v<T, _Float16> ? 1.0f / 16384.0f : 1.0f;  // undoes kLiftBack
  const float c = a.scale * kLog2e, scale = a.scale * kDown;
  const uint8_t* mask = kMask ? a.mask + int64_t(w.batch) * a.ms[0] + key : nullptr;
  f32x16 dk[L::kOut], dv[L::kOut];
#pragma unroll
  for (int dt = 0; dt < L::kOut; ++dt) dk[dt] = dv[dt] = f32x16{};
  Ranged<T, DK> range;
  // the newest tile's statistics to LDS, beside its rows; a row that saw no key or does not exist gets p = 0
  auto put_stats = [&](int buf) {
    if (tid < QT) {
      s_lse[buf][tid] = lse == -INFINITY ? -INFINITY : kLiftBack<T> - lse * kLog2e;
      s_delta[buf][tid] = lse == -INFINITY ? 0.0f : -delta * scale;
      if constexpr (kMask) s_mask[buf][tid] = mask_at;
    }
  };
  // the mask bytes of a tile, one row each of this lane's 16 values of a block, a tile ahead
  uint8_t seen_row[kMask ? kBlocks * 16 : 1];
  auto fetch_mask = [&](uint32_t t, int buf) {
    if constexpr (kMask) {
#pragma unroll
      for (int e = 0; e < kBlocks * 16; ++e) {
        const int r = 32 * (e / 16) + 8 * (e % 16 / 4) + 4 * h + e % 4;
        seen_row[e] = valid && t * QT + r < a.rows ? mask[s_mask[buf][r]] : uint8_t(0);
      }
    }
  };
  clear_tiles<T, DK>(s_tile, 2 * kRing * kTile, dim_in);
  if constexpr (kOwn) clear_tiles<T, DK>(s_own, kAttnRows * L::kRowBytes, dim_in);
  if constexpr (kMask) s_bad.clear();
  __syncthreads();
  if (t0 < t1) {
    start(t0, s_tile);
    if (kRing == 3) put_stats(0);
    if constexpr (kMask) {
      lds_barrier();
      fetch_mask(t0, 0);
    }
  }
  if (kRing == 3 && t0 + 1 < t1) start(t0 + 1, s_tile + 2 * kTile);
  if (kOwn && t0 < t1) {
    const T* vb = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(w.kv_head) * a.vs[2];
    const uint32_t first = w.tile * kAttnRows;
    Copier<T, DK, kAttnRows>::start(s_own, len - first, dim_in,
                                    [&](int r) { return vb + int64_t(first + r) * a.vs[1]; });
  }
  Vec<T, 8> kf[DK / 16], vf[DK / 16];
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk) kf[kk] = vf[kk] = zero_frag<T>();
  if (valid) {
    const T* kr = static_cast<const T*>(a.k) + int64_t(w.batch) * a.ks[0] + int64_t(key) * a.ks[1] +
                  int64_t(w.kv_head) * a.ks[2];
    const T* vr = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(key) * a.vs[1] +
                  int64_t(w.kv_head) * a.vs[2];
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) {
      kf[kk] = load_frag(kr, kk, dim_in);
      if constexpr (!kOwn) vf[kk] = load_frag(vr, kk, dim_in);
    }
  }
  int buf = 0;
  for (uint32_t t = t0; t < t1; ++t) {
    char *s_q = s_tile + buf * 2 * kTile, *s_d = s_q + kTile;
    const int next = buf == kRing - 1 ? 0 : buf + 1;
    if (kRing == 2) put_stats(buf);
    if (kRing == 3 && t + 1 < t1) put_stats(next);
    if (kRing == 3 && t + 1 < t1 && (t + 2) * QT <= a.rows)
      tile_barrier<2 * Copy::kSteps>();
    else
      tile_barrier<0>();
    uint32_t seen[kBlocks] = {};
    if constexpr (kMask) {  // the next tile's bytes before the copies start, as above
#pragma unroll
      for (int e = 0; e < kBlocks * 16; ++e) seen[e / 16] |= uint32_t(seen_row[e] != 0) << (e % 16);
      if (t + 1 < t1) fetch_mask(t + 1, next);
    }
    bool odd = false;
    if constexpr (kMask)  // a row that saw no key is taken as zeros, whatever it holds
      odd = tile_make_finite<T, DK, 2 * QT>(s_q, t - t0, s_bad,
                                            [&](int r) { return s_lse[buf][r % QT] != -INFINITY; });
    if (kRing == 2 && t + 1 < t1) start(t + 1, s_tile + next * 2 * kTile);
    if (kRing == 3 && t + 2 < t1) start(t + 2, s_tile + (next == 2 ? 0 : next + 1) * 2 * kTile);
    if (key0 < len) {
      f32x16 s[kBlocks], dp[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        s[b] = dp[b] = f32x16{};
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) s[b] = mma(L::frag(s_q, 32 * b, kk), kf[kk], s[b]);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
          dp[b] = mma(L::frag(s_d, 32 * b, kk), kOwn ? L::frag(s_own, (tid >> 6) * 32, kk) : vf[kk], dp[b]);
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        // elements of the tile's q and do in memory, for the bad ones
        auto element = [&](const void* x, const int64_t* st, int r, int d) {
          uint32_t query, head;
          row_of(a, w.kv_head, t * QT + r, &query, &head);
          return static_cast<const T*>(x)[int64_t(w.batch) * st[0] + int64_t(query) * st[1] + int64_t(head) * st[2] + d];
        };
        auto q_element = [&](int r, int d) { return element(a.q, a.qs, r, d); };
        auto do_element = [&](int r, int d) { return element(a.dout, a.dos, r - QT, d); };
        if constexpr (kMask) {
          if (odd) {
            const T* kr = static_cast<const T*>(a.k) + int64_t(w.batch) * a.ks[0] + int64_t(keep_here(key)) * a.ks[1] +
                          int64_t(w.kv_head) * a.ks[2];
            const T* vr = static_cast<const T*>(a.v) + int64_t(w.batch) * a.vs[0] + int64_t(keep_here(key)) * a.vs[1] +
                          int64_t(w.kv_head) * a.vs[2];
            add_products<T, DK, 2 * QT>(s[b], seen[b], 32 * b, t - t0, s_bad, q_element, [&](int d) { return kr[d]; });
            add_products<T, DK, 2 * QT>(dp[b], seen[b], QT + 32 * b, t - t0, s_bad, do_element,
                                        [&](int d) { return vr[d]; });
          }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * b + 8 * g + 4 * h;
          const Vec<float, 4> ls = *reinterpret_cast<const Vec<float, 4>*>(&s_lse[buf][r]);
          const Vec<float, 4> dl = *reinterpret_cast<const Vec<float, 4>*>(&s_delta[buf][r]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * g + i;
            s[b][e] = exp2_fast(fmaf(s[b][e], c, ls[i]));
            dp[b][e] = s[b][e] * fmaf(dp[b][e], scale, dl[i]);
            if constexpr (kMask) {
              const bool vis = (seen[b] >> e) & 1;
              s[b][e] = vis ? s[b][e] : 0.0f;
              dp[b][e] = vis ? dp[b][e] : 0.0f;
            }
          }
        }
        contract<T, DK>(dv, s_d, 32 * b, s[b]);
        range.fit(dp[b], dk);
        contract<T, DK, (sizeof(T) == 2)>(dk, s_q, 32 * b, dp[b]);
        if constexpr (kMask) {
          if (odd) {
            add_outputs<T, DK, 2 * QT>(dv, s[b], seen[b], QT + 32 * b, t - t0, s_bad, do_element);
            add_outputs<T, DK, 2 * QT>(dk, dp[b], seen[b], 32 * b, t - t0, s_bad, q_element);
          }
        }
      }
    }
    buf = next;
  }
  if (key >= a.keys) return;
  if (!valid) {  // past the length: zeros
#pragma unroll
    for (int dt = 0; dt < L::kOut; ++dt) dk[dt] = dv[dt] = f32x16{};
  }
  if (a.splits > 1) {
    const int64_t group = int64_t(w.batch) * a.kv_heads + w.kv_head, all = int64_t(a.batch) * a.kv_heads;
    const int64_t part = (group * a.splits + w.split) * a.keys + key;
    store_column<L::kOut>(a.part + part * dim, dk, range.undo(), dim);
    store_column<L::kOut>(a.part + (all * a.splits * a.keys + part) * dim, dv, kDown, dim);
    return;
  }
  T* ok = static_cast<T*>(a.dk) + int64_t(w.batch) * a.dks[0] + int64_t(key) * a.dks[1] + int64_t(w.kv_head) * a.dks[2];
  T* ov = static_cast<T*>(a.dv) + int64_t(w.batch) * a.dvs[0] + int64_t(key) * a.dvs[1] + int64_t(w.kv_head) * a.dvs[2];
  store_column<L::kOut>(ok, dk, range.undo(), dim);
  store_column<L::kOut>(ov, dv, kDown, dim);
}

// Adds the parts of split rows, in a fixed order: kTurns threads to each (row, four elements), taking every kTurns-th
// part. blockIdx.y = 1 adds dv after dk.
// 40,000 rows of 128 float32: 16 us for dq in four parts (92 MB, 5.7 TB/s), 23 us for dk and dv in three.
template <typename T, bool kKeys, int kTurns>
__global__ __launch_bounds__(kAttnThreads) void k_attn_add(AttnArgs a) {
  constexpr int kQuads = kAttnThreads / kTurns;
  __shared__ float s_part[kTurns > 1 ? kAttnThreads : 1][4];
  const uint32_t lane = threadIdx.x % kQuads, turn = threadIdx.x / kQuads;
  const uint64_t id = uint64_t(blockIdx.x) * kQuads + lane;
  const uint32_t per = kKeys ? a.keys : a.rows, quads = (a.dim + 3) / 4;
  const uint64_t rows = uint64_t(a.batch) * a.kv_heads * per;
  const uint32_t d = uint32_t(id % quads) * 4;
  const int n = int(a.dim - d);
  const uint64_t at = id / quads, group = at / per;
  const uint32_t row = uint32_t(at % per), kv_head = uint32_t(group % a.kv_heads), b = uint32_t(group / a.kv_heads);
  const float* part = a.part + (group * a.splits * per + row) * a.dim + d;
  if (kKeys && blockIdx.y) part += rows * a.splits * a.dim;
  float v[4] = {};
  if (id < rows * quads) {
#pragma unroll 4
    for (uint32_t s = turn; s < a.splits; s += kTurns) {
      float x[4];
      load_f32<4>(part + uint64_t(s) * per * a.dim, n, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += x[i];
    }
  }
  if constexpr (kTurns > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[threadIdx.x][i] = v[i];
    __syncthreads();
    if (turn) return;
#pragma unroll
    for (int k = 1; k < kTurns; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += s_part[k * kQuads + lane][i];
  }
  if (id >= rows * quads) return;
  if constexpr (kKeys) {
    const int64_t* st = blockIdx.y ? a.dvs : a.dks;
    T* out = static_cast<T*>(blockIdx.y ? a.dv : a.dk);
    store_f32<4>(out + int64_t(b) * st[0] + int64_t(row) * st[1] + int64_t(kv_head) * st[2] + d, n, v);
  } else {
    uint32_t query, head;
    row_of(a, kv_head, row, &query, &head);
    store_f32<4>(static_cast<T*>(a.dq) + int64_t(b) * a.dqs[0] + int64_t(query) * a.dqs[1] +
                     int64_t(head) * a.dqs[2] + d, n, v);
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
  // one scratch buffer: copies of inputs, do.o of every row, then the parts of whichever kernel splits (in turn)
  AttnArgs b = a;
  // as the kernels' kStreamBlocks and kWavesPerSimd have it: rows of a streamed tile, workgroups at once on the card
  const bool half = d->dtype != GSR_F32, open = half && !mask;
  const bool one_q = open && a.dim > 64 && a.dim <= 96, one_k = open && a.dim > 64;
  const uint32_t streamed_q = open && !one_q ? 64 : 32, streamed_k = open && !one_k ? 64 : 32;
  const uint32_t cost = half ? 2 : 1;  // 16 bits step faster: 96 wide, 2,500 x 2,500, 378 -> 342 us against 1
  const uint32_t slots_q = a.dim <= (half ? 64u : 48u) || one_q ? 512 : 256;
  const uint32_t slots_k = (half ? a.dim <= 64 || one_k : a.dim <= (mask ? 32u : 48u)) ? 512 : 256;
  const dim3 grid_q = attention_grid(&a, (a.rows + kAttnRows - 1) / kAttnRows,
                                     (uint64_t(a.keys) + streamed_q - 1) / streamed_q, slots_q, cost);
  const dim3 grid_k = attention_grid(&b, (b.keys + kAttnRows - 1) / kAttnRows,
                                     (uint64_t(b.rows) + streamed_k - 1) / streamed_k, slots_k, 2 * cost);
  const size_t groups = size_t(a.batch) * a.kv_heads, deltas = (groups * a.rows + 3) / 4 * 4;
  size_t parts = 0;
  if (a.splits > 1) parts = groups * a.splits * a.rows * a.dim;
  if (b.splits > 1) parts = std::max(parts, 2 * groups * b.splits * b.keys * b.dim);
  const auto inputs = {AttnInput{&a.q, a.qs, a.queries, a.heads},      AttnInput{&a.k, a.ks, a.keys, a.kv_heads},
                       AttnInput{&a.v, a.vs, a.keys, a.kv_heads},      AttnInput{&a.o, a.os, a.queries, a.heads},
                       AttnInput{&a.dout, a.dos, a.queries, a.heads}};
  const size_t packed = attention_pack_bytes(a, d->dtype, inputs);
  if ((st = grow(ctx, ctx->arena.feat_part, packed + (deltas + parts) * sizeof(float)))) return st;
  a.delta = reinterpret_cast<float*>(static_cast<char*>(ctx->arena.feat_part.ptr) + packed);
  a.part = a.delta + deltas;
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_ATTENTION_BACKWARD, s, false);
  attention_pack(&a, d->dtype, inputs, ctx->arena.feat_part.ptr, s);
  const uint32_t tiles = b.tiles, splits = b.splits, works = b.works, per_xcd = b.per_xcd;
  b = a;
  b.tiles = tiles;
  b.splits = splits;
  b.works = works;
  b.per_xcd = per_xcd;
  attention_by_kind(d->dtype, a.dim, mask != nullptr && a.keys, [&](auto t, auto dk_, auto masked) {
    using T = decltype(t);
    constexpr int DK = decltype(dk_)::value;
    constexpr bool kMask = decltype(masked)::value;
    const dim3 block(kAttnThreads);
    // eight threads an element where the parts are many (and the elements few)
    auto add = [&](auto keys, const AttnArgs& x, uint64_t rows) {
      constexpr bool kKeys = decltype(keys)::value;
      const uint64_t n = rows * ((x.dim + 3) / 4);
      if (x.splits > 8)
        hipLaunchKernelGGL((k_attn_add<T, kKeys, 8>), dim3(uint32_t((n + 31) / 32), kKeys ? 2 : 1), block, 0, s, x);
      else if (x.splits > 1)
        hipLaunchKernelGGL((k_attn_add<T, kKeys, 1>), dim3(uint32_t((n + 255) / 256), kKeys ? 2 : 1), block, 0, s, x);
    };
    if (has_q) {
      hipLaunchKernelGGL((k_attn_dq<T, DK, kMask>), grid_q, block, 0, s, a);
      add(std::false_type(), a, groups * a.rows);
    }
    if (has_k) {
      hipLaunchKernelGGL((k_attn_dkv<T, DK, kMask>), grid_k, block, 0, s, b);
      add(std::true_type(), b, groups * b.keys);
    }
  });
  timing_mark(ctx, GSR_STAGE_ATTENTION_BACKWARD, s, true);
  return check_launch(ctx, who);
}
