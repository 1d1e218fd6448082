// Cross attention, forward: o = softmax(scale q k^T) v in one pass over the keys, with the running maximum and sum of
// the softmax (in base 2: exp(scale s) = 2^(c s), c = scale log2 e).
//
// A workgroup holds 128 rows (query, head of one key head's group: heads that share keys share the tiles), 32 to a
// wave, and streams tiles of keys and values through three LDS buffers: the copies of the next two tiles, which go from
// memory to LDS without passing registers, are in flight while a tile is multiplied, and one barrier a tile suffices.
// Scores are computed transposed (keys down, queries
// across), so that a query's maximum and sum are a lane's own registers plus one exchange between the wave's halves.
// With at most 32 rows (a served token) the waves take 32 keys each of a tile of 128 instead, and their results are
// joined in LDS. With few rows and many keys, the keys are split over workgroups and k_attn_join adds the parts in
// order.
#include <type_traits>

#include "attention_common.hpp"

namespace gsr {
namespace {

// The maximum a row's exponents are taken relative to follows its true maximum only when that has moved by more than
// this power of two: rescaling the accumulators is then rare, and a probability of 2^8 is as exact as one of 1.
constexpr float kSlack = 8.0f;

// One row's softmax state and output, a column of the transposed blocks.
template <typename T, int DK>
struct Running {
  using L = Tile<T, DK>;
  float m = -INFINITY;  // reference exponent; -inf while no key was seen
  float m_c = 0.0f;     // the same, 0 while no key was seen
  float l = 0.0f;       // this half's sum of 2^(c s - m_c + kLift)
  f32x16 o[L::kOut];

  // Adds kBlocks blocks of scores of the keys in tile rows r0 .., whose values are rows of s_v.
  template <int kBlocks>
  __device__ __forceinline__ void add(f32x16* s, float c, const char* s_v, int r0) {
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = fmaxf(top, other_half(top)) * c;
    if (__any(top > m + kSlack)) {
      const float m_new = fmaxf(m, top), mc_new = m_new == -INFINITY ? 0.0f : m_new;
      const float f = m == -INFINITY ? 0.0f : exp2_fast(m_c - mc_new);
      m = m_new;
      m_c = mc_new;
      l *= f;
#pragma unroll
      for (int dt = 0; dt < L::kOut; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
    }
    const float lift = kLift<T> - m_c;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = exp2_fast(fmaf(s[b][i], c, lift));
        l += s[b][i];
      }
      // 16-bit probabilities are rounded once: o is then within 1.43 times the error of a float32 form that rounds its
      // output. Twice the bits, as ds has, bring that to 1.0 and take 320 us instead of 246 (4,096 x 10,000, 16 heads, 64
      // wide), 25.6 instead of 24.6 for one query on 10,000 keys.
      contract<T, DK>(o, s_v, r0 + 32 * b, s[b]);
    }
  }
};

template <typename T, int DK>
constexpr int kKeyTile = sizeof(T) == 2 && DK <= 64 ? 64 : 32;  // keys of a tile; wider heads leave registers for 32

// kFew: at most 32 rows, the waves share them and split each tile's keys.
// 4,096 queries x 10,000 keys, 16 heads, 64 wide, bfloat16: 237 to 246 us, about 700 TFLOP/s where a large product of
// matrices reaches 1,235; 2 x 2,500 x 2,500, 8 heads, 128 wide: 105 us, 488 TFLOP/s. Bound by issue and by the latency
// of LDS: the matrix cores are busy 29 % of the cycles (19 % at 128 wide), exponentials and conversions take the
// vector units half of them, and a wave issues one or the other. A 128-row tile keeps a wave's rows in registers, so a
// byte of LDS feeds 32 rows; waves of 64 rows (half the LDS reads) were no faster at 64 wide (261 against 268 us then)
// and slower at 128 (177 against 118), more splits for three or four waves a SIMD slower (279 to 283 against 267),
// scores a tile ahead of their softmax no faster (260 against 257). kFew: 4 x 10,000 ragged keys, 16 heads on 4 key
// heads, 128 wide, 17 us, about 3.6 TB/s of keys and values.
template <typename T, int DK, bool kMask, bool kFew>
__global__ __launch_bounds__(kAttnThreads, DK <= 64 || (sizeof(T) == 2 && !kMask) ? 2 : 1) void k_attn_fwd(AttnArgs a) {
  using L = Tile<T, DK>;
  constexpr int KT = kFew ? 128 : kKeyTile<T, DK>, kBlocks = kFew ? 1 : KT / 32;
  constexpr int kTile = KT * L::kRowBytes, kBuffers = !kFew ? 3 : (kTile <= (32 << 10) ? 2 : 1);
  constexpr int kJoin = kFew ? kAttnWaves * 32 * (L::kOut * 32 + 4) * 4 : 0;  // the waves' outputs
  constexpr int kBytes = 2 * kBuffers * kTile > kJoin ? 2 * kBuffers * kTile : kJoin;
  __shared__ __attribute__((aligned(16))) char s_tile[kBytes];
  __shared__ float2 s_ml[kFew ? kAttnWaves * 32 : 1];
  __shared__ BadBits<T, DK, kMask ? KT : 1> s_bad;
  AttnWork w;
  if (!w.set(a)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, dim = int(a.dim), dim_in = int(a.dim_in);
  const uint32_t row0 = kFew ? 0 : w.tile * kAttnRows + wave * 32;
  const uint32_t row = row0 + (lane & 31);
  const bool valid = row < a.rows;
  uint32_t query = 0, head = 0;
  if (valid) row_of(a, w.kv_head, row, &query, &head);
  Vec<T, 8> qf[DK / 16];
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk) qf[kk] = zero_frag<T>();
  if (valid) {
    const T* qr = static_cast<const T*>(a.q) + int64_t(w.batch) * a.qs[0] + int64_t(query) * a.qs[1] +
                  int64_t(head) * a.qs[2];
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) qf[kk] = load_frag(qr, kk, dim_in);
  }
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

  const float c = a.scale * kLog2e;
  const int r0 = kFew ? wave * 32 : 0;  // the tile rows of this wave's keys
  Running<T, DK> run;
#pragma unroll
  for (int dt = 0; dt < L::kOut; ++dt) run.o[dt] = f32x16{};
  uint32_t words[kBlocks][4], seen[kBlocks] = {};  // the mask of the tile that comes next; what this one shows
  auto multiply = [&](uint32_t t, const char* s_k, const char* s_v, bool odd, auto edge) {
    f32x16 s[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      s[b] = f32x16{};
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) s[b] = mma(L::frag(s_k, r0 + 32 * b, kk), qf[kk], s[b]);
    }
    if constexpr (kMask || decltype(edge)::value) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        if constexpr (!kMask) seen[b] = visible<false>(nullptr, t * KT + r0 + 32 * b, len);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = (seen[b] >> i) & 1 ? s[b][i] : -INFINITY;
      }
    }
    run.template add<kBlocks>(s, c, s_v, r0);
    if constexpr (kMask) {
      if (odd) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          add_outputs<T, DK, KT>(run.o, s[b], seen[b], r0 + 32 * b, t - t0, s_bad,
                                 [&](int r, int d) { return vb[int64_t(t * KT + r) * a.vs[1] + d]; });
      }
    }
  };
  if (kMask && t0 < t1) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) mask_words(mask, t0 * KT + r0 + 32 * b, len, words[b]);
  }
  clear_tiles<T, DK>(s_tile, 2 * kBuffers * kTile, dim_in);
  if constexpr (kMask) s_bad.clear();
  __syncthreads();
  constexpr int kAhead = kBuffers - 1;  // tiles in flight while one is multiplied
  if (t0 < t1) start(t0, s_tile);
  if (kAhead == 2 && t0 + 1 < t1) start(t0 + 1, s_tile + 2 * kTile);
  int buf = 0;
  for (uint32_t t = t0; t < t1; ++t) {
    char *s_k = s_tile + buf * 2 * kTile, *s_v = s_k + kTile;
    if (kAhead == 2 && t + 1 < t1 && (t + 2) * KT <= len)
      tile_barrier<2 * Copy::kSteps>();
    else
      tile_barrier<0>();
    if constexpr (kMask) {  // before the copies start, so that waiting for these loads does not wait for those
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        seen[b] = visible<true>(words[b], 0, 0);
        mask_words(t + 1 < t1 ? mask : nullptr, (t + 1) * KT + r0 + 32 * b, len, words[b]);
      }
    }
    if (kAhead > 0 && t + kAhead < t1) start(t + kAhead, s_tile + (buf == 0 ? kAhead : buf - 1) * 2 * kTile);
    bool odd = false;
    if constexpr (kMask) odd = tile_make_finite<T, DK, KT>(s_v, t - t0, s_bad, [](int) { return true; });
    if (row0 < a.rows) {
      if ((t + 1) * KT <= len)
        multiply(t, s_k, s_v, odd, std::false_type());
      else
        multiply(t, s_k, s_v, odd, std::true_type());
    }
    buf = buf == kAhead ? 0 : buf + 1;
    if (kAhead == 0 && t + 1 < t1) {
      tile_barrier<0>();
      start(t + 1, s_tile);
    }
  }
  if constexpr (kFew) __syncthreads();  // the tiles' memory takes the waves' outputs
  float l = run.l + other_half(run.l);
  const int64_t part = (int64_t(w.batch * a.kv_heads + w.kv_head) * a.splits + w.split) * a.rows;
  if constexpr (kFew) {
    // rows by waves in LDS, then a thread per (row, four elements)
    constexpr int kWide = L::kOut * 32 + 4;
    float* s_o = reinterpret_cast<float*>(s_tile);
    if (valid) {
      store_column<L::kOut>(s_o + (wave * 32 + lane % 32) * kWide, run.o, 1.0f, L::kOut * 32);
      if (h == 0) s_ml[wave * 32 + lane] = make_float2(l == 0.0f ? -INFINITY : run.m_c, l);
    }
    __syncthreads();
    for (uint32_t e = tid; e < a.rows * (L::kOut * 8); e += kAttnThreads) {
      const uint32_t r = e / (L::kOut * 8), d = e % (L::kOut * 8) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) top = fmaxf(top, s_ml[k * 32 + r].x);
      float sum = 0.0f, v[4] = {};
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) {
        const float2 ml = s_ml[k * 32 + r];
        if (ml.x == -INFINITY) continue;
        const float f = exp2_fast(ml.x - top);
        sum = fmaf(ml.y, f, sum);
        const Vec<float, 4> x = *reinterpret_cast<const Vec<float, 4>*>(s_o + (k * 32 + r) * kWide + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(x[i], f, v[i]);
      }
      if (int(d) >= dim) continue;
      if (a.splits > 1) {
        store_f32<4>(a.part + (part + r) * dim + d, dim - int(d), v);
        if (d == 0) reinterpret_cast<float2*>(a.part_ml)[part + r] = make_float2(top, sum);
        continue;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= inv;
      uint32_t qr, hd;
      row_of(a, w.kv_head, r, &qr, &hd);
      T* out = static_cast<T*>(a.out) + int64_t(w.batch) * a.os[0] + int64_t(qr) * a.os[1] + int64_t(hd) * a.os[2];
      store_f32<4>(out + d, dim - int(d), v);
      if (a.lse && d == 0)
        a.lse[(int64_t(w.batch) * a.heads + hd) * a.queries + qr] =
            sum == 0.0f ? -INFINITY : (top - kLift<T> + log2f(sum)) * kLn2;
    }
    return;
  }
  if (!valid) return;
  if (a.splits > 1) {
    store_column<L::kOut>(a.part + (part + row) * dim, run.o, 1.0f, dim);
    if (h == 0) reinterpret_cast<float2*>(a.part_ml)[part + row] = make_float2(l == 0.0f ? -INFINITY : run.m_c, l);
    return;
  }
  T* out = static_cast<T*>(a.out) + int64_t(w.batch) * a.os[0] + int64_t(query) * a.os[1] + int64_t(head) * a.os[2];
  store_column<L::kOut>(out, run.o, l == 0.0f ? 0.0f : 1.0f / l, dim);
  if (a.lse && h == 0)
    a.lse[(int64_t(w.batch) * a.heads + head) * a.queries + query] =
        l == 0.0f ? -INFINITY : (run.m_c - kLift<T> + log2f(l)) * kLn2;
}

// Joins the parts of rows whose keys were split: a wave per row, its halves taking every other part (four elements a
// lane). 64 rows of 16 parts 5.8 us; 9,324 rows of 6 parts, 48 wide, 9.6 us.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void k_attn_join(AttnArgs a) {
  const uint64_t at = uint64_t(blockIdx.x) * kAttnWaves + (threadIdx.x >> 6), group = at / a.rows;
  if (at >= uint64_t(a.batch) * a.kv_heads * a.rows) return;
  const uint32_t row = uint32_t(at % a.rows), kv_head = uint32_t(group % a.kv_heads), b = uint32_t(group / a.kv_heads);
  const int lane = threadIdx.x & 63, dim = int(a.dim), d = (lane & 31) * 4;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + group * a.splits * a.rows + row;
  const float* part = a.part + (group * a.splits * a.rows + row) * a.dim + d;
  float top = -INFINITY;
  for (uint32_t s = lane; s < a.splits; s += 64) top = fmaxf(top, ml[uint64_t(s) * a.rows].x);
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor(top, k));
  float l = 0.0f, o[4] = {};
#pragma unroll 4
  for (uint32_t s = lane >> 5; s < a.splits; s += 2) {
    const float2 v = ml[uint64_t(s) * a.rows];
    const float f = v.x == -INFINITY ? 0.0f : exp2_fast(v.x - top);
    float x[4] = {};
    if (d < dim && v.x != -INFINITY) load_f32<4>(part + uint64_t(s) * a.rows * a.dim, dim - d, x);
    l = fmaf(v.y, f, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(x[i], f, o[i]);
  }
  l += other_half(l);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] += other_half(o[i]);
  if (lane >= 32 || d >= dim) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  uint32_t query, head;
  row_of(a, kv_head, row, &query, &head);
  T* out = static_cast<T*>(a.out) + int64_t(b) * a.os[0] + int64_t(query) * a.os[1] + int64_t(head) * a.os[2];
  store_f32<4>(out + d, dim - d, o);
  if (a.lse && d == 0)
    a.lse[(int64_t(b) * a.heads + head) * a.queries + query] =
        l == 0.0f ? -INFINITY : (top - kLift<T> + log2f(l)) * kLn2;
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

namespace {

// Rows of one input, [batch][tokens][heads] of dim elements, to adjacent rows of dim_in: a thread per 16-byte chunk.
template <typename T>
__global__ __launch_bounds__(kAttnThreads) void k_attn_pack(const T* __restrict__ x, int64_t s0, int64_t s1,
                                                            int64_t s2, uint32_t tokens, uint32_t heads, uint32_t dim,
                                                            uint64_t chunks, uint32_t per_row, T* __restrict__ out) {
  constexpr int kPer = 16 / int(sizeof(T));
  const uint64_t id = grid_index() * kAttnThreads + threadIdx.x;
  if (id >= chunks) return;
  const uint32_t c = uint32_t(id % per_row) * kPer;
  const uint64_t row = id / per_row, token = row / heads;
  const T* p = x + int64_t(token / tokens) * s0 + int64_t(token % tokens) * s1 + int64_t(row % heads) * s2 + c;
  Vec<T, kPer> v;
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = c + i < dim ? p[i] : T(0.0f);
  reinterpret_cast<Vec<T, kPer>*>(out)[id] = v;
}

bool lies_in_chunks(const AttnArgs& a, size_t eb, const AttnInput& in) {
  if (a.dim * eb % 16 || reinterpret_cast<uintptr_t>(*in.p) % 16) return false;
  for (int i = 0; i < 3; ++i)
    if (in.stride[i] * int64_t(eb) % 16) return false;
  return true;
}

}  // namespace

size_t attention_pack_bytes(const AttnArgs& a, uint32_t dtype, std::initializer_list<AttnInput> in) {
  const size_t eb = elem_bytes(dtype), row = (a.dim * eb + 15) / 16 * 16;
  size_t total = 0;
  for (const AttnInput& t : in)
    if (!lies_in_chunks(a, eb, t)) total += size_t(a.batch) * t.tokens * t.heads * row;
  return total;
}

void attention_pack(AttnArgs* a, uint32_t dtype, std::initializer_list<AttnInput> in, void* scratch, hipStream_t s) {
  const size_t eb = elem_bytes(dtype), row = (a->dim * eb + 15) / 16 * 16;
  char* to = static_cast<char*>(scratch);
  a->dim_in = uint32_t(row / eb);
  for (const AttnInput& t : in) {
    if (lies_in_chunks(*a, eb, t)) continue;
    const uint64_t chunks = uint64_t(a->batch) * t.tokens * t.heads * (row / 16);
    if (chunks) {
      auto launch = [&](auto e) {
        using T = decltype(e);
        hipLaunchKernelGGL((k_attn_pack<T>), grid_rows((chunks + kAttnThreads - 1) / kAttnThreads),
                           dim3(kAttnThreads), 0, s, static_cast<const T*>(*t.p), t.stride[0], t.stride[1],
                           t.stride[2], t.tokens, t.heads, a->dim, chunks, uint32_t(row / 16),
                           reinterpret_cast<T*>(to));
      };
      if (eb == 4)
        launch(float());
      else
        launch(_Float16());  // any two bytes
    }
    *t.p = to;
    t.stride[2] = int64_t(row / eb);
    t.stride[1] = t.stride[2] * t.heads;
    t.stride[0] = t.stride[1] * t.tokens;
    to += chunks * 16;
  }
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
  const bool few = a.rows <= 32;
  const uint32_t key_tile = few ? 128 : (d->dtype != GSR_F32 && d->head_dim <= 64 ? 64 : 32);
  // The costs of a split, in tiles. What they are matters little between 2 and 16: one query on 10,000 ragged keys takes
  // 24.5 us with 2 to 12 and 128 without splits; 600 x 2,500 in float32 84 us with 0 to 8 and 229 without; 300 x 5,000
  // in bfloat16 27 us with 2 to 16 and 88 without. But 0 splits the keys of one query on 257 (20.7 us against 17.6), and
  // 2 splits 16-bit tiles that a round holds anyway (2 x 2,500 x 2,500, 8 heads, 64 wide: 71 us against 63).
  const dim3 grid = attention_grid(&a, few ? 1 : (a.rows + kAttnRows - 1) / kAttnRows,
                                   (uint64_t(a.keys) + key_tile - 1) / key_tile, few ? 256 : 512,
                                   few ? 6 : (d->dtype == GSR_F32 ? 2 : 16));
  const auto inputs = {AttnInput{&a.q, a.qs, a.queries, a.heads}, AttnInput{&a.k, a.ks, a.keys, a.kv_heads},
                       AttnInput{&a.v, a.vs, a.keys, a.kv_heads}};
  const size_t packed = attention_pack_bytes(a, d->dtype, inputs);
  const size_t parts = a.splits > 1 ? size_t(a.batch) * a.kv_heads * a.splits * a.rows : 0;
  if ((st = grow(ctx, ctx->arena.feat_part, packed + parts * (a.dim + 2) * sizeof(float)))) return st;
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ctx->arena.feat_part.ptr) + packed);
  a.part = a.part_ml + parts * 2;
  hipStream_t s = static_cast<hipStream_t>(stream);
  timing_mark(ctx, GSR_STAGE_ATTENTION_FORWARD, s, false);
  attention_pack(&a, d->dtype, inputs, ctx->arena.feat_part.ptr, s);
  attention_by_kind(d->dtype, a.dim, mask != nullptr && a.keys, [&](auto t, auto dk, auto masked) {
    using T = decltype(t);
    constexpr int DK = decltype(dk)::value;
    constexpr bool kMask = decltype(masked)::value;
    if (few)
      hipLaunchKernelGGL((k_attn_fwd<T, DK, kMask, true>), grid, dim3(kAttnThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_attn_fwd<T, DK, kMask, false>), grid, dim3(kAttnThreads), 0, s, a);
    if (a.splits > 1) {
      const uint64_t n = uint64_t(a.batch) * a.kv_heads * a.rows;
      hipLaunchKernelGGL((k_attn_join<T>), dim3(uint32_t((n + kAttnWaves - 1) / kAttnWaves)), dim3(kAttnThreads), 0,
                         s, a);
    }
  });
  timing_mark(ctx, GSR_STAGE_ATTENTION_FORWARD, s, true);
  return check_launch(ctx, who);
}
