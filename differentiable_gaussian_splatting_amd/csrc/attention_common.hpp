// Tiles, matrix fragments and arguments shared by the cross attention kernels.
//
// Every product is computed on 32 x 32 blocks of the matrix cores, 16 deep. With l the lane and h = l / 32, a lane holds
//   an operand fragment: 8 values of row (or column) l % 32, at depths 8 h .. 8 h + 7;
//   a result block: column l % 32, rows 8 (i / 4) + 4 h + i % 4 for i = 0 .. 15.
// The depth order of a product may be permuted freely if both operands agree, so a 32 x 32 result block of scores is,
// as it lies in registers, the right operand of the product that sums over its rows: its values 8 s .. 8 s + 7 are the
// fragment of rows 16 s + 4 h + {0..3} and 16 s + 8 + 4 h + {0..3}. Probabilities therefore never pass through LDS; the
// left operand (the transposed tile) is read from LDS in that order, with the hardware's transposing reads for 16-bit
// types. float32 features use the same fragments, each fed to eight 32 x 32 x 2 float products.
#pragma once

#include <type_traits>

#include "feature_common.hpp"

namespace gsr {

constexpr int kAttnThreads = 256, kAttnWaves = 4;
constexpr int kAttnRows = 32 * kAttnWaves;  // rows (queries, or keys in the key gradient) of a workgroup
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

using f32x16 = Vec<float, 16>;
using u32x4 = Vec<uint32_t, 4>;

// Powers of two by which probabilities are kept too large: a float16 probability below 2^-14 would lose bits, and in a
// long flat context most are. The forward's are at most 2^8 (kSlack) over the running maximum, so 2^7 more stays
// finite; the backward's are at most 1. The sums divide them out.
template <typename T>
constexpr float kLift = std::is_same_v<T, _Float16> ? 7.0f : 0.0f;
template <typename T>
constexpr float kLiftBack = std::is_same_v<T, _Float16> ? 14.0f : 0.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// a * b + c on one block.
__device__ __forceinline__ f32x16 mma(Vec<__bf16, 8> a, Vec<__bf16, 8> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(Vec<_Float16, 8> a, Vec<_Float16, 8> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(Vec<float, 8> a, Vec<float, 8> b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// The other half's value of the same column (lane ^ 32).
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

struct AttnArgs {
  const void *q, *k, *v, *o, *dout;
  void *out, *dq, *dk, *dv;
  const int32_t* kv_len;
  const uint8_t* mask;
  float *lse, *delta, *part, *part_ml;
  uint32_t batch, heads, kv_heads, queries, keys, dim;
  uint32_t rows;   // queries * (heads / kv_heads): the rows that meet one key head
  uint32_t tiles;  // workgroups across rows (keys in the key gradient)
  uint32_t splits, works, per_xcd;
  uint32_t dim_in;  // elements of a row of q, k, v, o and do: dim, or dim padded with zeros to whole 16-byte chunks
  float scale;
  FastDiv share;   // row -> query; the rest is the head within its group
  int64_t qs[3], ks[3], vs[3], os[3], ms[3], dos[3], dqs[3], dks[3], dvs[3];
};

// What a workgroup works on. Workgroups are dealt to the dies round-robin, so consecutive works (the row tiles of one
// key head, which read the same keys and values) are given to one die and share its L2.
struct AttnWork {
  uint32_t tile, split, kv_head, batch;
  __device__ __forceinline__ bool set(const AttnArgs& a) {
    const uint32_t id = uint32_t(grid_index());
    uint32_t w = (id % kFeatXcds) * a.per_xcd + id / kFeatXcds;
    if (w >= a.works || id / kFeatXcds >= a.per_xcd) return false;
    tile = w % a.tiles;
    w /= a.tiles;
    split = w % a.splits;
    w /= a.splits;
    kv_head = w % a.kv_heads;
    batch = w / a.kv_heads;
    return true;
  }
};

// The (query, head) of a packed row.
__device__ __forceinline__ void row_of(const AttnArgs& a, uint32_t kv_head, uint32_t row, uint32_t* query,
                                       uint32_t* head) {
  *query = a.share.div(row);
  *head = kv_head * a.share.d + (row - *query * a.share.d);
}

__device__ __forceinline__ uint32_t keys_of(const AttnArgs& a, uint32_t batch) {
  return a.kv_len ? uint32_t(min(max(a.kv_len[batch], 0), int32_t(a.keys))) : a.keys;
}

// An LDS tile of rows of DK elements (a multiple of 16, the head dimension padded with zeros), in 16-byte chunks, each
// row starting a power of two apart. The chunks of a row are permuted (xor) so that both kinds of reads touch each of
// the 64 banks once per pass: sixteen rows at one chunk (operand fragments), and four adjacent rows at four adjacent
// chunks (transposing reads).
template <typename T, int DK>
struct Tile {
  static constexpr int kPer = 16 / int(sizeof(T));                 // elements per chunk
  static constexpr int kRow = DK <= 32 ? 32 : (DK <= 64 ? 64 : 128);  // elements from row to row
  static constexpr int kChunks = kRow / kPer;
  static constexpr int kRowBytes = kRow * int(sizeof(T));
  static constexpr int kOut = (DK + 31) / 32;                      // 32-wide blocks of the transposed tile
  static constexpr int kLow = kChunks >= 16 ? 0 : (kChunks == 8 ? 1 : 2);

  __device__ static __forceinline__ int swizzle(int r) {
    return (((r >> kLow) & ((4 >> kLow) - 1)) << 2) | ((r >> 2) & 3);
  }
  __device__ static __forceinline__ int at(int r, int chunk) { return r * kRowBytes + ((chunk ^ swizzle(r)) << 4); }

  // Depths 16 kk + 8 h .. + 7 of row r0 + l % 32.
  __device__ static __forceinline__ Vec<T, 8> frag(const char* s, int r0, int kk) {
    const int l = threadIdx.x & 63, r = r0 + (l & 31), h = l >> 5;
    if constexpr (sizeof(T) == 2) {
      return *reinterpret_cast<const Vec<T, 8>*>(s + at(r, 2 * kk + h));
    } else {
      const Vec<T, 4> a = *reinterpret_cast<const Vec<T, 4>*>(s + at(r, 4 * kk + 2 * h));
      const Vec<T, 4> b = *reinterpret_cast<const Vec<T, 4>*>(s + at(r, 4 * kk + 2 * h + 1));
      return Vec<T, 8>{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }

  // The transposed fragment: element column 32 dt + l % 32 at rows r0 + 4 h + {0..3} and r0 + 8 + 4 h + {0..3}.
  __device__ static __forceinline__ Vec<T, 8> frag_t(const char* s, int r0, int dt) {
    const int l = threadIdx.x & 63, h = l >> 5;
    if constexpr (sizeof(T) == 2) {
      // sixteen lanes read four rows of sixteen columns; lane j of them receives column j
      const int r = r0 + 4 * h + ((l & 15) >> 2), chunk = dt * 4 + ((l >> 4) & 1) * 2 + ((l & 3) >> 1);
      using s16x4 = Vec<short, 4>;
      using P = __attribute__((address_space(3))) s16x4*;
      const Vec<T, 4> a = __builtin_bit_cast(
          Vec<T, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(s + at(r, chunk) + (l & 1) * 8)));
      const Vec<T, 4> b = __builtin_bit_cast(
          Vec<T, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(s + at(r + 8, chunk) + (l & 1) * 8)));
      return Vec<T, 8>{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    } else {
      Vec<T, 8> f;
      const int c = dt * 32 + (l & 31);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + 4 * h + (j & 3) + (j >> 2) * 8;
        f[j] = *reinterpret_cast<const T*>(s + at(r, c / kPer) + (c % kPer) * int(sizeof(T)));
      }
      return f;
    }
  }
};

template <typename T>
__device__ __forceinline__ bool finite_bits(T x) {
  if constexpr (sizeof(T) == 4)
    return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) != 0x7f800000u;
  else if constexpr (std::is_same_v<T, _Float16>)
    return (__builtin_bit_cast(uint16_t, x) & 0x7c00u) != 0x7c00u;
  else
    return (__builtin_bit_cast(uint16_t, x) & 0x7f80u) != 0x7f80u;
}

template <typename T>
__device__ __forceinline__ bool any_nonfinite(u32x4 c) {
  constexpr int kPer = 16 / int(sizeof(T));
  const Vec<T, kPer> e = __builtin_bit_cast(Vec<T, kPer>, c);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) bad |= !finite_bits<T>(e[i]);
  return bad;
}

// Copies tiles of R rows to LDS, 1 KiB a wave at a time: thread (row, slot) = (tid / kChunks, tid % kChunks) of every
// kPass rows, the slot holding the chunk that the permutation puts there.
template <typename T, int DK, int R>
struct Copier {
  using L = Tile<T, DK>;
  static constexpr int kPass = kAttnThreads / L::kChunks;
  static constexpr int kSteps = (R + kPass - 1) / kPass;
  static constexpr int kBytes = R * L::kRowBytes;

  __device__ static __forceinline__ int row(int i) { return int(threadIdx.x) / L::kChunks + i * kPass; }
  __device__ static __forceinline__ int col(int i) {
    return ((int(threadIdx.x) % L::kChunks) ^ L::swizzle(row(i))) * L::kPer;
  }

  // Starts the copies of tile rows 0 .. from the addresses at(row), those at or past `rows` as zeros. The chunks travel
  // from memory to LDS by themselves: every wave that has rows starts kSteps of them for a whole tile, and the caller
  // waits.
  template <typename F>
  __device__ static __forceinline__ void start(char* tile, uint32_t rows, int dim, F at) {
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = row(i), c = col(i);
      if (kSteps * kPass != R && r >= R) continue;
      if (c >= dim) continue;
      if (rows >= R || r < int(rows))
        load_lds(at(r) + c, tile + (i * kPass * L::kRowBytes + wave * 1024));
      else
        *reinterpret_cast<u32x4*>(tile + (i * kPass * L::kRowBytes + int(threadIdx.x) * 16)) = u32x4{0, 0, 0, 0};
    }
  }
  __device__ static __forceinline__ void load_lds(const T* p, char* s) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                     (__attribute__((address_space(3))) void*)s, 16, 0, 0);
  }
};

// The barrier of a tile: this wave's copies but the newest kPending have landed, its LDS accesses are done, and so are
// every other wave's. kPending > 0 needs that many copies started after the awaited ones, which a whole tile has and a
// tile that ends early may not have.
template <int kPending>
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kPending) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Clears the chunks past the head dimension, which no copy writes.
template <typename T, int DK>
__device__ __forceinline__ void clear_tiles(char* s, int bytes, int dim) {
  if (dim < Tile<T, DK>::kRow)
    for (int e = int(threadIdx.x) * 16; e < bytes; e += kAttnThreads * 16)
      *reinterpret_cast<u32x4*>(s + e) = u32x4{0, 0, 0, 0};
}

// An operand fragment straight from a row in memory, zeros from `dim` (a whole number of chunks) on.
template <typename T>
__device__ __forceinline__ Vec<T, 8> load_frag(const T* row, int kk, int dim) {
  const int col = 16 * kk + 8 * int((threadIdx.x & 63) >> 5);
  Vec<T, 8> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = T(0.0f);
  if constexpr (sizeof(T) == 2) {
    if (col < dim) f = *reinterpret_cast<const Vec<T, 8>*>(row + col);
  } else {
    Vec<T, 4> a = {}, b = {};
    if (col < dim) a = *reinterpret_cast<const Vec<T, 4>*>(row + col);
    if (col + 4 < dim) b = *reinterpret_cast<const Vec<T, 4>*>(row + col + 4);
    f = Vec<T, 8>{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  return f;
}

template <typename T>
__device__ __forceinline__ Vec<T, 8> zero_frag() {
  Vec<T, 8> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = T(0.0f);
  return f;
}

// Values 8 s .. 8 s + 7 of a block, rounded to the features' type, as an operand fragment.
template <typename T>
__device__ __forceinline__ Vec<T, 8> to_frag(const f32x16& p, int s) {
  Vec<T, 8> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = T(p[8 * s + j]);
  return f;
}

// A barrier for LDS alone: copies from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Which elements of a tile are not finite, a bit each: [tile turn % 3][row][32 columns a word].
template <typename T, int DK, int kRows>
struct BadBits {
  static constexpr int kWords = Tile<T, DK>::kRow / 32;
  uint32_t bits[3][kRows][kWords];
  int any[3];

  __device__ __forceinline__ void clear() {
    for (int e = int(threadIdx.x); e < 3 * kRows * kWords; e += kAttnThreads) (&bits[0][0][0])[e] = 0;
    if (threadIdx.x < 3) any[threadIdx.x] = 0;
  }
};

// Makes the non-finite elements of a tile zeros and notes them (a masked value is 0 as a probability, but 0 * NaN is
// NaN); the caller adds what they contribute where they are seen (add_products, add_outputs). keep(row) false makes that
// row zeros. Returns whether there were any, to every thread; turn counts the tiles.
template <typename T, int DK, int kRows, typename F>
__device__ __forceinline__ bool tile_make_finite(char* tile, uint32_t turn, BadBits<T, DK, kRows>& bad, F keep) {
  using L = Tile<T, DK>;
  const uint32_t now = turn % 3, next = (turn + 1) % 3;
#pragma unroll
  for (int e = int(threadIdx.x); e < kRows * L::kChunks; e += kAttnThreads) {
    u32x4* p = reinterpret_cast<u32x4*>(tile) + e;
    const int row = e / L::kChunks;
    if (!keep(row)) {
      *p = u32x4{0, 0, 0, 0};
    } else if (any_nonfinite<T>(*p)) {
      Vec<T, L::kPer> v = __builtin_bit_cast(Vec<T, L::kPer>, *p);
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < L::kPer; ++j)
        if (!finite_bits<T>(v[j])) {
          bits |= 1u << j;
          v[j] = T(0.0f);
        }
      *p = __builtin_bit_cast(u32x4, v);
      const int col = ((e % L::kChunks) ^ L::swizzle(row)) * L::kPer;
      atomicOr(&bad.bits[now][row][col / 32], bits << (col % 32));
      bad.any[now] = 1;
    }
  }
  for (int e = int(threadIdx.x); e < kRows * bad.kWords; e += kAttnThreads) (&bad.bits[next][0][0])[e] = 0;
  if (threadIdx.x == 0) bad.any[next] = 0;
  lds_barrier();
  return bad.any[now] != 0;
}

// x, in a way that keeps what a rare path computes from it inside that path: hoisted out of the loop over the tiles,
// addresses would hold registers that the loop needs.
__device__ __forceinline__ uint32_t keep_here(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Adds to the visible values of a block (tile rows r0 .. by this lane's column) the products of the rows' bad elements,
// as they lie in memory, with the column's: value(row, element) value of the tile, column(element) of the lane.
template <typename T, int DK, int kRows, typename F, typename G>
__device__ __forceinline__ void add_products(f32x16& s, uint32_t seen, int r0, uint32_t turn,
                                             const BadBits<T, DK, kRows>& bad, F value, G column) {
  const int h = int(threadIdx.x & 63) >> 5;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    if (!((seen >> i) & 1)) continue;
    const int row = r0 + 8 * (i / 4) + 4 * h + i % 4;
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < bad.kWords; ++k)
      for (uint32_t w = bad.bits[turn % 3][row][k]; w; w &= w - 1) {
        const int d = 32 * k + __ffs(int(w)) - 1;
        sum = fmaf(float(value(row, d)), float(column(d)), sum);
      }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j == i) s[j] += sum;
  }
}

// Adds to a column's outputs the bad elements of the tile rows r0 .. r0 + 31 that it sees, each times its value of the
// block p (whose tile rows they are): an infinity times a weight above 0 is that infinity, 0 times it is NaN.
template <typename T, int DK, int kRows, typename F>
__device__ __forceinline__ void add_outputs(f32x16* o, const f32x16& p, uint32_t seen, int r0, uint32_t turn,
                                            const BadBits<T, DK, kRows>& bad, F value) {
  const int h = int(threadIdx.x & 63) >> 5;
  const uint32_t other = __float_as_uint(other_half(__uint_as_float(seen)));
#pragma unroll 1
  for (int r = 0; r < 32; ++r) {
    const int i = (r >> 3) * 4 + (r & 3);
    const bool mine = ((r >> 2) & 1) == h;  // whose half holds row r
    float f = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) f = j == i ? p[j] : f;
    const float theirs = other_half(f);
    f = mine ? f : theirs;
    if (!(((mine ? seen : other) >> i) & 1)) continue;
#pragma unroll
    for (int dt = 0; dt < Tile<T, DK>::kOut; ++dt) {
      const uint32_t w = bad.bits[turn % 3][r0 + r][dt];
      if (!w) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int d = 8 * (j / 4) + 4 * h + j % 4;
        if ((w >> d) & 1) o[dt][j] = fmaf(f, float(value(r0 + r, 32 * dt + d)), o[dt][j]);
      }
    }
  }
}

// acc[dt] += (transposed tile rows) * (block p), over the block's 32 rows, which are tile rows r0 .. With kTwice, p keeps
// about twice the bits of a 16-bit type: what rounding left of it is multiplied too.
template <typename T, int DK, bool kTwice = false>
__device__ __forceinline__ void contract(f32x16* acc, const char* tile, int r0, const f32x16& p) {
  using L = Tile<T, DK>;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const Vec<T, 8> b = to_frag<T>(p, s);
    Vec<T, 8> rest;
    if constexpr (kTwice) {
#pragma unroll
      for (int j = 0; j < 8; ++j) rest[j] = T(p[8 * s + j] - float(b[j]));
    }
#pragma unroll
    for (int dt = 0; dt < L::kOut; ++dt) {
      const Vec<T, 8> f = L::frag_t(tile, r0 + 16 * s, dt);
      acc[dt] = mma(f, b, acc[dt]);
      if constexpr (kTwice) acc[dt] = mma(f, rest, acc[dt]);
    }
  }
}

// Writes a column's accumulated elements (4 adjacent ones per group of the block) times f.
template <int kOut, typename T>
__device__ __forceinline__ void store_column(T* row, const f32x16* acc, float f, int dim) {
  const int h = int(threadIdx.x & 63) >> 5;
#pragma unroll
  for (int dt = 0; dt < kOut; ++dt)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = dt * 32 + 8 * g + 4 * h;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[dt][4 * g + i] * f;
      if (d < dim) store_f32<4>(row + d, dim - d, v);
    }
}

// The mask bytes of the 32 keys from `key0` on, as this lane's 16 values of the block see them: four adjacent keys a
// word. `mask` is the row's (null: a row beyond the last sees nothing); keys past `len` are not read.
__device__ __forceinline__ void mask_words(const uint8_t* mask, uint32_t key0, uint32_t len, uint32_t* words) {
  const uint32_t h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t key = key0 + 8 * g + 4 * h;
    words[g] = 0;
    if (mask && key < len) {
      if (key + 4 <= len) {
        __builtin_memcpy(&words[g], mask + key, 4);
      } else {
        for (uint32_t i = 0; i < 4 && key + i < len; ++i) words[g] |= uint32_t(mask[key + i]) << (8 * i);
      }
    }
  }
}

// Bit i: value i of the block of keys from `key0` on is visible, by its mask words (kMask) and the length.
template <bool kMask>
__device__ __forceinline__ uint32_t visible(const uint32_t* words, uint32_t key0, uint32_t len) {
  const uint32_t h = (threadIdx.x & 63) >> 5;
  uint32_t seen = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      seen |= uint32_t(kMask ? ((words[g] >> (8 * i)) & 0xffu) != 0 : key0 + 8 * g + 4 * h + i < len) << (4 * g + i);
  return seen;
}

// Host side (attention_fwd.hip): checks the descriptor and the inputs both directions share and fills the arguments.
gsr_status attention_args(gsr_ctx* ctx, const gsr_attention* d, const void* q, const void* k, const void* v,
                          const int32_t* kv_lengths, const uint8_t* mask, const void* o, const char* who,
                          AttnArgs* a);

// An input of the kernels: its tensor and strides in the arguments, and the tokens and heads it has.
struct AttnInput {
  const void** p;
  int64_t* stride;
  uint32_t tokens, heads;
};

// The kernels read rows in aligned 16-byte chunks. Inputs that do not lie so (a head dimension of no whole number of
// chunks, odd strides, a shifted pointer) are first copied, each row padded with zeros, to `scratch`: attention_pack
// queues the copies and points the arguments at them, attention_pack_bytes says how much they take.
size_t attention_pack_bytes(const AttnArgs& a, uint32_t dtype, std::initializer_list<AttnInput> in);
void attention_pack(AttnArgs* a, uint32_t dtype, std::initializer_list<AttnInput> in, void* scratch, hipStream_t s);

// Fills tiles, splits and the grid of a launch: `tiles` workgroups per key head, each streaming `steps` tiles, `slots`
// workgroups at once on the card. The stream is split so that the last round is full: the time goes as rounds *
// (steps of a part + cost), cost the steps that writing and adding a part take.
inline dim3 attention_grid(AttnArgs* a, uint32_t tiles, uint64_t steps, uint32_t slots, uint32_t cost) {
  const uint64_t base = uint64_t(tiles) * a->kv_heads * a->batch;
  a->tiles = tiles;
  a->splits = 1;
  uint64_t best = ~uint64_t(0);
  for (uint64_t n = 1; base && n <= std::max<uint64_t>(1, std::min<uint64_t>(steps, 4 * slots / base + 4)); ++n) {
    const uint64_t rounds = (base * n + slots - 1) / slots, t = rounds * ((steps + n - 1) / n + (n > 1 ? cost : 0));
    if (t < best) {
      best = t;
      a->splits = uint32_t(n);
    }
    if (base >= 8 * slots) break;  // an unfull last round is little of eight
  }
  a->works = uint32_t(base * a->splits);
  a->per_xcd = (a->works + kFeatXcds - 1) / kFeatXcds;
  return grid_rows(uint64_t(a->per_xcd) * kFeatXcds);
}

// Calls f(element type, head dimension padded to 32, 48, 64, 96 or 128, whether there is a mask). Heads between two of
// these pay for the wider one: five widths by three types and two masks are what the kernels are built for.
template <typename F>
void attention_by_kind(uint32_t dtype, uint32_t dim, bool mask, F f) {
  auto m = [&](auto t, auto dk) {
    if (mask)
      f(t, dk, std::true_type());
    else
      f(t, dk, std::false_type());
  };
  auto d = [&](auto t) {
    if (dim <= 32)
      m(t, std::integral_constant<int, 32>());
    else if (dim <= 48)
      m(t, std::integral_constant<int, 48>());
    else if (dim <= 64)
      m(t, std::integral_constant<int, 64>());
    else if (dim <= 96)
      m(t, std::integral_constant<int, 96>());
    else
      m(t, std::integral_constant<int, 128>());
  };
  if (dtype == GSR_F32)
    d(float());
  else if (dtype == GSR_F16)
    d(_Float16());
  else
    d(__bf16());
}

}  // namespace gsr
