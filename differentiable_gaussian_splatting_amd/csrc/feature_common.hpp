// Element types, wide loads and argument checks shared by the feature operators (group norm, rotary positions, cross
// attention).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "gsr_internal.hpp"

namespace gsr {

constexpr uint32_t kFeatXcds = 8;  // accelerator dies; workgroups are dealt to them round-robin

// A launch's dimension holds fewer than 2^32 threads: more workgroups than kGridRow are laid out in rows of that many
// (a multiple of the dies, so that their order stays), the last row perhaps past the count.
constexpr uint32_t kGridRow = 1u << 23;

inline dim3 grid_rows(uint64_t workgroups) {
  if (workgroups <= kGridRow) return dim3(uint32_t(workgroups));
  return dim3(kGridRow, uint32_t((workgroups + kGridRow - 1) / kGridRow));
}

__device__ __forceinline__ uint64_t grid_index() { return uint64_t(blockIdx.y) * kGridRow + blockIdx.x; }

// Storage types: float, _Float16, __bf16. Conversions to and from float round to nearest even.
template <typename T, int N>
using Vec = T __attribute__((ext_vector_type(N)));

// n / d by multiplication, for n < 2^31.
struct FastDiv {
  uint32_t m, s, d;
  void set(uint32_t by) {
    d = by;
    s = 0;
    while ((uint64_t(1) << s) < by) ++s;
    m = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - by)) / by + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

// N adjacent elements as floats in one load of any alignment (global memory takes unaligned wide accesses; 16-byte
// aligned ones touch the fewest cache lines), or the first `n` of them, the rest 0.
template <int N, typename T>
__device__ __forceinline__ void load_f32(const T* p, int n, float* f) {
  if (n >= N) {
    Vec<T, N> v;
    __builtin_memcpy(&v, p, sizeof v);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = i < n ? float(p[i]) : 0.0f;
  }
}

template <int N, typename T>
__device__ __forceinline__ void store_f32(T* p, int n, const float* f) {
  if (n >= N) {
    Vec<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = T(f[i]);
    __builtin_memcpy(p, &v, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = T(f[i]);
  }
}

inline bool misaligned(const void* p, size_t elem) { return reinterpret_cast<uintptr_t>(p) % elem != 0; }

inline size_t elem_bytes(uint32_t dtype) { return dtype == GSR_F32 ? 4 : 2; }

// Whether the elements of an output with these (stride, extent) pairs and `inner` adjacent elements are distinct:
// sorted by stride, each stride clears the whole extent below it. Negative strides are refused.
inline bool distinct(std::initializer_list<std::pair<int64_t, uint64_t>> strides, uint64_t inner) {
  std::pair<int64_t, uint64_t> s[4];
  int n = 0;
  for (auto& e : strides) {
    if (e.second == 0) return true;
    if (e.second > 1) s[n++] = e;
  }
  std::sort(s, s + n);
  __int128 span = inner;
  for (int i = 0; i < n; ++i) {
    if (s[i].first < 0 || __int128(s[i].first) < span) return false;
    span += __int128(s[i].first) * __int128(s[i].second - 1);
  }
  return span < (__int128(1) << 62);
}

}  // namespace gsr
