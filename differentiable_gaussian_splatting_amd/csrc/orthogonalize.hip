// Orthogonalised matrix updates by Newton-Schulz products, and the optimiser step that applies them.
//
// A matrix G [rows, cols], transposed if it is tall (r <= c from here on), is scaled to X_0 = G / (|G|_F + eps), whose
// singular values are at most 1, and each step moves every singular value s to s (a + b s^2 + c s^4) by three products:
//   A = X X^T;  P = b A + c A A^T;  X <- a X + P X.
// A and A A^T are symmetric: tiles on and below the diagonal are computed and written twice.
//
// Numbers. A rounding of X is amplified where X is small (a singular value near 0 grows by a at every step, 485 times
// over five), so X in 16 bits would be 2 to 15 % off for the decaying spectra of gradients. X is therefore kept as two
// float16 numbers, x = hi + lo, scaled by a power of two so that the largest singular value a step can reach is near
// 2^14: 22 bits down to 2^-11 of that size and an absolute 2^-39 below, as good as float32 here. The left factors A and
// P only mix what is there, so their roundings are not amplified. float32 and float16 results keep them in two numbers
// too, and every product is hi hi + hi lo + lo hi on the 16-bit matrix cores with float32 sums (three products of
// 2.5 PFLOP/s against one of 157 TFLOP/s in float32; the missing lo lo is 2^-24 of a term): the error of a float32
// evaluation, 1e-6 of the result's norm for flat spectra and 1e-5 for steep ones. bfloat16 results, which round by
// 1.7e-3 of their norm, keep A and P in one float16 number and take A from X's hi alone: 1.0e-3 to 1.6e-3.
#include "attention_common.hpp"

namespace gsr {
namespace {

constexpr int kThreads = 256;
constexpr int kDeep = 32;  // depth of a stage of a product
using half = _Float16;

// The matrices of a call and where their planes lie in the scratch. rp and cp: r and c padded with zeros to whole tiles.
struct OrthShape {
  uint32_t batch, rows, cols, r, c;
  uint64_t rp, cp;
  bool tall;
  uint32_t parts;  // partial sums of squares of a matrix
  float eps, first;  // first: the power of two that X_0 is scaled by
  FastDiv by_vec;  // vectors of kNormVec elements in a row
};

constexpr int kNormVec = 4;

__device__ __forceinline__ void split(float x, half* hi, half* lo) {
  *hi = half(x);
  *lo = half(x - float(*hi));
}

// Sources of the matrix to orthogonalise: the gradient, or the momentum that includes it.
template <typename T, bool MUON>
struct Source {
  const T* grad;
  int64_t gb, gr;  // strides of a matrix and of a row
  float* momentum;
  int64_t mb, mr;
  float mu;
  bool nesterov;
};

// Elements col .. of a row, read once: the momentum is updated here.
template <typename T, bool MUON>
__device__ __forceinline__ void take_new(const Source<T, MUON>& s, uint32_t b, uint32_t row, uint32_t col, int n,
                                         float* u) {
  load_f32<kNormVec>(s.grad + int64_t(b) * s.gb + int64_t(row) * s.gr + col, n, u);
  if constexpr (MUON) {
    float m[kNormVec];
    float* p = s.momentum + int64_t(b) * s.mb + int64_t(row) * s.mr + col;
    load_f32<kNormVec>(p, n, m);
#pragma unroll
    for (int i = 0; i < kNormVec; ++i) m[i] = fmaf(s.mu, m[i], u[i]);
    store_f32<kNormVec>(p, n, m);
#pragma unroll
    for (int i = 0; i < kNormVec; ++i) u[i] = s.nesterov ? fmaf(s.mu, m[i], u[i]) : m[i];
  }
}

// The same elements again, the momentum as take_new left it.
template <typename T, bool MUON>
__device__ __forceinline__ float take_again(const Source<T, MUON>& s, uint32_t b, uint32_t row, uint32_t col) {
  const float g = float(s.grad[int64_t(b) * s.gb + int64_t(row) * s.gr + col]);
  if constexpr (MUON) {
    const float m = s.momentum[int64_t(b) * s.mb + int64_t(row) * s.mr + col];
    return s.nesterov ? fmaf(s.mu, m, g) : m;
  }
  return g;
}

// Partial sums of squares in float64 (no gradient is too small or too large for it), and the new momentum.
template <typename T, bool MUON>
__global__ __launch_bounds__(kThreads) void k_orth_norm(OrthShape g, Source<T, MUON> src, double* __restrict__ part) {
  __shared__ double s[kThreads / 64];
  const uint32_t b = blockIdx.y, vecs = g.by_vec.d * g.rows;
  double sum = 0.0;
  for (uint32_t v = blockIdx.x * kThreads + threadIdx.x; v < vecs; v += g.parts * kThreads) {
    const uint32_t row = g.by_vec.div(v), col = (v - row * g.by_vec.d) * kNormVec;
    float u[kNormVec];
    take_new(src, b, row, col, int(g.cols - col), u);
#pragma unroll
    for (int i = 0; i < kNormVec; ++i)
      if (col + i < g.cols) sum = fma(double(u[i]), double(u[i]), sum);
  }
  for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[size_t(b) * g.parts + blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// X_0 in two planes, transposed if the matrix is tall, zeros in the padding. A workgroup takes a 64 x 64 tile.
template <typename T, bool MUON>
__global__ __launch_bounds__(kThreads) void k_orth_start(OrthShape g, Source<T, MUON> src,
                                                         const double* __restrict__ part, half* __restrict__ x) {
  __shared__ float tile[64][65];
  __shared__ double scale_s;
  const uint32_t b = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  if (threadIdx.x < 64) {
    double sum = 0.0;
    for (uint32_t i = threadIdx.x; i < g.parts; i += 64) sum += part[size_t(b) * g.parts + i];
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
    if (threadIdx.x == 0) {
      const double norm = sqrt(sum) + double(g.eps);
      // a matrix of zeros stays one; one that holds an infinity or NaN gives NaN throughout
      scale_s = norm - norm == 0.0 ? (norm > 0.0 ? double(g.first) / norm : 0.0) : norm - norm;
    }
  }
  __syncthreads();
  const double scale = scale_s;
  // tile[i][j] is X[r0 + i][c0 + j]; the source's rows are walked along its own columns
  const uint32_t row0 = g.tall ? c0 : r0, col0 = g.tall ? r0 : c0;
#pragma unroll 4
  for (int e = threadIdx.x; e < 64 * 64; e += kThreads) {
    const uint32_t i = e / 64, j = e % 64, row = row0 + i, col = col0 + j;
    float v = 0.0f;
    if (row < g.rows && col < g.cols) v = float(double(take_again(src, b, row, col)) * scale);
    if (g.tall)
      tile[j][i] = v;
    else
      tile[i][j] = v;
  }
  __syncthreads();
  const uint64_t plane = g.rp * g.cp;
  half* out = x + 2 * plane * b;
  for (int e = threadIdx.x; e < 64 * 8; e += kThreads) {
    const uint32_t i = e / 8, j = (e % 8) * 8;
    Vec<half, 8> hi, lo;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      half h, l;
      split(tile[i][j + k], &h, &l);
      hi[k] = h;
      lo[k] = l;
    }
    const uint64_t at = (r0 + i) * g.cp + c0 + j;
    *reinterpret_cast<Vec<half, 8>*>(out + at) = hi;
    *reinterpret_cast<Vec<half, 8>*>(out + plane + at) = lo;
  }
}

// One operand of a product: `planes` of [.][ld] float16 from base, `stride` apart.
struct Operand {
  const half* base;
  uint64_t plane, ld;
};

__device__ __forceinline__ void to_lds(const half* p, char* s) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                   (__attribute__((address_space(3))) void*)s, 16, 0, 0);
}

// The two kinds of LDS tiles: kTile rows of kDeep values (both operands' depths adjacent), or kDeep rows of kTile values.
template <int kTile, bool DEEP_ROWS>
struct Stage {
  using L = Tile<half, DEEP_ROWS ? kTile : kDeep>;
  static constexpr int kRows = DEEP_ROWS ? kDeep : kTile;
  static constexpr int kBytes = kTile * kDeep * 2;
  static constexpr int kPass = kThreads / L::kChunks;  // rows that the workgroup copies at a time
  static constexpr int kCopies = kRows / kPass;

  // Starts the copy of rows row .. , values col .. of one plane.
  __device__ static __forceinline__ void start(const half* p, uint64_t ld, uint64_t row, uint64_t col, char* s) {
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int r = int(threadIdx.x) / L::kChunks + i * kPass;
      const int c = ((int(threadIdx.x) % L::kChunks) ^ L::swizzle(r)) * 8;
      to_lds(p + (row + r) * ld + col + c, s + i * kPass * L::kRowBytes + wave * 1024);
    }
  }

  // Depths 16 kk + 8 h .. + 7 of row (or column) at + l % 32.
  __device__ static __forceinline__ Vec<half, 8> frag(const char* s, int at, int kk) {
    if constexpr (!DEEP_ROWS) {
      return L::frag(s, at, kk);
    } else {
      // sixteen lanes read four rows of sixteen columns; lane j of them receives column j
      const int l = threadIdx.x & 63, r = 16 * kk + 8 * (l >> 5) + ((l & 15) >> 2);
      const int chunk = at / 8 + ((l >> 4) & 1) * 2 + ((l & 3) >> 1);
      using s16x4 = Vec<short, 4>;
      using P = __attribute__((address_space(3))) s16x4*;
      const Vec<half, 4> a = __builtin_bit_cast(
          Vec<half, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(s + L::at(r, chunk) + (l & 1) * 8)));
      const Vec<half, 4> b = __builtin_bit_cast(
          Vec<half, 4>, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(s + L::at(r + 4, chunk) + (l & 1) * 8)));
      return Vec<half, 8>{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
};

// One kTile x kTile tile of a product of depth `deep`, on 2 x 2 waves: rows row .. of the left operand (LP planes, depths
// adjacent), columns col .. of the right one (RP planes; its depths adjacent, or its columns where DEEP_ROWS). The
// blocks are computed transposed, so that a lane holds one row of the result (l % 32 of its block) and adjacent columns:
// f(row, column, four sums) is called for each four.
template <int kTile, int LP, int RP, bool DEEP_ROWS, typename F>
__device__ __forceinline__ void product(const Operand& left, const Operand& right, uint64_t row, uint64_t col,
                                        uint64_t deep, F f) {
  using SL = Stage<kTile, false>;
  using SR = Stage<kTile, DEEP_ROWS>;
  constexpr int kStage = LP * SL::kBytes + RP * SR::kBytes;
  constexpr int kBlocks = kTile / 64;
  __shared__ alignas(16) char lds[2][kStage];
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int wr = (wave >> 1) * (kTile / 2), wc = (wave & 1) * (kTile / 2);
  f32x16 acc[kBlocks][kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto start = [&](uint64_t k, char* s) {
#pragma unroll
    for (int p = 0; p < LP; ++p) SL::start(left.base + p * left.plane, left.ld, row, k, s + p * SL::kBytes);
#pragma unroll
    for (int p = 0; p < RP; ++p)
      SR::start(right.base + p * right.plane, right.ld, DEEP_ROWS ? k : col, DEEP_ROWS ? col : k,
                s + LP * SL::kBytes + p * SR::kBytes);
  };
  start(0, lds[0]);
  int turn = 0;
  for (uint64_t k = 0; k < deep; k += kDeep, turn ^= 1) {
    tile_barrier<0>();
    if (k + kDeep < deep) start(k + kDeep, lds[turn ^ 1]);
    const char *sl = lds[turn], *sr = lds[turn] + LP * SL::kBytes;
#pragma unroll
    for (int kk = 0; kk < kDeep / 16; ++kk) {
      Vec<half, 8> a[LP][kBlocks], b[RP][kBlocks];
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
#pragma unroll
        for (int p = 0; p < LP; ++p) a[p][i] = SL::frag(sl + p * SL::kBytes, wr + 32 * i, kk);
#pragma unroll
        for (int p = 0; p < RP; ++p) b[p][i] = SR::frag(sr + p * SR::kBytes, wc + 32 * i, kk);
      }
#pragma unroll
      for (int p = 0; p < LP; ++p)
#pragma unroll
        for (int q = 0; q + p < (LP > RP ? LP : RP); ++q)  // not lo lo
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
              if (q < RP) acc[i][j] = mma(b[q][j], a[p][i], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f(row + wr + 32 * i + (l & 31), col + wc + 32 * j + 8 * q + 4 * (l >> 5),
          Vec<float, 4>{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
}

template <int PLANES>
__device__ __forceinline__ Vec<float, 4> load_split(const half* p, uint64_t plane) {
  const Vec<half, 4> h = *reinterpret_cast<const Vec<half, 4>*>(p);
  Vec<float, 4> v = {float(h[0]), float(h[1]), float(h[2]), float(h[3])};
  if constexpr (PLANES == 2) {
    const Vec<half, 4> l = *reinterpret_cast<const Vec<half, 4>*>(p + plane);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += float(l[i]);
  }
  return v;
}

template <int PLANES>
__device__ __forceinline__ void store_split(half* p, uint64_t plane, Vec<float, 4> v) {
  Vec<half, 4> hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    half h, l;
    split(v[i], &h, &l);
    hi[i] = h;
    lo[i] = l;
  }
  *reinterpret_cast<Vec<half, 4>*>(p) = hi;
  if constexpr (PLANES == 2) *reinterpret_cast<Vec<half, 4>*>(p + plane) = lo;
}

// Which tile a workgroup computes: workgroups are dealt to the dies round-robin, so consecutive tiles go to one die.
struct Works {
  uint64_t works, per_xcd;
  __device__ __forceinline__ bool mine(uint64_t* w) const {
    const uint64_t id = grid_index();
    *w = (id % kFeatXcds) * per_xcd + id / kFeatXcds;
    return *w < works && id / kFeatXcds < per_xcd;
  }
};

// (i, j) of the t-th tile of a lower triangle, row by row.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t* i, uint32_t* j) {
  uint32_t r = uint32_t((sqrtf(8.0f * float(t) + 1.0f) - 1.0f) * 0.5f);
  while (uint64_t(r) * (r + 1) / 2 > t) --r;
  while (uint64_t(r + 1) * (r + 2) / 2 <= t) ++r;
  *i = r;
  *j = t - uint32_t(uint64_t(r) * (r + 1) / 2);
}

// out = alpha in + beta (x x^T) [r, r], PLANES planes each of x (XP read), in (none if alpha is 0) and out, symmetric.
template <int kTile, int PLANES, bool ADD>
__global__ __launch_bounds__(kThreads) void k_orth_symmetric(Works w, uint32_t tiles, Operand x, uint64_t x_matrix,
                                                             uint64_t deep, const half* __restrict__ in,
                                                             half* __restrict__ out, uint64_t rp, float alpha,
                                                             float beta) {
  uint64_t id;
  if (!w.mine(&id)) return;
  const uint64_t b = id / tiles;
  uint32_t ti, tj;
  triangle(uint32_t(id - b * tiles), &ti, &tj);
  const uint64_t plane = rp * rp;
  x.base += b * x_matrix;
  in += b * PLANES * plane;
  out += b * PLANES * plane;
  product<kTile, PLANES, PLANES, false>(
      x, x, uint64_t(ti) * kTile, uint64_t(tj) * kTile, deep, [&](uint64_t row, uint64_t col, Vec<float, 4> v) {
        v *= beta;
        if constexpr (ADD) v += alpha * load_split<PLANES>(in + row * rp + col, plane);
        store_split<PLANES>(out + row * rp + col, plane, v);
        if (ti != tj)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            half h, l;
            split(v[k], &h, &l);
            out[(col + k) * rp + row] = h;
            if constexpr (PLANES == 2) out[plane + (col + k) * rp + row] = l;
          }
      });
}

// What the last product is for: nothing (X' = its planes are written), a result in type T, or a parameter's update.
template <typename T>
struct Result {
  T* p;
  int64_t mat, row;  // strides
  float decay, lr;   // parameters: p = decay p - lr x
};

enum { kNext = 0, kWrite = 1, kUpdate = 2 };

// X' = alpha X + beta (P X), PP planes of P.
template <int kTile, int PP, int WHAT, typename T>
__global__ __launch_bounds__(kThreads) void k_orth_apply(Works w, OrthShape g, uint32_t tiles_r, uint32_t tiles_c,
                                                         Operand p, const half* x, half* next, float alpha, float beta,
                                                         Result<T> res) {
  uint64_t id;
  if (!w.mine(&id)) return;
  const uint32_t tr = uint32_t(id % tiles_r);
  id /= tiles_r;
  const uint32_t tc = uint32_t(id % tiles_c);
  const uint64_t b = id / tiles_c, plane = g.rp * g.cp;
  p.base += b * PP * p.plane;
  x += b * 2 * plane;
  const Operand right{x, plane, g.cp};
  product<kTile, PP, 2, true>(
      p, right, uint64_t(tr) * kTile, uint64_t(tc) * kTile, g.rp, [&](uint64_t row, uint64_t col, Vec<float, 4> v) {
        v = v * beta + alpha * load_split<2>(x + row * g.cp + col, plane);
        if constexpr (WHAT == kNext) {
          store_split<2>(next + b * 2 * plane + row * g.cp + col, plane, v);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (row >= g.r || col + k >= g.c) continue;
            T* o = res.p + int64_t(b) * res.mat +
                   (g.tall ? int64_t(col + k) * res.row + int64_t(row) : int64_t(row) * res.row + int64_t(col + k));
            if constexpr (WHAT == kUpdate)
              *o = res.decay * *o - res.lr * v[k];
            else
              *o = T(v[k]);
          }
        }
      });
}

struct Step {
  float a, b, c;
};

// The steps' coefficients and the powers of two that keep X, A and P in float16's range: `top` is the largest singular
// value that X can have, from the polynomial's largest magnitude on [0, top] (at the ends or where its slope is 0).
struct Plan {
  int steps;
  Step step[GSR_ORTHOGONALIZE_MAX_STEPS];
  int x_exp[GSR_ORTHOGONALIZE_MAX_STEPS + 1], a_exp[GSR_ORTHOGONALIZE_MAX_STEPS], p_exp[GSR_ORTHOGONALIZE_MAX_STEPS];
};

int room(double top) { return 14 - std::max(-8, int(std::ceil(std::log2(std::max(top, 1e-30))))); }

bool plan_of(const gsr_newton_schulz* d, Plan* p) {
  p->steps = int(d->steps);
  double top = 1.0;
  for (int k = 0; k < p->steps; ++k) {
    const double a = d->coefficients[k][0], b = d->coefficients[k][1], c = d->coefficients[k][2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    p->step[k] = Step{float(a), float(b), float(c)};
    p->x_exp[k] = room(top);
    p->a_exp[k] = room(top * top);
    p->p_exp[k] = room(std::fabs(b) * top * top + std::fabs(c) * top * top * top * top);
    auto value = [&](double u) { return std::sqrt(u) * std::fabs(a + b * u + c * u * u); };
    double next = value(top * top);
    const double disc = 9 * b * b - 20 * a * c;  // slope a + 3 b u + 5 c u^2 in u = s^2
    for (int sign = -1; sign <= 1 && disc >= 0; sign += 2) {
      const double q = -3 * b + sign * std::sqrt(disc);
      const double u = c != 0 ? q / (10 * c) : (b != 0 ? -a / (3 * b) : -1.0);
      if (u > 0 && u < top * top) next = std::max(next, value(u));
    }
    top = next;
    if (!(top <= 8.0)) return false;
  }
  p->x_exp[p->steps] = 0;
  return true;
}

uint64_t round_up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

template <int kTile, int PLANES, typename T, bool MUON, typename R>
void launch_steps(hipStream_t s, const OrthShape& g, const Plan& plan, const Source<T, MUON>& src, double* part, half* x0,
                  half* x1, half* am, half* pm, const Result<R>& res) {
  hipLaunchKernelGGL((k_orth_norm<T, MUON>), dim3(g.parts, g.batch), dim3(kThreads), 0, s, g, src, part);
  hipLaunchKernelGGL((k_orth_start<T, MUON>), dim3(uint32_t(g.cp / 64), uint32_t(g.rp / 64), g.batch), dim3(kThreads), 0,
                     s, g, src, part, x0);
  const uint64_t plane = g.rp * g.cp, square = g.rp * g.rp;
  const uint32_t tr = uint32_t(g.rp / kTile), tc = uint32_t(g.cp / kTile), tri = uint32_t(uint64_t(tr) * (tr + 1) / 2);
  auto works = [](uint64_t n) { return Works{n, (n + kFeatXcds - 1) / kFeatXcds}; };
  const Works half_square = works(uint64_t(tri) * g.batch), whole = works(uint64_t(tr) * tc * g.batch);
  auto grid = [](const Works& w) { return grid_rows(w.per_xcd * kFeatXcds); };
  for (int k = 0; k < plan.steps; ++k) {
    const Step& c = plan.step[k];
    const int ex = plan.x_exp[k], ea = plan.a_exp[k], ep = plan.p_exp[k], en = plan.x_exp[k + 1];
    hipLaunchKernelGGL((k_orth_symmetric<kTile, PLANES, false>), grid(half_square), dim3(kThreads), 0, s, half_square,
                       tri, Operand{x0, plane, g.cp}, 2 * plane, g.cp, am, am, g.rp, 0.0f,
                       std::ldexp(1.0f, ea - 2 * ex));
    hipLaunchKernelGGL((k_orth_symmetric<kTile, PLANES, true>), grid(half_square), dim3(kThreads), 0, s, half_square,
                       tri, Operand{am, square, g.rp}, PLANES * square, g.rp, am, pm, g.rp, std::ldexp(c.b, ep - ea),
                       std::ldexp(c.c, ep - 2 * ea));
    const float alpha = std::ldexp(c.a, en - ex), beta = std::ldexp(1.0f, en - ep - ex);
    const Operand p{pm, square, g.rp};
    if (k + 1 < plan.steps)
      hipLaunchKernelGGL((k_orth_apply<kTile, PLANES, kNext, R>), grid(whole), dim3(kThreads), 0, s, whole, g, tr, tc, p,
                         x0, x1, alpha, beta, res);
    else
      hipLaunchKernelGGL((k_orth_apply<kTile, PLANES, MUON ? kUpdate : kWrite, R>), grid(whole), dim3(kThreads), 0, s,
                         whole, g, tr, tc, p, x0, x1, alpha, beta, res);
    std::swap(x0, x1);
  }
}

// The checks that both entry points share, and the shape of the work; an empty call leaves g->batch 0.
gsr_status check_desc(gsr_ctx* ctx, const gsr_newton_schulz* d, const char* who, Plan* plan) {
  if (!d) return fail(ctx, GSR_EINVAL, "%s: null descriptor", who);
  if (d->dtype > GSR_BF16) return fail(ctx, GSR_EINVAL, "%s: unknown dtype %u", who, d->dtype);
  if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return fail(ctx, GSR_EINVAL, "%s: eps must be finite and >= 0", who);
  if (d->steps < 1 || d->steps > GSR_ORTHOGONALIZE_MAX_STEPS)
    return fail(ctx, GSR_EINVAL, "%s: 1 to %d steps are supported, got %u", who, GSR_ORTHOGONALIZE_MAX_STEPS, d->steps);
  if (!plan_of(d, plan))
    return fail(ctx, GSR_EINVAL, "%s: the coefficients must be finite and keep singular values up to 1 below 8", who);
  if (d->batch >= (1u << 16)) return fail(ctx, GSR_EOVERFLOW, "%s: batch >= 2^16", who);
  if (d->rows >= (1u << 20) || d->cols >= (1u << 20) || uint64_t(d->rows) * d->cols >= (uint64_t(1) << 31))
    return fail(ctx, GSR_EOVERFLOW, "%s: rows or cols >= 2^20 or rows * cols >= 2^31", who);
  return GSR_OK;
}

template <typename T, bool MUON, typename R>
gsr_status run(gsr_ctx* ctx, hipStream_t s, const gsr_newton_schulz* d, const Plan& plan,
               const Source<T, MUON>& src, const Result<R>& res, int stage, const char* who) {
  constexpr int kPlanes = std::is_same_v<R, __bf16> ? 1 : 2;
  OrthShape g{};
  g.batch = d->batch;
  g.rows = d->rows;
  g.cols = d->cols;
  g.tall = d->rows > d->cols;
  g.r = std::min(d->rows, d->cols);
  g.c = std::max(d->rows, d->cols);
  g.eps = d->eps;
  g.first = std::ldexp(1.0f, plan.x_exp[0]);
  g.by_vec.set((d->cols + kNormVec - 1) / kNormVec);
  g.parts = uint32_t(std::min<uint64_t>(256, (uint64_t(g.by_vec.d) * g.rows + 4 * kThreads - 1) / (4 * kThreads)));
  const int tile = g.r <= 512 ? 64 : 128;
  g.rp = round_up(g.r, tile);
  g.cp = round_up(g.c, tile);
  const size_t plane = g.rp * g.cp, square = g.rp * g.rp, parts = round_up(size_t(g.batch) * g.parts, 2);
  gsr_status st = grow(ctx, ctx->arena.feat_part,
                       parts * sizeof(double) + g.batch * (4 * plane + 2 * kPlanes * square) * sizeof(half));
  if (st) return st;
  double* part = static_cast<double*>(ctx->arena.feat_part.ptr);
  half* x0 = reinterpret_cast<half*>(part + parts);
  half* x1 = x0 + 2 * plane * g.batch;
  half* am = x1 + 2 * plane * g.batch;
  half* pm = am + kPlanes * square * g.batch;
  timing_mark(ctx, stage, s, false);
  if (tile == 64)
    launch_steps<64, kPlanes>(s, g, plan, src, part, x0, x1, am, pm, res);
  else
    launch_steps<128, kPlanes>(s, g, plan, src, part, x0, x1, am, pm, res);
  timing_mark(ctx, stage, s, true);
  return check_launch(ctx, who);
}

// Calls f(element type) with the descriptor's type.
template <typename F>
gsr_status by_type(uint32_t dtype, F f) {
  if (dtype == GSR_F32) return f(float());
  if (dtype == GSR_F16) return f(half());
  return f(__bf16());
}

}  // namespace
}  // namespace gsr

using namespace gsr;

extern "C" gsr_status gsr_orthogonalize(gsr_ctx* ctx, void* stream, const gsr_newton_schulz* d, const void* g,
                                        void* out) {
  static const char* who = "gsr_orthogonalize";
  if (!ctx) return GSR_EINVAL;
  Plan plan;
  gsr_status st = check_desc(ctx, d, who, &plan);
  if (st) return st;
  if (!d->batch || !d->rows || !d->cols) return GSR_OK;
  if (!g || !out) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  const size_t eb = elem_bytes(d->dtype);
  if (misaligned(g, eb) || misaligned(out, eb))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!distinct({{d->out_stride[0], d->batch}, {d->out_stride[1], d->rows}}, d->cols))
    return fail(ctx, GSR_EINVAL, "%s: the strides of out overlap", who);
  if ((st = enter(ctx))) return st;
  return by_type(d->dtype, [&](auto t) {
    using T = decltype(t);
    const Source<T, false> src{static_cast<const T*>(g), d->grad_stride[0], d->grad_stride[1]};
    const Result<T> res{static_cast<T*>(out), d->out_stride[0], d->out_stride[1], 0.0f, 0.0f};
    return run(ctx, static_cast<hipStream_t>(stream), d, plan, src, res, GSR_STAGE_ORTHOGONALIZE, who);
  });
}

extern "C" gsr_status gsr_muon_step(gsr_ctx* ctx, void* stream, const gsr_newton_schulz* d, const void* grad,
                                    float* param, float* momentum, float lr, float mu, int32_t nesterov, float decay) {
  static const char* who = "gsr_muon_step";
  if (!ctx) return GSR_EINVAL;
  Plan plan;
  gsr_status st = check_desc(ctx, d, who, &plan);
  if (st) return st;
  if (!std::isfinite(lr) || !std::isfinite(mu) || !std::isfinite(decay))
    return fail(ctx, GSR_EINVAL, "%s: lr, mu and decay must be finite", who);
  if (!d->batch || !d->rows || !d->cols) return GSR_OK;
  if (!grad || !param || !momentum) return fail(ctx, GSR_EINVAL, "%s: null pointer", who);
  if (misaligned(grad, elem_bytes(d->dtype)) || misaligned(param, 4) || misaligned(momentum, 4))
    return fail(ctx, GSR_EINVAL, "%s: a pointer is not aligned to its element", who);
  if (!distinct({{d->out_stride[0], d->batch}, {d->out_stride[1], d->rows}}, d->cols))
    return fail(ctx, GSR_EINVAL, "%s: the strides of param overlap", who);
  if (!distinct({{d->momentum_stride[0], d->batch}, {d->momentum_stride[1], d->rows}}, d->cols))
    return fail(ctx, GSR_EINVAL, "%s: the strides of momentum overlap", who);
  if ((st = enter(ctx))) return st;
  return by_type(d->dtype, [&](auto t) {
    using T = decltype(t);
    const Source<T, true> src{static_cast<const T*>(grad), d->grad_stride[0], d->grad_stride[1], momentum,
                              d->momentum_stride[0], d->momentum_stride[1], mu, nesterov != 0};
    const Result<float> res{param, d->out_stride[0], d->out_stride[1], decay, lr};
    return run(ctx, static_cast<hipStream_t>(stream), d, plan, src, res, GSR_STAGE_MUON, who);
  });
}
