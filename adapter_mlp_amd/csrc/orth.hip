// Orthogonalised adapter updates: Newton-Schulz steps on U / (|U| + eps),
//   X <- a X + (b S + c S S) X,   S = X X^T on the short side,
// and the optimizer step that applies the result.
//
// An adapter's gradient has a short side r <= 64 (its rank) and a long side n
// of thousands, so the steps are not taken on X.  With X_0 = U / (|U| + eps)
// tall and G = X_0^T X_0 (r x r), every step multiplies X from the right by
// p(G_k) = a I + b G_k + c G_k^2, and G_{k+1} = p(G_k)^2 G_k; all of these are
// polynomials of G and commute.  So U is read once for U^T U, the steps run
// on r x r matrices (Q = p p ... p), and U is read once more for U Q: two
// passes instead of two per step, bound by HBM (muon: 28 bytes an element in
// fp32, of which 20 must move).
//
// Everything between the fp32 update U and the last rounding is fp64.  The
// steps grow a direction of small singular value by a per step (3.4 by
// default), and the r x r form would also square the rounding of small
// singular values.  fp64 costs little here: v_mfma_f64_16x16x4_f64 takes 64
// cycles (measured) for 2048 flops, 16 per byte of U at r = 64, and runs
// beside the loads.
//
// Labels.  The short side is cut into NT = ceil(r / 16) tiles; label 16 t + c
// (c < 16) stands for index NT c + t.  A lane that holds column c of all
// tiles then owns NT consecutive elements of a row of a tall matrix.  The
// r x r matrices are kept in label order (padded with zeros), which none of
// their products notices.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>

#include "abi.hpp"
#include "common.hpp"

namespace lora {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxGroups = 24;  // stacks per launch (their table is a kernel argument)
constexpr int kSub = 2048;      // elements of U that a wavefront takes at a time, at most
constexpr int kVecs = kSub / 256;    // 4-element vectors per lane of them
constexpr int kRegion = 2560 + 64;   // floats of LDS a wavefront holds them in
// A launch has fewer than 2^32 threads: blocks of 256, and of up to 1024 for the steps.  A stack of fewer
// than 2^30 long-side elements in all has fewer blocks than that (a sub-tile has at least 32 of them).
constexpr int64_t kMaxBlocks = (1 << 24) - 1, kMaxMats = (1 << 22) - 1, kMaxLong = 1 << 30;

// Where U has (nearly) no singular value, rounding leaves +-2^-53 |G| in G, and
// every step multiplies it by a^2.  Once it is of order one a negative value
// makes p(g) exceed a, and G and Q run away (from 16 steps on with the default
// coefficients, for gradients of fewer tokens than the rank).  Up to there the
// error of an entry of O (entries are about 1 at most) is below 2^-53 a^(2 steps):
// measured at most 0.007 of it for five sets of coefficients, ranks 16 to 64, full,
// steep and deficient spectra.  At |a|^steps = 2^22 that is 2^-9, measured 8e-6:
// 12 steps of the default coefficients, 22 at a = 2, 32 at a = 1.5.
constexpr double kMaxGrowth = 1 << 22;

// One stack of `count` matrices with the same shape.
struct OrthGroup {
  const void* G;
  float* M;     // momentum (nullptr: U = G)
  void* P;      // result, or the parameter that takes it
  double* part; // [count][chunks][NT (NT + 1) / 2][4][64] partial U^T U
  double* Q;    // [count][16 NT][16 NT]
  int32_t n, r; // long and short side
  int32_t wide; // 1: [r, n], 0: [n, r]
  int32_t chunks;      // blocks that form U^T U of one matrix
  int32_t sub, pitch;  // long-side elements per sub-tile (wide: a power of two), and its row pitch in LDS
  int32_t sub_log2;
  uint32_t inv_r;      // ceil(2^20 / r): e inv_r >> 20 = e / r for e < 2^11 + 2^9
  int32_t vec_lds;     // vectors of four stay within a row of LDS
  int32_t nsub;        // sub-tiles per wavefront of a block that forms U^T U
  int32_t subs;        // blocks of one sub-tile per wavefront that form U Q
  float scale;
};

// The first blocks of the groups in the three launches (past the last group:
// INT_MAX), side by side so that a few wide scalar loads bring them in.
enum { GRAM, STEPS, APPLY };
struct OrthArgs {
  int32_t first[3][kMaxGroups];
  OrthGroup g[kMaxGroups];
  int32_t ngroups, steps;
  float mu;
  double a, b, c, eps;
  double decay, lr;  // P <- decay P - lr scale O
};

// Four consecutive elements with no more alignment than their own.
__device__ __forceinline__ f32x4 load4(const float* p) {
  typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
  return *reinterpret_cast<const v4*>(p);
}
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  typedef uint16_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  const v4 v = *reinterpret_cast<const v4*>(p);
  return f32x4{bf2f(v[0]), bf2f(v[1]), bf2f(v[2]), bf2f(v[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4 x) {
  typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
  *reinterpret_cast<v4*>(p) = x;
}
__device__ __forceinline__ void store4(uint16_t* p, f32x4 x) {
  typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(2)));
  *reinterpret_cast<v2*>(p) = v2{pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3])};
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = (uint16_t)f2bf(x); }

// The first `valid` of four elements (the rest read 0).
template <typename T>
__device__ __forceinline__ f32x4 load_some(const T* p, int valid) {
  if (valid >= 4) return load4(p);
  f32x4 x = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < valid) x[i] = load1(p + i);
  return x;
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int valid, f32x4 x) {
  if (valid >= 4) {
    store4(p, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < valid) store1(p + i, x[i]);
}

// Hand-off between the lanes of a wavefront through its own LDS region.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A sub-tile of one matrix: `len` (at most g.sub) long-side elements.  Its
// elements are numbered as they lie in memory, tall: row by row, wide: row by
// row of g.sub columns, and vector j of a lane holds four of them from
// 4 (64 j + lane), so every global access is 16 (or, in bf16, 8) bytes of a
// contiguous run whatever the rank.  In LDS element (row, column) is at
// row * pitch + column.
struct SubTile {
  int64_t first;        // first element
  int64_t off, step;    // vector j of the lane is at off + j step
  int len, total;
  int col, row, rows;   // wide: column, and row of vector j: row + j rows
  __device__ __forceinline__ SubTile(const OrthGroup& g, int mat, int i) {
    const int l0 = i * g.sub, e = 4 * ((int)threadIdx.x & 63);
    const int64_t base = (int64_t)mat * g.n * g.r;
    len = g.n - l0 < g.sub ? g.n - l0 : g.sub;
    total = g.sub * g.r;
    row = e >> g.sub_log2;
    col = e & (g.sub - 1);
    rows = 256 >> g.sub_log2;  // g.sub is at most 256
    first = base + (g.wide ? (int64_t)l0 : (int64_t)l0 * g.r);
    off = first + (g.wide ? (int64_t)row * g.n + col : (int64_t)e);
    step = g.wide ? (int64_t)rows * g.n : 256;
  }
  // how many elements of vector j exist (four at least: all)
  __device__ __forceinline__ int valid(const OrthGroup& g, int j) const {
    const int tall = len * g.r - 4 * (64 * j + ((int)threadIdx.x & 63)), wide = row + j * rows < g.r ? len - col : 0;
    return g.wide ? wide : tall;
  }
  // where vector j starts in LDS
  __device__ __forceinline__ void at(const OrthGroup& g, int j, int& r, int& c) const {
    const int e = 4 * (64 * j + ((int)threadIdx.x & 63)), q = (int)(((uint32_t)e * g.inv_r) >> 20);
    r = g.wide ? row + j * rows : q;
    c = g.wide ? col : e - q * g.r;
  }
  // The lane's vectors of a tensor.  FULL (len = g.sub): every vector exists
  // whole or not at all, and is loaded without a branch (one that does not
  // exist reads the first and is not used): the compiler waits for a load at
  // the end of the branch it stands in, so that in branches the loads of a lane
  // follow one another instead of flying together.
  template <bool FULL, typename T>
  __device__ __forceinline__ void load(const OrthGroup& g, const T* p, f32x4 (&x)[kVecs]) const {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if constexpr (FULL) x[j] = load4(p + (valid(g, j) > 0 ? off + j * step : first));
      else x[j] = load_some(p + off + j * step, valid(g, j));
    }
  }
  template <bool FULL, typename T>
  __device__ __forceinline__ void store(const OrthGroup& g, T* p, const f32x4 (&x)[kVecs]) const {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if constexpr (FULL) {
        if (valid(g, j) > 0) store4(p + off + j * step, x[j]);
      } else {
        store_some(p + off + j * step, valid(g, j), x[j]);
      }
    }
  }
};
// The four elements of a vector that starts at (row, column): a tall one may run over row ends.
template <typename F>
__device__ __forceinline__ void each4(const OrthGroup& g, int row, int col, F&& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f(i, row * g.pitch + col);
    if (++col == g.r && !g.wide) {
      col = 0;
      ++row;
    }
  }
}
__device__ __forceinline__ void put4(const OrthGroup& g, float* lds, int row, int col, f32x4 x) {
  if (g.vec_lds) *reinterpret_cast<f32x4*>(lds + row * g.pitch + col) = x;
  else each4(g, row, col, [&](int i, int o) { lds[o] = x[i]; });
}
__device__ __forceinline__ f32x4 get4(const OrthGroup& g, const float* lds, int row, int col) {
  if (g.vec_lds) return *reinterpret_cast<const f32x4*>(lds + row * g.pitch + col);
  f32x4 x;
  each4(g, row, col, [&](int i, int o) { x[i] = lds[o]; });
  return x;
}

// U: the gradient, or the momentum form of it.
enum { ORTH, PLAIN, NESTEROV };

// U of a sub-tile into LDS (zeros past len).  FIRST: the momentum is brought
// up to date (M <- mu M + G) and stored; later passes read the new one.
template <typename T, int MODE, bool FIRST, bool FULL>
__device__ __forceinline__ void load_u(const OrthArgs& a, const OrthGroup& g, const SubTile& st, float* lds) {
  f32x4 x[kVecs], m[kVecs];
  if constexpr (MODE != PLAIN || FIRST) st.load<FULL>(g, static_cast<const T*>(g.G), x);
  if constexpr (MODE != ORTH) st.load<FULL>(g, static_cast<const float*>(g.M), m);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    f32x4 u = x[j];
    if constexpr (MODE != ORTH)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (FIRST) m[j][i] = fmaf(a.mu, m[j][i], x[j][i]);
        u[i] = MODE == NESTEROV ? fmaf(a.mu, m[j][i], x[j][i]) : m[j][i];
      }
    int row, col;
    st.at(g, j, row, col);
    if (4 * (64 * j + ((int)threadIdx.x & 63)) < st.total) put4(g, lds, row, col, u);
  }
  if constexpr (MODE != ORTH && FIRST) st.store<FULL>(g, g.M, m);
}

// The group of this block, and the block's number within it.
__device__ __forceinline__ const OrthGroup& my_group(const OrthArgs& a, int launch, int& b) {
  int k = 0, at = 0;
#pragma unroll
  for (int i = 1; i < kMaxGroups; ++i)
    if ((int)blockIdx.x >= a.first[launch][i]) {
      k = i;
      at = a.first[launch][i];
    }
  b = (int)blockIdx.x - at;
  return a.g[__builtin_amdgcn_readfirstlane(k)];
}

// Partial U^T U of one matrix over one chunk of its long side.  An operand of
// tile t holds, in lane 16 q + c, U at long index k + q (any assignment of the
// four k to the lane groups gives the same sum) and short index NT c + t, and
// serves as both sides of the product.  Only the tiles on and above the
// diagonal are formed.  The wavefronts work alone until their sums meet.
// Measured: momentum form over 448 rank-16 matrices, 503 MB: 95 us, 5.3 TB/s, the
// bound there.  14 rank-64 matrices, 63 MB: 25 us; the matrix cores need 8 of
// them (10 tiles a sub-tile of 16), the rest is a call too short to fill the
// chip: one wave of blocks loads, multiplies, and joins its sums.
template <typename T, int NT, int MODE>
__global__ __launch_bounds__(256, NT <= 2 ? 3 : 2) void orth_gram_kernel(const OrthArgs a) {
  constexpr int NP = NT * (NT + 1) / 2;
  __shared__ __attribute__((aligned(16))) float us[4][kRegion];
  constexpr int AT = NT == 4 ? 5 : NP;  // tiles whose sums meet at a time, in the regions
  static_assert(sizeof(double) * 3 * AT * 256 <= sizeof(us) && NP % AT == 0, "the exchange fits the regions");
  double* const red = reinterpret_cast<double*>(&us[0][0]);
  int b;
  const OrthGroup& g = my_group(a, GRAM, b);
  const int mat = b / g.chunks, chunk = b % g.chunks;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, c = lane & 15;
  float* const u = us[w];
  f64x4 acc[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) acc[i] = f64x4{0, 0, 0, 0};
  auto mma = [&](const float (&x)[NT]) {
    double d[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) d[t] = (double)x[t];
    int i = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = t; s < NT; ++s, ++i) acc[i] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[t], d[s], acc[i], 0, 0, 0);
  };
  for (int i = 0; i < g.nsub; ++i) {
    const SubTile st(g, mat, (chunk * 4 + w) * g.nsub + i);
    if (st.len <= 0) break;
    if (st.len == g.sub) load_u<T, MODE, true, true>(a, g, st, u);
    else load_u<T, MODE, true, false>(a, g, st, u);
    wave_sync();
    if (!g.wide) {
      for (int k = 0; k < st.len; k += 16) {  // rows up to the sub-tile's (a multiple of 16) are zero past len
        float x[4][NT];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int t = 0; t < NT; ++t) x[v][t] = NT * c + t < g.r ? u[(k + 4 * v + q) * g.pitch + NT * c + t] : 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) mma(x[v]);
      }
    } else {
      for (int k = 0; k < st.len; k += 16) {
        f32x4 y[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
          y[t] = NT * c + t < g.r ? *reinterpret_cast<const f32x4*>(u + (NT * c + t) * g.pitch + k + 4 * q) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float x[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) x[t] = y[t][v];
          mma(x);
        }
      }
    }
    wave_sync();
  }
  double* out = g.part + ((int64_t)mat * g.chunks + chunk) * (NP * 256);
#pragma unroll
  for (int i0 = 0; i0 < NP; i0 += AT) {
    __syncthreads();
    if (w > 0)
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[((w - 1) * AT * 4 + i * 4 + v) * 64 + lane] = acc[i0 + i][v];
    __syncthreads();
    if (w == 0)
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int o = (i * 4 + v) * 64 + lane;
          out[i0 * 256 + o] = acc[i0 + i][v] + red[o] + red[AT * 256 + o] + red[2 * AT * 256 + o];
        }
  }
}

// The steps of one matrix on its r x r Gram matrix, one block.  Per step:
// p = a I + b G + c G G; V = G p and Q <- Q p; G <- V p.  All matrices are
// symmetric and commute, so both operands of a product are read along rows,
// and only the tiles on and above the diagonal are formed (10 of 16 at NT =
// 4) and written to both sides.  G is made symmetric to the last bit, in tiles
// on the diagonal too (p then is, as its elements are the same sums): in G and p
// rounding that is not symmetric would grow by a^3 a step instead of a^2.  A
// matrix has only its CU's matrix cores, 2048 flops in 64 cycles each, and at NT =
// 4 that is the bound: one tile a
// wavefront, so that the four matrix cores share each product evenly and one
// wavefront's LDS reads hide behind another's MFMAs.  Rows are 16 NT + 2
// doubles apart, which spreads the 16 rows of a fragment read over all banks.
// Measured: 5 steps 46 to 53 us at rank 64, 33 of them the steps (6.5 each, 4.7 of
// it the matrix cores, which are busy 29% of the kernel on the CUs that have a
// matrix) and up to 20 the way in and out: one block sums the chunks of its matrix,
// 20 KB each, 1.1 MB for a long side of 14336.  9.6 us at rank 16 (0.9 a step, a
// chain of products), whatever the number of matrices up to the chip's CUs.
// fp32 products would halve the steps and lose the small singular values: an error
// of 2^-24 |G| in a direction of G's null space grows by a^2 a step.  In fp64 it is
// 2^-53 |G|, and kMaxGrowth keeps it small.
template <int NT>
__global__ __launch_bounds__(NT >= 3 ? 1024 : 256 * NT) void orth_steps_kernel(const OrthArgs a) {
  constexpr int N = 16 * NT, LD = N + 2, NP = NT * (NT + 1) / 2, THREADS = NT >= 3 ? 1024 : 256 * NT;
  constexpr int WAVES = THREADS / 64;
  __shared__ double mg[N * LD], mp[N * LD], mv[N * LD], mq[N * LD];
  int mat;
  const OrthGroup& g = my_group(a, STEPS, mat);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, c = lane & 15;

  // sum of the chunks, ascending; element (i, v, lane) is row 16 t + 4 v + q, column 16 s + c
  // (every thread's elements of AHEAD chunks are loaded together; past the last chunk it is read again)
  const double* part = g.part + (int64_t)mat * g.chunks * (NP * 256);
  constexpr int PER = (NP * 256 + THREADS - 1) / THREADS, AHEAD = PER > 2 ? 12 : 16;
  double sum[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) sum[j] = 0.0;
  for (int k0 = 0; k0 < g.chunks; k0 += AHEAD) {
    double x[AHEAD][PER];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int j = 0; j < PER; ++j)
        x[k][j] = part[(int64_t)min(k0 + k, g.chunks - 1) * (NP * 256) + min((int)threadIdx.x + j * THREADS, NP * 256 - 1)];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int j = 0; j < PER; ++j) sum[j] = k0 + k < g.chunks ? sum[j] + x[k][j] : sum[j];
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = threadIdx.x + j * THREADS;
    if (e >= NP * 256) break;
    const int i = e >> 8, v = (e >> 6) & 3, l = e & 63;
    int t = 0, first = 0;
    while (i >= first + NT - t) first += NT - t++;
    const int row = 16 * t + 4 * v + (l >> 4), col = 16 * (t + i - first) + (l & 15);
    if (row <= col) mg[row * LD + col] = mg[col * LD + row] = sum[j];
  }
  __syncthreads();
  double trace = lane < N ? mg[lane * LD + lane] : 0.0;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) trace += __shfl_xor(trace, d);
  const double norm = sqrt(trace) + a.eps;
  const double inv = norm == 0.0 ? 0.0 : 1.0 / norm;  // zeros stay zeros whatever eps is
  __syncthreads();
  for (int e = threadIdx.x; e < N * N; e += THREADS) mg[e / N * LD + e % N] *= inv * inv;
  __syncthreads();
  auto product = [&](const double* A, const double* B, int t, int s) {
    f64x4 o = f64x4{0, 0, 0, 0};
    const double* ar = A + (16 * t + c) * LD + q;
    const double* br = B + (16 * s + c) * LD + q;
#pragma unroll
    for (int k = 0; k < N / 4; ++k) o = __builtin_amdgcn_mfma_f64_16x16x4f64(ar[4 * k], br[4 * k], o, 0, 0, 0);
    return o;
  };
  auto corner = [&](int i, int& t, int& s) {  // tile i of the upper triangle, row by row
    int first = 0;
    t = 0;
    while (i >= first + NT - t) first += NT - t++;
    s = t + i - first;
  };
  auto put = [&](double* D, int t, int s, int v, double x) {
    const int row = 16 * t + 4 * v + q, col = 16 * s + c;
    D[row * LD + col] = x;
    if (t != s) D[col * LD + row] = x;
  };
  constexpr int MOST = (2 * NP + WAVES - 1) / WAVES;  // tiles of a pair of products per wavefront
  f64x4 x[MOST];
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    for (int i = w; i < NP; i += WAVES) {
      int t, s;
      corner(i, t, s);
      const f64x4 o = product(mg, mg, t, s);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = 16 * t + 4 * v + q, col = 16 * s + c;
        const double p = fma(a.c, o[v], a.b * mg[row * LD + col]) + (row == col ? a.a : 0.0);
        put(mp, t, s, v, p);
        if (k == 0) put(mq, t, s, v, p);  // Q = I before
      }
    }
    __syncthreads();
    // product 0: V = G p (unless this is the last step), product 1: Q p (unless it is the first)
    const bool need[2] = {!last, k > 0};
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      const int i = w + j * WAVES;
      if (i < 2 * NP && need[i >= NP]) {
        int t, s;
        corner(i >= NP ? i - NP : i, t, s);
        x[j] = product(i >= NP ? mq : mg, mp, t, s);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
      const int i = w + j * WAVES;
      if (i < 2 * NP && need[i >= NP]) {
        int t, s;
        corner(i >= NP ? i - NP : i, t, s);
#pragma unroll
        for (int v = 0; v < 4; ++v) put(i >= NP ? mq : mv, t, s, v, x[j][v]);
      }
    }
    __syncthreads();
    if (last) break;
    for (int i = w; i < NP; i += WAVES) {
      int t, s;
      corner(i, t, s);
      const f64x4 o = product(mv, mp, t, s);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = 16 * t + 4 * v + q, col = 16 * s + c;
        if (row <= col) mg[row * LD + col] = mg[col * LD + row] = o[v];
      }
    }
    __syncthreads();
  }
  double* Q = g.Q + (int64_t)mat * N * N;
  for (int e = threadIdx.x; e < N * N; e += THREADS) Q[e] = mq[e / N * LD + e % N] * inv;
}

// O = U Q (tall) or Q U (wide) over four sub-tiles, and its use.
// A wavefront works alone on its sub-tile: U goes to LDS, 16 rows
// (columns) at a time are multiplied and replaced there by O, which is then
// read back as it lies in memory for the update of P (loaded with U).
// Measured: the update of 448 rank-16 matrices, 671 MB: 130 us, 5.2 TB/s, the
// bound.  14 rank-64 matrices, 84 MB: 35 us, of which the full products in fp64
// (16 tiles a sub-tile) take 13.  At NT = 4 the momentum forms spill 16 to 21 of 256
// registers (P, U and the sums of a sub-tile at once).
template <typename T, int NT, int MODE>
__global__ __launch_bounds__(256, NT <= 2 ? 3 : 2) void orth_apply_kernel(const OrthArgs a) {
  constexpr int N = 16 * NT, LD = N + 2, S = N / 4;
  __shared__ __attribute__((aligned(16))) float us[4][kRegion];
  __shared__ double mq[N * LD];
  int b;
  const OrthGroup& g = my_group(a, APPLY, b);
  const int mat = b / g.subs;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, c = lane & 15;
  T* const P = static_cast<T*>(g.P);
  const double lrs = a.lr * (double)g.scale;
  float* const u = us[w];
  const double* Q = g.Q + (int64_t)mat * N * N;
#pragma unroll
  for (int i = 0; i < N * N / 256; ++i) {
    const int e = 256 * i + threadIdx.x;
    mq[e / N * LD + e % N] = Q[e];
  }
  __syncthreads();
  const SubTile st(g, mat, (b % g.subs) * 4 + w);
  if (st.len <= 0) return;
  auto body = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    f32x4 p[kVecs];
    if constexpr (MODE != ORTH) st.load<FULL>(g, static_cast<const T*>(P), p);
    load_u<T, MODE, false, FULL>(a, g, st, u);
    wave_sync();
    if (!g.wide) {
      // lane 16 q + c reads row c, short indices S q .. S q + S - 1, and ends with rows 4 v + q,
      // short indices NT c .. NT c + NT - 1
      for (int k = 0; k < st.len; k += 16) {
        float x[S];
#pragma unroll
        for (int s = 0; s < S; ++s) x[s] = S * q + s < g.r ? u[(k + c) * g.pitch + S * q + s] : 0.0f;
        f64x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f64x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int label = 16 * (s % NT) + 4 * q + s / NT;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)x[s], mq[label * LD + 16 * t + c], acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (NT * c + t < g.r) u[(k + 4 * v + q) * g.pitch + NT * c + t] = (float)acc[t][v];
      }
    } else {
      // lane 16 q + c reads column c of the rows with labels 4 s + q, and ends with that column of
      // the rows with labels 16 t + 4 v + q
      for (int k = 0; k < st.len; k += 16) {
        float x[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int row = NT * (4 * (s % 4) + q) + s / 4;
          x[s] = row < g.r ? u[row * g.pitch + k + c] : 0.0f;
        }
        f64x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f64x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[t] = __builtin_amdgcn_mfma_f64_16x16x4f64(mq[(16 * t + c) * LD + 4 * s + q], (double)x[s], acc[t], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int row = NT * (4 * v + q) + t;
            if (row < g.r) u[row * g.pitch + k + c] = (float)acc[t][v];
          }
      }
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      int row, col;
      st.at(g, j, row, col);
      f32x4 o = f32x4{0, 0, 0, 0};
      if (4 * (64 * j + lane) < st.total) o = get4(g, u, row, col);
#pragma unroll
      for (int v = 0; v < 4; ++v) p[j][v] = MODE == ORTH ? o[v] : (float)fma(a.decay, (double)p[j][v], -lrs * (double)o[v]);
    }
    st.store<FULL>(g, P, p);
  };
  if (st.len == g.sub) body(std::true_type{});
  else body(std::false_type{});
}

template <typename T, int NT, int MODE>
hipError_t launch_orth(const OrthArgs& a, const int64_t (&blocks)[3], hipStream_t st) {
  {
    TraceScope ts("orth_gram", st);
    hipLaunchKernelGGL((orth_gram_kernel<T, NT, MODE>), dim3((unsigned)blocks[GRAM]), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  {
    TraceScope ts("orth_steps", st);
    hipLaunchKernelGGL((orth_steps_kernel<NT>), dim3((unsigned)blocks[STEPS]), dim3(NT >= 3 ? 1024 : 256 * NT), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  TraceScope ts("orth_apply", st);
  hipLaunchKernelGGL((orth_apply_kernel<T, NT, MODE>), dim3((unsigned)blocks[APPLY]), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <typename T, int NT>
hipError_t launch_orth_mode(int mode, const OrthArgs& a, const int64_t (&blocks)[3], hipStream_t st) {
  return mode == ORTH ? launch_orth<T, NT, ORTH>(a, blocks, st)
                      : mode == PLAIN ? launch_orth<T, NT, PLAIN>(a, blocks, st) : launch_orth<T, NT, NESTEROV>(a, blocks, st);
}
template <typename T>
hipError_t launch_orth_nt(int nt, int mode, const OrthArgs& a, const int64_t (&blocks)[3], hipStream_t st) {
  switch (nt) {
    case 1: return launch_orth_mode<T, 1>(mode, a, blocks, st);
    case 2: return launch_orth_mode<T, 2>(mode, a, blocks, st);
    case 3: return launch_orth_mode<T, 3>(mode, a, blocks, st);
    default: return launch_orth_mode<T, 4>(mode, a, blocks, st);
  }
}

// ---------------------------------------------------------------------------
// Checks of the entry points.
// ---------------------------------------------------------------------------
struct Shape {
  int64_t n, r, chunks, nt;
  int32_t sub, sub_log2, pitch, nsub;
  size_t part, q;  // workspace bytes
};
// most: sub-tiles per wavefront of a block that forms U^T U, at most
Shape shape_of(const lora_orth_mat& m, int most = 4) {
  Shape s;
  s.n = m.rows > m.cols ? m.rows : m.cols;
  s.r = m.rows > m.cols ? m.cols : m.rows;
  s.nt = cdiv(s.r, 16);
  // as much of the long side as kSub elements hold: a multiple of 16 rows of a tall matrix, a
  // power of two (16 at least) of columns of a wide one.  LDS rows are padded against bank
  // conflicts, to 16 bytes where vectors of four do not run over row ends.
  s.sub_log2 = 0;
  if (m.cols > m.rows) {
    s.sub_log2 = 4;
    while (s.sub_log2 < 8 && (2 << s.sub_log2) * s.r <= kSub) ++s.sub_log2;
    s.sub = 1 << s.sub_log2;
    s.pitch = s.sub + 4;
  } else {
    s.pitch = (int32_t)(s.r % 4 == 0 ? s.r + 4 : s.r | 1);
    s.sub = (int32_t)std::min<int64_t>(256, std::min(kSub / s.r, 2560 / (int64_t)s.pitch) / 16 * 16);
  }
  // more sub-tiles per block where a partial Gram matrix is larger
  s.nsub = (int32_t)std::min<int64_t>(s.nt, most);
  s.chunks = cdiv(s.n, (int64_t)4 * s.sub * s.nsub);
  s.part = (size_t)(m.count * s.chunks * (s.nt * (s.nt + 1) / 2) * 256 * 8);
  s.q = (size_t)(m.count * s.nt * s.nt * 256 * 8);
  return s;
}

// Fewer sub-tiles a block where the call would not fill the chip.
int most_sub_tiles(const lora_orth_desc* d, const lora_orth_mat* mats) {
  int most = 4;
  for (; most > 1; most /= 2) {
    int64_t blocks = 0;
    for (int i = 0; i < d->n && blocks < 256; ++i) blocks += mats[i].count * shape_of(mats[i], most).chunks;
    if (blocks >= 256) break;
  }
  return most;
}

lora_status check_orth(const lora_orth_desc* d, const lora_orth_mat* mats) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16, LORA_EDTYPE, "dtype %d is not LORA_F32 or LORA_BF16", d->dtype);
  CHECK(d->n >= 0 && (d->n == 0 || mats != nullptr), LORA_EINVAL, "%d matrices at NULL", d->n);
  CHECK(d->steps >= 1 && d->steps <= 32, LORA_EINVAL, "steps = %d is not in [1, 32]", d->steps);
  CHECK(std::isfinite(d->a) && std::isfinite(d->b) && std::isfinite(d->c), LORA_EINVAL, "a coefficient is not finite");
  CHECK(std::pow(std::fabs(d->a), d->steps) <= kMaxGrowth, LORA_EINVAL,
        "%d steps with a = %g multiply rounding errors by more than 2^44", d->steps, d->a);
  CHECK(std::isfinite(d->eps) && d->eps >= 0.0, LORA_EINVAL, "eps must be finite and not negative");
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  for (int i = 0; i < d->n; ++i) {
    const lora_orth_mat& m = mats[i];
    CHECK(m.count >= 0 && m.rows > 0 && m.cols > 0, LORA_ESHAPE, "mats[%d] is %lld x [%lld, %lld]", i, (long long)m.count,
          (long long)m.rows, (long long)m.cols);
    CHECK(m.rows <= 64 || m.cols <= 64, LORA_ESHAPE, "mats[%d]: neither side of [%lld, %lld] is at most 64", i,
          (long long)m.rows, (long long)m.cols);
    const Shape s = shape_of(m, 1);
    CHECK(m.count < kMaxMats && s.n < kMaxLong && m.count < kMaxLong / s.n, LORA_ESHAPE,
          "mats[%d]: %lld x [%lld, %lld] is too large", i, (long long)m.count, (long long)m.rows, (long long)m.cols);
    CHECK(m.reserved == 0, LORA_EINVAL, "mats[%d].reserved must be 0", i);
  }
  return LORA_OK;
}

size_t orth_bytes(const lora_orth_desc* d, const lora_orth_mat* mats) {
  Ws w(nullptr);
  const int most = most_sub_tiles(d, mats);
  for (int i = 0; i < d->n; ++i) {
    const Shape s = shape_of(mats[i], most);
    w.take(s.part);
    w.take(s.q);
  }
  return w.off;
}

// Every tensor is aligned to its type, and what is written (results, momenta,
// the workspace) overlaps nothing else, except that an orthogonalised stack
// may be exactly its input.
lora_status check_mats(const lora_orth_desc* d, const lora_orth_mat* mats, bool muon, const void* ws, size_t need) {
  struct Span {
    uintptr_t at, end;
    bool written;
    int entry;  // -1: the workspace
  };
  const size_t es = d->dtype == LORA_F32 ? 4 : 2;
  std::unique_ptr<Span[]> span(new (std::nothrow) Span[3 * (size_t)d->n + 1]);
  CHECK(span != nullptr, LORA_EINVAL, "no memory to check %d matrices", d->n);
  size_t ns = 0;
  auto add = [&](const void* p, size_t bytes, bool written, int entry) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    span[ns++] = Span{at, at + bytes, written, entry};
  };
  for (int i = 0; i < d->n; ++i) {
    const lora_orth_mat& m = mats[i];
    const size_t ne = (size_t)m.count * m.rows * m.cols;
    if (ne == 0) continue;
    CHECK(m.G && m.P, LORA_EINVAL, "mats[%d]: G or P is NULL", i);
    CHECK((m.M != nullptr) == muon, LORA_EINVAL, "mats[%d]: M is %s", i, muon ? "NULL" : "not used here and must be NULL");
    CHECK(aligned(m.G, es) && aligned(m.P, es) && aligned(m.M, 4), LORA_EALIGN, "mats[%d]: a pointer is not aligned", i);
    CHECK(std::isfinite(m.scale), LORA_EINVAL, "mats[%d].scale is not finite", i);
    add(m.P, ne * es, true, i);
    if (m.G != m.P || muon) add(m.G, ne * es, false, i);
    if (muon) add(m.M, ne * 4, true, i);
  }
  if (need > 0) add(ws, need, true, -1);
  std::sort(span.get(), span.get() + ns, [](const Span& x, const Span& y) { return x.at < y.at; });
  uintptr_t read_end = 0, written_end = 0;  // furthest ends of the spans that begin earlier
  for (size_t k = 0; k < ns; ++k) {
    const Span& x = span[k];
    CHECK(x.at >= written_end && (!x.written || x.at >= read_end), LORA_EUNSUPPORTED,
          "a tensor of mats[%d] overlaps another that is written", x.entry < 0 && k > 0 ? span[k - 1].entry : x.entry);
    uintptr_t& end = x.written ? written_end : read_end;
    if (x.end > end) end = x.end;
  }
  return LORA_OK;
}

lora_status run_orth(const lora_orth_desc* d, const lora_orth_mat* mats, int mode, OrthArgs a, void* ws, hipStream_t st) {
  a.steps = d->steps;
  a.a = d->a;
  a.b = d->b;
  a.c = d->c;
  a.eps = d->eps;
  // one set of three launches for all stacks with the same number of tiles, kMaxGroups at a time
  const int most = most_sub_tiles(d, mats);
  for (int nt = 1; nt <= 4; ++nt) {
    int64_t blocks[3] = {0, 0, 0};
    a.ngroups = 0;
    Ws w(ws);
    auto flush = [&]() -> hipError_t {
      if (a.ngroups == 0) return hipSuccess;
      for (int k = 0; k < 3; ++k)
        for (int i = a.ngroups; i < kMaxGroups; ++i) a.first[k][i] = INT32_MAX;
      const hipError_t e = d->dtype == LORA_F32 ? launch_orth_nt<float>(nt, mode, a, blocks, st)
                                                : launch_orth_nt<uint16_t>(nt, mode, a, blocks, st);
      a.ngroups = 0;
      blocks[GRAM] = blocks[STEPS] = blocks[APPLY] = 0;
      return e;
    };
    for (int i = 0; i < d->n; ++i) {
      const lora_orth_mat& m = mats[i];
      const Shape s = shape_of(m, most);
      const int64_t subs = cdiv(s.n, 4 * s.sub), add[3] = {m.count * s.chunks, m.count, m.count * subs};
      double* part = static_cast<double*>(w.take(s.part));
      double* Q = static_cast<double*>(w.take(s.q));
      if (s.nt != nt || m.count == 0) continue;
      if (a.ngroups == kMaxGroups || blocks[APPLY] + add[APPLY] > kMaxBlocks || blocks[STEPS] + add[STEPS] > kMaxMats)
        LAUNCH(flush());
      for (int k = 0; k < 3; ++k) {
        a.first[k][a.ngroups] = (int32_t)blocks[k];
        blocks[k] += add[k];
      }
      OrthGroup& g = a.g[a.ngroups++];
      g.wide = m.cols > m.rows;
      g.G = m.G;
      g.M = m.M;
      g.P = m.P;
      g.part = part;
      g.Q = Q;
      g.n = (int32_t)s.n;
      g.r = (int32_t)s.r;
      g.chunks = (int32_t)s.chunks;
      g.sub = s.sub;
      g.sub_log2 = s.sub_log2;
      g.pitch = s.pitch;
      g.nsub = s.nsub;
      g.inv_r = (uint32_t)cdiv((int64_t)1 << 20, s.r);
      g.vec_lds = g.wide || s.r % 4 == 0;
      g.subs = (int32_t)subs;
      g.scale = m.scale;
    }
    LAUNCH(flush());
  }
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_orth_workspace_size(const lora_orth_desc* d, const lora_orth_mat* mats, size_t* bytes) {
  TRY(check_orth(d, mats));
  if (bytes) *bytes = orth_bytes(d, mats);
  return LORA_OK;
}

lora_status lora_orthogonalize(const lora_orth_desc* d, const lora_orth_mat* mats, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_orth(d, mats));
  const size_t need = orth_bytes(d, mats);
  TRY(check_ws(ws, ws_bytes, need));
  TRY(check_mats(d, mats, false, ws, need));
  OrthArgs a{};
  return run_orth(d, mats, ORTH, a, ws, static_cast<hipStream_t>(stream));
}

lora_status lora_muon_step(const lora_muon_desc* d, const lora_orth_mat* mats, void* ws, size_t ws_bytes, void* stream) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  TRY(check_orth(&d->orth, mats));
  CHECK(std::isfinite(d->lr) && std::isfinite(d->weight_decay) && std::isfinite(d->momentum), LORA_EINVAL,
        "lr, momentum or weight_decay is not finite");
  CHECK(d->nesterov == 0 || d->nesterov == 1, LORA_EINVAL, "nesterov = %d is not 0 or 1", d->nesterov);
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  const size_t need = orth_bytes(&d->orth, mats);
  TRY(check_ws(ws, ws_bytes, need));
  TRY(check_mats(&d->orth, mats, true, ws, need));
  OrthArgs a{};
  a.mu = (float)d->momentum;
  a.lr = d->lr;
  a.decay = 1.0 - d->lr * d->weight_decay;
  return run_orth(&d->orth, mats, d->nesterov ? NESTEROV : PLAIN, a, ws, static_cast<hipStream_t>(stream));
}

}  // extern "C"
