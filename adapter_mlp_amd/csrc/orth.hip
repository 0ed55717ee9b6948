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

#include "abi.hpp"
#include "common.hpp"

namespace lora {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 512;     // long-side elements per block of the passes over U
constexpr int kMaxGroups = 24;  // stacks per launch (their table is a kernel argument)

// One stack of `count` matrices with the same shape.
struct OrthGroup {
  const void* G;
  float* M;     // momentum (nullptr: U = G)
  void* P;      // result, or the parameter that takes it
  double* part; // [count][chunks][NT (NT + 1) / 2][4][64] partial U^T U
  double* Q;    // [count][16 NT][16 NT]
  int32_t n, r; // long and short side
  int32_t wide; // 1: [r, n], 0: [n, r]
  int32_t count, chunks;
  int32_t blk0; // first block of the group in the passes over U
  int32_t mat0; // first block of the group in the r x r steps
  float scale;
};

struct OrthArgs {
  OrthGroup g[kMaxGroups];
  int32_t ngroups, nesterov;
  int32_t steps, muon;
  float mu;
  double a, b, c, eps;
  double decay, lr;  // P <- decay P - lr scale O
};

// Up to four consecutive elements with no more alignment than their own.
template <typename T, int N>
struct Run;
template <int N>
struct Run<float, N> {
  typedef float vec __attribute__((ext_vector_type(N), aligned(4)));
  static __device__ __forceinline__ void load(const float* p, float (&x)[N]) {
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    vec v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i];
    *reinterpret_cast<vec*>(p) = v;
  }
};
template <>
struct Run<float, 1> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[1]) { x[0] = *p; }
  static __device__ __forceinline__ void store(float* p, const float (&x)[1]) { *p = x[0]; }
};
template <int N>
struct Run<uint16_t, N> {
  typedef uint16_t vec __attribute__((ext_vector_type(N), aligned(2)));
  static __device__ __forceinline__ void load(const uint16_t* p, float (&x)[N]) {
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = bf2f(v[i]);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[N]) {
    vec v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (uint16_t)f2bf(x[i]);
    *reinterpret_cast<vec*>(p) = v;
  }
};
template <>
struct Run<uint16_t, 1> {
  static __device__ __forceinline__ void load(const uint16_t* p, float (&x)[1]) { x[0] = bf2f(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[1]) { *p = (uint16_t)f2bf(x[0]); }
};

// A vector type of three would be read and written as four.
template <typename T>
struct Run3 {
  static __device__ __forceinline__ void load(const T* p, float (&x)[3]) {
    float a[2], b[1];
    Run<T, 2>::load(p, a);
    Run<T, 1>::load(p + 2, b);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
  }
  static __device__ __forceinline__ void store(T* p, const float (&x)[3]) {
    const float a[2] = {x[0], x[1]}, b[1] = {x[2]};
    Run<T, 2>::store(p, a);
    Run<T, 1>::store(p + 2, b);
  }
};

template <>
struct Run<float, 3> : Run3<float> {};
template <>
struct Run<uint16_t, 3> : Run3<uint16_t> {};

// N consecutive elements of which the first `valid` exist (the rest read 0).
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* p, int valid, float (&x)[N]) {
  if constexpr (N > 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      float y[4];
      load_run<T, 4>(p + j, valid - j, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j + i] = y[i];
    }
  } else if (valid >= N) {
    Run<T, N>::load(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float y[1] = {0.0f};
      if (i < valid) Run<T, 1>::load(p + i, y);
      x[i] = y[0];
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_run(T* p, int valid, const float (&x)[N]) {
  if (valid >= N) {
    Run<T, N>::store(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y[1] = {x[i]};
      if (i < valid) Run<T, 1>::store(p + i, y);
    }
  }
}

// U at elements o .. o + N - 1 of a stack.  FIRST: the momentum is brought up
// to date (M <- mu M + G) and stored; later passes read the new one.
template <typename T, int N, bool FIRST>
__device__ __forceinline__ void load_u(const OrthArgs& a, const OrthGroup& g, int64_t o, int valid, float (&u)[N]) {
  const T* G = static_cast<const T*>(g.G);
  if (!a.muon) {
    load_run<T, N>(G + o, valid, u);
    return;
  }
  float m[N], x[N];
  load_run<float, N>(g.M + o, valid, m);
  if (FIRST || a.nesterov) load_run<T, N>(G + o, valid, x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (FIRST) m[i] = fmaf(a.mu, m[i], x[i]);
    u[i] = a.nesterov ? fmaf(a.mu, m[i], x[i]) : m[i];
  }
  if (FIRST) store_run<float, N>(g.M + o, valid, m);
}

// The group of block b (first blocks blk0 or mat0 ascending).
__device__ __forceinline__ int find_group(const OrthArgs& a, int b, bool mats) {
  int k = 0;
  for (int i = 1; i < a.ngroups; ++i)
    if (b >= (mats ? a.g[i].mat0 : a.g[i].blk0)) k = i;
  return __builtin_amdgcn_readfirstlane(k);
}

// Partial U^T U of one matrix over kChunk of its long side: four wavefronts
// share the chunk.  An operand of tile t holds, in lane 16 q + c, U at long
// index k + q (any assignment of the four k to the lane groups gives the same
// sum) and short index NT c + t, and serves as both sides of the product.
// Only the tiles on and above the diagonal are formed.
template <typename T, int NT>
__global__ __launch_bounds__(256) void orth_gram_kernel(const OrthArgs a) {
  constexpr int NP = NT * (NT + 1) / 2;
  __shared__ double red[3][NP * 4 * 64];
  const OrthGroup& g = a.g[find_group(a, blockIdx.x, false)];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, c = lane & 15;
  const int b = (int)blockIdx.x - g.blk0, mat = b / g.chunks, chunk = b % g.chunks;
  const int64_t base = (int64_t)mat * g.n * g.r;
  const int k0 = chunk * kChunk + w * (kChunk / 4);
  const int left = g.n - k0;
  const int len = left < kChunk / 4 ? left : kChunk / 4;
  f64x4 acc[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) acc[i] = f64x4{0, 0, 0, 0};
  auto mma = [&](const float (&u)[NT]) {
    double d[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) d[t] = (double)u[t];
    int i = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int s = t; s < NT; ++s, ++i) acc[i] = __builtin_amdgcn_mfma_f64_16x16x4f64(d[t], d[s], acc[i], 0, 0, 0);
  };
  if (!g.wide) {
    constexpr int UN = NT == 1 ? 8 : 4;
    const int valid = g.r - NT * c;
    for (int k = 0; k < len; k += 4 * UN) {
      float u[UN][NT];
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        const int kk = k + 4 * j + q;
        load_u<T, NT, true>(a, g, base + (int64_t)(k0 + kk) * g.r + NT * c, kk < len ? valid : 0, u[j]);
      }
#pragma unroll
      for (int j = 0; j < UN; ++j) mma(u[j]);
    }
  } else {
    constexpr int UN = NT == 1 ? 4 : NT == 2 ? 2 : 1;
    for (int k = 0; k < len; k += 16 * UN) {
      float u[UN][NT][4];
#pragma unroll
      for (int j = 0; j < UN; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int kk = k + 16 * j + 4 * q, i = NT * c + t;
          load_u<T, 4, true>(a, g, base + (int64_t)i * g.n + k0 + kk, i < g.r ? len - kk : 0, u[j][t]);
        }
#pragma unroll
      for (int j = 0; j < UN; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float x[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) x[t] = u[j][t][v];
          mma(x);
        }
    }
  }
  if (w > 0)
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[w - 1][(i * 4 + v) * 64 + lane] = acc[i][v];
  __syncthreads();
  if (w == 0) {
    double* out = g.part + ((int64_t)mat * g.chunks + chunk) * (NP * 256);
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int o = (i * 4 + v) * 64 + lane;
        out[o] = acc[i][v] + red[0][o] + red[1][o] + red[2][o];
      }
  }
}

// The steps of one matrix on its r x r Gram matrix, one block of four
// wavefronts.  Per step: p = a I + b G + c G G; V = G p and Q <- Q p; G <- V p.
// All matrices are symmetric, so both operands of a product are read along
// rows; rows are 16 NT + 2 doubles apart, which spreads the 16 rows of a
// fragment read over all banks.
template <int NT>
__global__ __launch_bounds__(256) void orth_steps_kernel(const OrthArgs a) {
  constexpr int N = 16 * NT, LD = N + 2, NP = NT * (NT + 1) / 2, TILES = NT * NT, PER = (TILES + 3) / 4;
  __shared__ double mg[N * LD], mp[N * LD], mv[N * LD], mq[N * LD];
  const OrthGroup& g = a.g[find_group(a, blockIdx.x, true)];
  const int mat = (int)blockIdx.x - g.mat0;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, c = lane & 15;

  // sum of the chunks, ascending; element (i, v, lane) is row 16 t + 4 v + q, column 16 s + c
  const double* part = g.part + (int64_t)mat * g.chunks * (NP * 256);
  for (int e = threadIdx.x; e < NP * 256; e += 256) {
    double s = 0.0;
#pragma unroll 8
    for (int k = 0; k < g.chunks; ++k) s += part[(int64_t)k * (NP * 256) + e];
    const int i = e >> 8, v = (e >> 6) & 3, l = e & 63;
    int t = 0, first = 0;
    while (i >= first + NT - t) first += NT - t++;
    const int row = 16 * t + 4 * v + (l >> 4), col = 16 * (t + i - first) + (l & 15);
    mg[row * LD + col] = s;
    if (t != t + i - first) mg[col * LD + row] = s;
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < N; ++i) trace += mg[i * LD + i];
  const double inv = 1.0 / (sqrt(trace) + a.eps);
  __syncthreads();
  for (int e = threadIdx.x; e < N * N; e += 256) {
    const int row = e / N, col = e % N;
    mg[row * LD + col] *= inv * inv;
    mq[row * LD + col] = row == col ? 1.0 : 0.0;
  }
  __syncthreads();

  f64x4 x[PER], y[PER];
  // this wavefront's tiles of the product A B
  auto product = [&](const double* A, const double* B, f64x4 (&o)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      o[j] = f64x4{0, 0, 0, 0};
      const int tile = w + 4 * j;
      if (tile < TILES) {
        const double* ar = A + (16 * (tile / NT) + c) * LD + q;
        const double* br = B + (16 * (tile % NT) + c) * LD + q;
#pragma unroll
        for (int s = 0; s < N / 4; ++s) o[j] = __builtin_amdgcn_mfma_f64_16x16x4f64(ar[4 * s], br[4 * s], o[j], 0, 0, 0);
      }
    }
  };
  // f(row, column, element) over this wavefront's tiles
  auto each = [&](f64x4 (&o)[PER], auto f) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int tile = w + 4 * j;
      if (tile < TILES)
#pragma unroll
        for (int v = 0; v < 4; ++v) f(16 * (tile / NT) + 4 * v + q, 16 * (tile % NT) + c, o[j][v]);
    }
  };
  for (int k = 0; k < a.steps; ++k) {
    product(mg, mg, x);
    each(x, [&](int row, int col, double s) {
      mp[row * LD + col] = fma(a.c, s, a.b * mg[row * LD + col]) + (row == col ? a.a : 0.0);
    });
    __syncthreads();
    const bool last = k + 1 == a.steps;
    product(mq, mp, x);
    if (!last) product(mg, mp, y);
    __syncthreads();
    each(x, [&](int row, int col, double s) { mq[row * LD + col] = s; });
    if (last) break;
    each(y, [&](int row, int col, double s) { mv[row * LD + col] = s; });
    __syncthreads();
    product(mv, mp, x);
    each(x, [&](int row, int col, double s) { mg[row * LD + col] = s; });
    __syncthreads();
  }
  __syncthreads();
  double* Q = g.Q + (int64_t)mat * N * N;
  for (int e = threadIdx.x; e < N * N; e += 256) Q[e] = mq[e / N * LD + e % N] * inv;
}

// O = U Q (tall) or Q U (wide) over kChunk of the long side, and its use.
template <typename T, int NT>
__global__ __launch_bounds__(256) void orth_apply_kernel(const OrthArgs a) {
  constexpr int N = 16 * NT, LD = N + 2, S = N / 4;
  __shared__ double mq[N * LD];
  const OrthGroup& g = a.g[find_group(a, blockIdx.x, false)];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, c = lane & 15;
  const int b = (int)blockIdx.x - g.blk0, mat = b / g.chunks, chunk = b % g.chunks;
  const double* Q = g.Q + (int64_t)mat * N * N;
  for (int e = threadIdx.x; e < N * N; e += 256) mq[e / N * LD + e % N] = Q[e];
  __syncthreads();
  const int64_t base = (int64_t)mat * g.n * g.r;
  T* const P = static_cast<T*>(g.P);
  const double lrs = a.lr * (double)g.scale;
  auto use = [&](double o, float p) { return a.muon ? (float)fma(a.decay, (double)p, -lrs * o) : (float)o; };
  const int k1 = chunk * kChunk + kChunk < g.n ? chunk * kChunk + kChunk : g.n;
  if (!g.wide) {
    // 16 rows a time: lane 16 q + c holds row c, short indices S q .. S q + S - 1, and ends with
    // rows 4 v + q, short indices NT c .. NT c + NT - 1
    for (int k = chunk * kChunk + 16 * w; k < k1; k += 64) {
      float u[S];
      load_u<T, S, false>(a, g, base + (int64_t)(k + c) * g.r + S * q, k + c < k1 ? g.r - S * q : 0, u);
      f64x4 acc[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = f64x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int i = S * q + s, label = 16 * (i % NT) + i / NT;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)u[s], mq[label * LD + 16 * t + c], acc[t], 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = k + 4 * v + q, valid = row < k1 ? g.r - NT * c : 0;
        const int64_t o = base + (int64_t)row * g.r + NT * c;
        float p[NT];
        if (a.muon) load_run<T, NT>(P + o, valid, p);
#pragma unroll
        for (int t = 0; t < NT; ++t) p[t] = use(acc[t][v], p[t]);
        store_run<T, NT>(P + o, valid, p);
      }
    }
  } else {
    // 64 columns a time: lane 16 q + c holds columns 4 c .. 4 c + 3 of the rows with labels
    // 4 s + q, and ends with the same columns of the rows with labels 16 t + 4 v + q
    for (int k = chunk * kChunk + 64 * w; k < k1; k += 256) {
      const int col = k + 4 * c, valid = k1 - col;
      float u[S][4];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int label = 4 * s + q, i = NT * (label % 16) + label / 16;
        load_u<T, 4, false>(a, g, base + (int64_t)i * g.n + col, i < g.r ? valid : 0, u[s]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f64x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f64x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const double m = mq[(16 * t + c) * LD + 4 * s + q];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f64_16x16x4f64(m, (double)u[s][j], acc[j], 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = NT * (4 * v + q) + t;
          const int64_t o = base + (int64_t)i * g.n + col;
          float p[4];
          if (a.muon) load_run<T, 4>(P + o, i < g.r ? valid : 0, p);
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = use(acc[j][v], p[j]);
          store_run<T, 4>(P + o, i < g.r ? valid : 0, p);
        }
      }
    }
  }
}

template <typename T, int NT>
hipError_t launch_orth(const OrthArgs& a, int blocks, int mats, hipStream_t st) {
  {
    TraceScope ts("orth_gram", st);
    hipLaunchKernelGGL((orth_gram_kernel<T, NT>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  {
    TraceScope ts("orth_steps", st);
    hipLaunchKernelGGL((orth_steps_kernel<NT>), dim3((unsigned)mats), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  TraceScope ts("orth_apply", st);
  hipLaunchKernelGGL((orth_apply_kernel<T, NT>), dim3((unsigned)blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <typename T>
hipError_t launch_orth_nt(int nt, const OrthArgs& a, int blocks, int mats, hipStream_t st) {
  switch (nt) {
    case 1: return launch_orth<T, 1>(a, blocks, mats, st);
    case 2: return launch_orth<T, 2>(a, blocks, mats, st);
    case 3: return launch_orth<T, 3>(a, blocks, mats, st);
    default: return launch_orth<T, 4>(a, blocks, mats, st);
  }
}

// ---------------------------------------------------------------------------
// Checks of the entry points.
// ---------------------------------------------------------------------------
struct Shape {
  int64_t n, r, chunks, nt;
  size_t part, q;  // workspace bytes
};
Shape shape_of(const lora_orth_mat& m) {
  Shape s;
  s.n = m.rows > m.cols ? m.rows : m.cols;
  s.r = m.rows > m.cols ? m.cols : m.rows;
  s.chunks = cdiv(s.n, kChunk);
  s.nt = cdiv(s.r, 16);
  s.part = (size_t)(m.count * s.chunks * (s.nt * (s.nt + 1) / 2) * 256 * 8);
  s.q = (size_t)(m.count * s.nt * s.nt * 256 * 8);
  return s;
}

lora_status check_orth(const lora_orth_desc* d, const lora_orth_mat* mats) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16, LORA_EDTYPE, "dtype %d is not LORA_F32 or LORA_BF16", d->dtype);
  CHECK(d->n >= 0 && (d->n == 0 || mats != nullptr), LORA_EINVAL, "%d matrices at NULL", d->n);
  CHECK(d->steps >= 1 && d->steps <= 32, LORA_EINVAL, "steps = %d is not in [1, 32]", d->steps);
  CHECK(std::isfinite(d->a) && std::isfinite(d->b) && std::isfinite(d->c), LORA_EINVAL, "a coefficient is not finite");
  CHECK(std::isfinite(d->eps) && d->eps >= 0.0, LORA_EINVAL, "eps must be finite and not negative");
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  for (int i = 0; i < d->n; ++i) {
    const lora_orth_mat& m = mats[i];
    CHECK(m.count >= 0 && m.rows > 0 && m.cols > 0, LORA_ESHAPE, "mats[%d] is %lld x [%lld, %lld]", i, (long long)m.count,
          (long long)m.rows, (long long)m.cols);
    CHECK(m.rows <= 64 || m.cols <= 64, LORA_ESHAPE, "mats[%d]: neither side of [%lld, %lld] is at most 64", i,
          (long long)m.rows, (long long)m.cols);
    const Shape s = shape_of(m);
    CHECK(s.n < ((int64_t)1 << 30) && m.count <= ((int64_t)1 << 30) / s.chunks, LORA_ESHAPE,
          "mats[%d]: %lld x [%lld, %lld] is too large", i, (long long)m.count, (long long)m.rows, (long long)m.cols);
    CHECK(m.reserved == 0, LORA_EINVAL, "mats[%d].reserved must be 0", i);
  }
  return LORA_OK;
}

size_t orth_bytes(const lora_orth_desc* d, const lora_orth_mat* mats) {
  Ws w(nullptr);
  for (int i = 0; i < d->n; ++i) {
    const Shape s = shape_of(mats[i]);
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

lora_status run_orth(const lora_orth_desc* d, const lora_orth_mat* mats, OrthArgs a, void* ws, hipStream_t st) {
  a.steps = d->steps;
  a.a = d->a;
  a.b = d->b;
  a.c = d->c;
  a.eps = d->eps;
  // one set of three launches for all stacks with the same number of tiles, kMaxGroups at a time
  for (int nt = 1; nt <= 4; ++nt) {
    int64_t blocks = 0, nmat = 0;
    a.ngroups = 0;
    Ws w(ws);
    auto flush = [&]() -> hipError_t {
      if (a.ngroups == 0) return hipSuccess;
      const hipError_t e = d->dtype == LORA_F32 ? launch_orth_nt<float>(nt, a, (int)blocks, (int)nmat, st)
                                                : launch_orth_nt<uint16_t>(nt, a, (int)blocks, (int)nmat, st);
      a.ngroups = 0;
      blocks = nmat = 0;
      return e;
    };
    for (int i = 0; i < d->n; ++i) {
      const lora_orth_mat& m = mats[i];
      const Shape s = shape_of(m);
      double* part = static_cast<double*>(w.take(s.part));
      double* Q = static_cast<double*>(w.take(s.q));
      if (s.nt != nt || m.count == 0) continue;
      if (a.ngroups == kMaxGroups || blocks + m.count * s.chunks > ((int64_t)1 << 30)) LAUNCH(flush());
      OrthGroup& g = a.g[a.ngroups++];
      g.G = m.G;
      g.M = m.M;
      g.P = m.P;
      g.part = part;
      g.Q = Q;
      g.n = (int32_t)s.n;
      g.r = (int32_t)s.r;
      g.wide = m.cols > m.rows;
      g.count = (int32_t)m.count;
      g.chunks = (int32_t)s.chunks;
      g.blk0 = (int32_t)blocks;
      g.mat0 = (int32_t)nmat;
      g.scale = m.scale;
      blocks += m.count * s.chunks;
      nmat += m.count;
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
  return run_orth(d, mats, a, ws, static_cast<hipStream_t>(stream));
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
  a.muon = 1;
  a.nesterov = d->nesterov;
  a.mu = (float)d->momentum;
  a.lr = d->lr;
  a.decay = 1.0 - d->lr * d->weight_decay;
  return run_orth(&d->orth, mats, a, ws, static_cast<hipStream_t>(stream));
}

}  // extern "C"
