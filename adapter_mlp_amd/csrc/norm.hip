// Norms before and after a block, with the block's gate and the residual:
//   p  = Y rms(Y)^-1 (o + w_post)  (or Y)        the block's output, normed
//   R' = a R + b g p                             the new residual
//   X  = R' rms(R')^-1 (o + w_pre)               the next block's input
// rms(v)^2 = mean(v^2) + eps over the row, o = 1 or 0, g a gate per column,
// per row or per element, and the gradients of all of it in one pass.
//
// Both directions are bound by HBM: 2 to 4 operands of [T, H] forward, 3 to 6
// backward, against some ten operations an element.  A row lives in the
// registers of one wavefront (H <= 1024) or one block, so every operand is
// read once; the row sums are the only exchange between threads.  Sums,
// norms and everything between a load and a store are fp32: X is formed from
// the unrounded R', so each output carries one rounding.
#include <algorithm>
#include <cmath>

#include "abi.hpp"
#include "common.hpp"

namespace lora {
namespace {

enum { GATE_NONE = LORA_GATE_NONE, GATE_COL = LORA_GATE_COL, GATE_ROW = LORA_GATE_ROW, GATE_ELEM = LORA_GATE_ELEM };

struct NormArgs {
  int64_t T;
  int32_t H, gate;
  float eps, res_scale, branch_scale, offset;
  const void *R, *Y, *g, *w_post, *w_pre;  // forward inputs (backward: R is the new residual)
  void *out, *X;                           // forward outputs
  const void *dR, *dX;                     // backward inputs
  void *dR_out, *dY, *dg;                  // backward outputs (dg: per-row and per-element gates)
  // per-block column sums of the parameter gradients, [blocks, H] each (nullptr: not wanted)
  float *p_pre, *p_post, *p_gate;
};

// VEC consecutive elements of a row as they are loaded: 16 bytes of
// activations (VEC = 8 bf16 or 4 fp32), or one element where the row length
// or a pointer does not allow that.
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<uint16_t, 8> {
  u32x4 v;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float operator[](int i) const { return (i & 1) ? hi_bf(v[i >> 1]) : lo_bf(v[i >> 1]); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* f) {
    const u32x4 w = {pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])};
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  }
};
template <int VEC>
struct Vec<float, VEC> {
  static constexpr int W = VEC < 4 ? VEC : 4;
  typedef float fv __attribute__((ext_vector_type(W)));
  fv v[VEC / W];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
#pragma unroll
    for (int k = 0; k < VEC / W; ++k) v[k] = *reinterpret_cast<const fv*>(static_cast<const float*>(p) + i + k * W);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < VEC / W; ++k) v[k] = fv(0.0f);
  }
  __device__ __forceinline__ float operator[](int i) const { return v[i / W][i % W]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* f) {
#pragma unroll
    for (int k = 0; k < VEC / W; ++k) {
      fv w;
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = f[k * W + j];
      *reinterpret_cast<fv*>(static_cast<float*>(p) + i + k * W) = w;
    }
  }
};

__device__ __forceinline__ float load1(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float f) { *p = (uint16_t)f2bf(f); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }

// Sums of N values over the TPR threads of a row, in a fixed order: a
// butterfly in the wavefront, then the wavefronts in ascending order through
// LDS.  `turn` alternates two LDS areas, so one barrier per sum is enough: an
// area is rewritten only after the barrier of the sum in between, which every
// thread passes after it has read.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[N][TPR / 64], int& turn) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[turn][i][w] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lds[turn][i][0];
#pragma unroll
      for (int k = 1; k < TPR / 64; ++k) v[i] += lds[turn][i][k];
    }
    turn ^= 1;
  }
}

template <int TPR>
constexpr int norm_block() {
  return TPR < 256 ? 256 : TPR;
}

// What fits the registers: a block of 1024 threads has 128 a thread, fewer
// threads 256 and two blocks a CU.  PREFETCH: the next row's operands are
// loaded before this row's sums are waited for.  KEEP: the weights stay in
// registers instead of being read again (from L2) for every row.
template <typename TA, int VEC, int TPR, int NV>
constexpr bool norm_prefetch(bool bwd) {
  return bwd ? (VEC * NV <= 16 && TPR < 1024 && (sizeof(TA) == 2 || VEC * NV == 8)) : (TPR < 1024 || sizeof(TA) == 2);
}
template <typename TA, int VEC, int TPR, int NV>
constexpr bool norm_keep(bool bwd) {
  return norm_prefetch<TA, VEC, TPR, NV>(bwd);
}

// Thread tx of a row's TPR threads owns the vectors tx, tx + TPR, ... (NV of
// them) in every row it meets.
// Measured: 8192 bf16 rows of 4096 with post-norm, column gate and pre-norm,
// 268 MB: 44 to 47 us, 5.7 to 6.1 TB/s (a large copy: 4.85 TB/s, half of it written here as
// there; operands that were just read or written partly come from the last-level
// cache).  One row of 4096: 3 us, the round trips of its loads and one sum.
template <typename TA, typename TP, int VEC, int TPR, int NV>
__global__ __launch_bounds__(norm_block<TPR>()) void norm_fwd_kernel(const NormArgs a) {
  constexpr bool PREFETCH = norm_prefetch<TA, VEC, TPR, NV>(false), KEEP = norm_keep<TA, VEC, TPR, NV>(false);
  __shared__ float lds[2][1][TPR / 64];
  constexpr int RPB = norm_block<TPR>() / TPR;
  const int tx = threadIdx.x % TPR;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool branch = a.Y != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const int gate = a.gate;
  int turn = 0;
  bool ok[NV];
  Vec<TP, VEC> wq[NV], wp[NV], gc[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) ok[v] = (v * TPR + tx) * VEC < H;
  auto weights = [&]() {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + tx) * VEC;
      wq[v].zero();
      wp[v].zero();
      gc[v].zero();
      if (ok[v] && post) wq[v].load(a.w_post, c);
      if (ok[v] && pre) wp[v].load(a.w_pre, c);
      if (ok[v] && gate == GATE_COL) gc[v].load(a.g, c);
    }
  };
  if constexpr (KEEP) weights();
  Vec<TA, VEC> nr[NV], ny[NV], ng[NV];
  const int64_t step = (int64_t)gridDim.x * RPB;
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t i = t * H + (v * TPR + tx) * VEC;
      nr[v].zero();
      ny[v].zero();
      ng[v].zero();
      if (t < a.T && ok[v]) {
        nr[v].load(a.R, i);
        if (branch) ny[v].load(a.Y, i);
        if (gate == GATE_ELEM) ng[v].load(a.g, i);
      }
    }
  };
  int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if constexpr (PREFETCH) fetch(t);
  for (; t < a.T; t += step) {
    if constexpr (!PREFETCH) fetch(t);
    if constexpr (!KEEP) weights();
    Vec<TA, VEC> r[NV], y[NV], ge[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      r[v] = nr[v];
      y[v] = ny[v];
      ge[v] = ng[v];
    }
    if constexpr (PREFETCH) fetch(t + step);
    float s[NV * VEC];
    if (branch) {
      float u = 1.0f;
      if (post) {
        float q[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < VEC; ++i) q[0] = fmaf(y[v][i], y[v][i], q[0]);
        row_sums<TPR, 1>(q, lds, turn);
        u = rsqrtf(fmaf(q[0], inv_h, a.eps));
      }
      float b = a.branch_scale;
      if (gate == GATE_ROW) b *= load1(static_cast<const TA*>(a.g) + t);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float p = y[v][i] * b;
          if (post) p *= u * (a.offset + wq[v][i]);
          if (gate == GATE_COL) p *= gc[v][i];
          if (gate == GATE_ELEM) p *= ge[v][i];
          s[v * VEC + i] = fmaf(a.res_scale, r[v][i], p);
        }
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (ok[v]) Vec<TA, VEC>::store(a.out, t * H + (v * TPR + tx) * VEC, s + v * VEC);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[v * VEC + i] = r[v][i];
    }
    if (pre) {
      float q[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (ok[v])
#pragma unroll
          for (int i = 0; i < VEC; ++i) q[0] = fmaf(s[v * VEC + i], s[v * VEC + i], q[0]);
      row_sums<TPR, 1>(q, lds, turn);
      const float u = rsqrtf(fmaf(q[0], inv_h, a.eps));
#pragma unroll
      for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[v * VEC + i] *= u * (a.offset + wp[v][i]);
        if (ok[v]) Vec<TA, VEC>::store(a.X, t * H + (v * TPR + tx) * VEC, s + v * VEC);
      }
    }
  }
}

// With n = R'/rms(R'), q = dX (o + w_pre), yn = Y/rms(Y), z = b g d (o + w_post):
//   d  = dR' + (q - n mean(q n)) / rms(R')      dw_pre = sum_t dX n
//   dR = a d     dg = b d p                     dw_post = sum_t b g d yn
//   dY = (z - yn mean(z yn)) / rms(Y)
// Two rounds of row sums: R'^2, q R', Y^2 together, then z Y and d p (both
// need d).  The column sums of the parameter gradients gather in the
// registers of the thread that owns the column, one slice per block, and
// norm_grad_kernel adds the slices in ascending order.
// Measured: 8192 bf16 rows of 4096 with all three gradients, 403 MB and 25 MB of
// slices: 80 us, 5.3 TB/s, and 5.8 us to add the slices.  1003 fp32 rows of 1001:
// 11.9 + 3.9 us for 24 MB, 2 TB/s.  Rows whose length is no multiple of four are
// loaded element by element (VEC = 1), and one wavefront a row makes 251 blocks
// of these, one wavefront a SIMD: too few loads in flight.
template <typename TA, typename TP, int VEC, int TPR, int NV>
__global__ __launch_bounds__(norm_block<TPR>(), TPR <= 256 ? 2 : 1) void norm_bwd_kernel(const NormArgs a) {
  constexpr bool PREFETCH = norm_prefetch<TA, VEC, TPR, NV>(true), KEEP = norm_keep<TA, VEC, TPR, NV>(true);
  constexpr int RPB = norm_block<TPR>() / TPR;
  constexpr int E = NV * VEC;
  __shared__ float lds3[2][3][TPR / 64];
  __shared__ float lds2[2][2][TPR / 64];
  const int tx = threadIdx.x % TPR;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool branch = a.dY != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool has_dr = a.dR != nullptr;
  const int gate = a.gate;
  const bool need_y = branch && (post || gate != GATE_NONE);
  int turn3 = 0, turn2 = 0;
  bool ok[NV];
  Vec<TP, VEC> wq[NV], wp[NV], gc[NV];
  float acc_pre[E], acc_post[E], acc_gate[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc_pre[e] = acc_post[e] = acc_gate[e] = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) ok[v] = (v * TPR + tx) * VEC < H;
  auto weights = [&]() {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + tx) * VEC;
      wq[v].zero();
      wp[v].zero();
      gc[v].zero();
      if (ok[v] && post) wq[v].load(a.w_post, c);
      if (ok[v] && pre) wp[v].load(a.w_pre, c);
      if (ok[v] && gate == GATE_COL) gc[v].load(a.g, c);
    }
  };
  if constexpr (KEEP) weights();
  const int64_t step = (int64_t)gridDim.x * RPB;
  Vec<TA, VEC> no[NV], ndx[NV], ndr[NV], ny[NV], nge[NV];  // the next row's operands
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t i = t * H + (v * TPR + tx) * VEC;
      no[v].zero();
      ndx[v].zero();
      ndr[v].zero();
      ny[v].zero();
      nge[v].zero();
      if (ok[v] && t < a.T) {
        if (pre) {
          no[v].load(a.R, i);
          ndx[v].load(a.dX, i);
        }
        if (need_y) ny[v].load(a.Y, i);
        if (has_dr) ndr[v].load(a.dR, i);
        if (gate == GATE_ELEM) nge[v].load(a.g, i);
      }
    }
  };
  int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if constexpr (PREFETCH) fetch(t);
  for (; t < a.T; t += step) {
    if constexpr (!PREFETCH) fetch(t);
    if constexpr (!KEEP) weights();
    Vec<TA, VEC> o[NV], dx[NV], dr[NV], y[NV], ge[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      o[v] = no[v];
      dx[v] = ndx[v];
      dr[v] = ndr[v];
      y[v] = ny[v];
      ge[v] = nge[v];
    }
    if constexpr (PREFETCH) fetch(t + step);
    float uo = 0.0f, mo = 0.0f, uy = 1.0f;
    if (pre || post) {
      float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          q[0] = fmaf(o[v][i], o[v][i], q[0]);
          q[1] = fmaf(dx[v][i] * (a.offset + wp[v][i]), o[v][i], q[1]);
          q[2] = fmaf(y[v][i], y[v][i], q[2]);
        }
      row_sums<TPR, 3>(q, lds3, turn3);
      if (pre) {
        uo = rsqrtf(fmaf(q[0], inv_h, a.eps));
        mo = q[1] * inv_h * uo * uo;  // mean(q n) / rms(R'): d's multiple of R' uo
      }
      if (post) uy = rsqrtf(fmaf(q[2], inv_h, a.eps));
    }
    float b = a.branch_scale;
    if (gate == GATE_ROW) b *= load1(static_cast<const TA*>(a.g) + t);
    float d[E];  // d, then z
    float q2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float outv[VEC], dgv[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int e = v * VEC + i;
        d[e] = 0.0f;
        if (!ok[v]) continue;  // columns past H take no part in the sums, whatever the row's factors
        const float n = o[v][i] * uo;
        float x = dr[v][i];
        if (pre) {
          x += fmaf(dx[v][i] * (a.offset + wp[v][i]), uo, -n * mo);
          acc_pre[e] = fmaf(dx[v][i], n, acc_pre[e]);
        }
        outv[i] = a.res_scale * x;
        if (branch) {
          const float yn = y[v][i] * uy;
          const float w = post ? a.offset + wq[v][i] : 1.0f;
          // the gate's gradient is b d p without the gate itself
          const float dp = a.branch_scale * x * (yn * w);
          if (gate == GATE_COL) acc_gate[e] += dp;
          dgv[i] = dp;
          q2[1] += dp;
          float z = b * x;
          if (gate == GATE_COL) z *= gc[v][i];
          if (gate == GATE_ELEM) z *= ge[v][i];
          if (post) {
            acc_post[e] = fmaf(z, yn, acc_post[e]);
            z *= w;
            q2[0] = fmaf(z, yn, q2[0]);
          }
          x = z;
        }
        d[e] = x;
      }
      if (ok[v]) {
        const int64_t i = t * H + (v * TPR + tx) * VEC;
        Vec<TA, VEC>::store(a.dR_out, i, outv);
        if (gate == GATE_ELEM) Vec<TA, VEC>::store(a.dg, i, dgv);
      }
    }
    if (branch) {
      if (post || gate == GATE_ROW) {
        row_sums<TPR, 2>(q2, lds2, turn2);
        if (gate == GATE_ROW && tx == 0) store1(static_cast<TA*>(a.dg) + t, q2[1]);
      }
      const float m = q2[0] * inv_h;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (post)
#pragma unroll
          for (int i = 0; i < VEC; ++i) d[v * VEC + i] = uy * (d[v * VEC + i] - y[v][i] * uy * m);
        if (ok[v]) Vec<TA, VEC>::store(a.dY, t * H + (v * TPR + tx) * VEC, d + v * VEC);
      }
    }
  }
  // one slice per block; the rows of a block's wavefronts (RPB > 1) meet in LDS first
  auto put = [&](float* dst, const float (&acc)[E]) {
    if (dst == nullptr) return;  // uniform
    if constexpr (RPB > 1) {
      __shared__ float sum[RPB][E * TPR];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) sum[threadIdx.x / TPR][(e / VEC * TPR + tx) * VEC + e % VEC] = acc[e];
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += norm_block<TPR>()) {
        float x = sum[0][c];
#pragma unroll
        for (int k = 1; k < RPB; ++k) x += sum[k][c];
        dst[(int64_t)blockIdx.x * H + c] = x;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (ok[v])
          Vec<float, VEC>::store(dst, (int64_t)blockIdx.x * H + (v * TPR + tx) * VEC, acc + v * VEC);
    }
  };
  put(a.p_pre, acc_pre);
  put(a.p_post, acc_post);
  put(a.p_gate, acc_gate);
}

// dst[c] = sum over the nb slices of part [nb, H], in ascending order within
// each of 16 runs of slices and then over the runs.  nb = 0 writes zeros.
struct NormGradArgs {
  const float* part[3];
  void* dst[3];
  int32_t n, H, nb;
};
template <typename TP>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormGradArgs a) {
  constexpr int AHEAD = 16;  // slices a thread loads together (past the last one it is read again)
  __shared__ float run[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
  const float* p = a.part[blockIdx.y];
  float s = 0.0f;
  if (c < a.H)
    for (int b0 = k; b0 < a.nb; b0 += 16 * AHEAD) {
      float x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) x[i] = p[(int64_t)min(b0 + 16 * i, a.nb - 1) * a.H + c];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s = b0 + 16 * i < a.nb ? s + x[i] : s;
    }
  run[k][threadIdx.x & 63] = s;
  __syncthreads();
  if (k == 0 && c < a.H) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += run[i][threadIdx.x];
    store1(static_cast<TP*>(a.dst[blockIdx.y]) + c, s);
  }
}

// Blocks of a backward pass, each of which writes one slice of column sums:
// two per CU keep enough loads in flight, more would only add slices.
int64_t bwd_blocks(int64_t T, int64_t H) {
  const int64_t rpb = H <= 1024 ? 4 : 1;
  const int64_t need = cdiv(T, rpb);
  return need < 512 ? need : 512;
}

// Threads per row and elements per thread: the smallest that hold the row.
template <bool BWD, typename TA, typename TP, int VEC, int TPR, int E>
hipError_t launch_cfg(const NormArgs& a, hipStream_t st) {
  constexpr int B = norm_block<TPR>(), RPB = B / TPR;
  if constexpr (BWD) {
    hipLaunchKernelGGL((norm_bwd_kernel<TA, TP, VEC, TPR, E / VEC>), dim3((unsigned)bwd_blocks(a.T, a.H)), dim3(B), 0, st,
                       a);
  } else {
    const int64_t need = cdiv(a.T, RPB), cap = 256 * std::max(2048 / B, 4);
    hipLaunchKernelGGL((norm_fwd_kernel<TA, TP, VEC, TPR, E / VEC>), dim3((unsigned)(need < cap ? need : cap)), dim3(B), 0,
                       st, a);
  }
  return hipGetLastError();
}
template <bool BWD, typename TA, typename TP, int VEC>
hipError_t launch_vec(const NormArgs& a, hipStream_t st) {
  if (a.H <= 512) return launch_cfg<BWD, TA, TP, VEC, 64, 8>(a, st);
  if (a.H <= 1024) return launch_cfg<BWD, TA, TP, VEC, 64, 16>(a, st);
  if (a.H <= 2048) return launch_cfg<BWD, TA, TP, VEC, 256, 8>(a, st);
  if constexpr (VEC == 1) {  // sixteen scalars of each operand do not fit the registers of a backward pass
    if (a.H <= 4096) return launch_cfg<BWD, TA, TP, VEC, 512, 8>(a, st);
  } else {
    if (a.H <= 4096) return launch_cfg<BWD, TA, TP, VEC, 256, 16>(a, st);
  }
  if constexpr (VEC == 8) {  // rows of 5120: 61 us forward with 512 threads of 16 elements, 51 us so
    if (a.H <= 5120) return launch_cfg<BWD, TA, TP, VEC, 640, 8>(a, st);
    if (a.H <= 6144) return launch_cfg<BWD, TA, TP, VEC, 768, 8>(a, st);
  }
  if (a.H <= 8192) return launch_cfg<BWD, TA, TP, VEC, 512, 16>(a, st);
  // A backward pass of wider rows holds three column sums beside five operands, which spill: a bf16 one
  // less from 512 threads of 32 elements than from 1024 of 16, which have 128 registers each (250 against
  // 336 us at 2048 rows of 16384).  Registers spilled a thread, and time at 2048 rows of 16384 with all
  // gradients: bf16 139, 250 us (1.6 TB/s); bf16 with fp32 parameters 557, 503 us (0.8); fp32 314, 831 us
  // (1.0); element by element 244 (655 us at 9001 columns, 0.7 TB/s), and from 4097 columns on 204 (245 us
  // at 5001, 1.0 TB/s).  Up to 8192 columns the vector forms spill 8 registers at most and keep 3.3 TB/s.
  if constexpr (BWD && VEC == 8) return launch_cfg<BWD, TA, TP, VEC, 512, 32>(a, st);
  else return launch_cfg<BWD, TA, TP, VEC, 1024, 16>(a, st);
}
template <bool BWD>
hipError_t launch_norm(const NormArgs& a, int32_t dtype, bool vec, hipStream_t st) {
  if (dtype == LORA_BF16) return launch_vec<BWD, uint16_t, uint16_t, 8>(a, st);
  if (dtype == LORA_BF16_F32LORA) return launch_vec<BWD, uint16_t, float, 8>(a, st);
  return vec ? launch_vec<BWD, float, float, 4>(a, st) : launch_vec<BWD, float, float, 1>(a, st);
}

// ---------------------------------------------------------------------------
// Checks of the entry points.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxH = 16384;

struct NormSizes {
  size_t es, ps;      // activation and parameter element sizes
  size_t act, par;    // bytes of a [T, H] tensor and of an [H] parameter
  size_t gate, align;
};

lora_status check_desc(const lora_norm_desc* d, NormSizes& z) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16 || d->dtype == LORA_BF16_F32LORA, LORA_EDTYPE, "unknown dtype %d",
        d->dtype);
  CHECK(d->gate >= LORA_GATE_NONE && d->gate <= LORA_GATE_ELEM, LORA_EINVAL, "unknown gate %d", d->gate);
  CHECK(d->unit_offset == 0 || d->unit_offset == 1, LORA_EINVAL, "unit_offset = %d is not 0 or 1", d->unit_offset);
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  CHECK(std::isfinite(d->eps) && d->eps >= 0.0f, LORA_EINVAL, "eps must be finite and not negative");
  CHECK(std::isfinite(d->res_scale) && std::isfinite(d->branch_scale), LORA_EINVAL, "a scale is not finite");
  CHECK(d->T >= 0, LORA_ESHAPE, "T = %lld is negative", (long long)d->T);
  CHECK(d->H > 0 && d->H <= kMaxH, LORA_ESHAPE, "H = %lld must be in [1, %lld]", (long long)d->H, (long long)kMaxH);
  const bool bf16 = d->dtype != LORA_F32;
  if (bf16) CHECK(d->H % 64 == 0, LORA_ESHAPE, "H = %lld must be a multiple of 64 for bf16", (long long)d->H);
  CHECK(d->T <= ((int64_t)1 << 46) / d->H, LORA_ESHAPE, "T = %lld rows of %lld are too many", (long long)d->T, (long long)d->H);
  z.es = bf16 ? 2 : 4;
  z.ps = d->dtype == LORA_BF16 ? 2 : 4;
  z.act = (size_t)d->T * d->H * z.es;
  z.par = (size_t)d->H * z.ps;
  z.gate = d->gate == LORA_GATE_COL ? z.par : d->gate == LORA_GATE_ROW ? (size_t)d->T * z.es : d->gate == LORA_GATE_ELEM ? z.act : 0;
  z.align = bf16 ? 16 : 4;
  return LORA_OK;
}

struct Buf {
  const void* p;
  size_t bytes;
  const char* name;
  bool rows;  // a [T, H] tensor, walked row by row: an output may be exactly this buffer
};

// Every tensor is aligned, and no output shares memory with another tensor,
// except that a [T, H] output may be exactly one of the [T, H] inputs.
lora_status check_bufs(const NormSizes& z, const Buf* in, int ni, const Buf* out, int no) {
  for (int i = 0; i < ni + no; ++i) {
    const Buf& b = i < ni ? in[i] : out[i - ni];
    CHECK(aligned(b.p, z.align), LORA_EALIGN, "%s is not %d-byte aligned", b.name, (int)z.align);
  }
  for (int i = 0; i < no; ++i) {
    if (out[i].p == nullptr) continue;
    for (int j = 0; j < ni; ++j) {
      if (in[j].p == nullptr || (out[i].p == in[j].p && out[i].rows && in[j].rows)) continue;
      CHECK(!overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes), LORA_EUNSUPPORTED, "%s overlaps %s", out[i].name,
            in[j].name);
    }
    for (int j = 0; j < i; ++j)
      CHECK(out[j].p == nullptr || !overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes), LORA_EUNSUPPORTED,
            "%s overlaps %s", out[i].name, out[j].name);
  }
  return LORA_OK;
}

NormArgs base_args(const lora_norm_desc* d) {
  NormArgs a{};
  a.T = d->T;
  a.H = (int32_t)d->H;
  a.gate = d->gate;
  a.eps = d->eps;
  a.res_scale = d->res_scale;
  a.branch_scale = d->branch_scale;
  a.offset = d->unit_offset ? 1.0f : 0.0f;
  return a;
}

// 16-byte accesses in fp32: whole vectors in every row, at aligned addresses.
bool vec_ok(const lora_norm_desc* d, const Buf* in, int ni, const Buf* out, int no) {
  if (d->H % 4) return false;
  for (int i = 0; i < ni; ++i)
    if (!aligned(in[i].p, 16)) return false;
  for (int i = 0; i < no; ++i)
    if (!aligned(out[i].p, 16)) return false;
  return true;
}

size_t bwd_bytes(const lora_norm_desc* d) {
  return d->T == 0 ? 0 : 3 * (size_t)bwd_blocks(d->T, d->H) * (size_t)((d->H + 63) / 64 * 64) * 4;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_block_norm_workspace_size(const lora_norm_desc* d, size_t* bwd) {
  NormSizes z;
  TRY(check_desc(d, z));
  if (bwd) *bwd = bwd_bytes(d);
  return LORA_OK;
}

lora_status lora_block_norm_fwd(const lora_norm_desc* d, const void* R, const void* Y, const void* gate,
                                const void* w_post, const void* w_pre, void* R_out, void* X, void* stream) {
  NormSizes z;
  TRY(check_desc(d, z));
  CHECK((gate != nullptr) == (d->gate != LORA_GATE_NONE) || (d->T == 0 && gate == nullptr), LORA_EINVAL,
        "gate and the descriptor's gate kind disagree");
  if (d->T == 0) return LORA_OK;
  CHECK(R != nullptr, LORA_EINVAL, "R is NULL");
  CHECK((Y != nullptr) == (R_out != nullptr), LORA_EINVAL, "R_out is written exactly when Y is given");
  CHECK((w_pre != nullptr) == (X != nullptr), LORA_EINVAL, "X is written exactly when w_pre is given");
  CHECK(Y != nullptr || w_pre != nullptr, LORA_EINVAL, "neither Y nor w_pre: nothing to compute");
  if (Y == nullptr)
    CHECK(w_post == nullptr && d->gate == LORA_GATE_NONE && d->res_scale == 1.0f, LORA_EINVAL,
          "w_post, a gate and res_scale need Y");
  const Buf in[] = {{R, z.act, "R", true}, {Y, z.act, "Y", true}, {gate, z.gate, "gate", d->gate == LORA_GATE_ELEM},
                    {w_post, z.par, "w_post", false}, {w_pre, z.par, "w_pre", false}};
  const Buf out[] = {{R_out, z.act, "R_out", true}, {X, z.act, "X", true}};
  TRY(check_bufs(z, in, 5, out, 2));
  NormArgs a = base_args(d);
  a.R = R;
  a.Y = Y;
  a.g = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.out = R_out;
  a.X = X;
  hipStream_t st = static_cast<hipStream_t>(stream);
  LAUNCHN("norm_fwd", st, launch_norm<false>(a, d->dtype, vec_ok(d, in, 5, out, 2), st));
  return LORA_OK;
}

lora_status lora_block_norm_bwd(const lora_norm_desc* d, const void* dR_out, const void* dX, const void* R_out,
                                const void* Y, const void* gate, const void* w_post, const void* w_pre, void* dR,
                                void* dY, const lora_norm_grads* grads, void* ws, size_t ws_bytes, void* stream) {
  NormSizes z;
  TRY(check_desc(d, z));
  CHECK(grads != nullptr, LORA_EINVAL, "grads is NULL");
  const bool rows = d->T > 0;
  CHECK((gate != nullptr) == (d->gate != LORA_GATE_NONE) || (!rows && gate == nullptr), LORA_EINVAL,
        "gate and the descriptor's gate kind disagree");
  CHECK((w_post != nullptr) == (grads->dw_post != nullptr) && (w_pre != nullptr) == (grads->dw_pre != nullptr),
        LORA_EINVAL, "a weight and its gradient are given together");
  if (rows || d->gate == LORA_GATE_COL)
    CHECK((d->gate != LORA_GATE_NONE) == (grads->dgate != nullptr), LORA_EINVAL, "a gate and its gradient are given together");
  if (rows) {
    CHECK(dR != nullptr, LORA_EINVAL, "dR is NULL");
    CHECK(dR_out != nullptr || w_pre != nullptr, LORA_EINVAL, "neither dR_out nor w_pre: no gradient comes in");
    CHECK((w_pre != nullptr) == (dX != nullptr), LORA_EINVAL, "dX is read exactly when w_pre is given");
    CHECK(w_pre == nullptr || R_out != nullptr, LORA_EINVAL, "R_out is NULL");
    CHECK((Y != nullptr) == (dY != nullptr), LORA_EINVAL, "dY is written exactly when Y is given");
    if (Y == nullptr)
      CHECK(w_post == nullptr && d->gate == LORA_GATE_NONE && d->res_scale == 1.0f, LORA_EINVAL,
            "w_post, a gate and res_scale need Y");
  }
  TRY(check_ws(ws, ws_bytes, bwd_bytes(d)));
  const Buf in[] = {{dR_out, z.act, "dR_out", true}, {dX, z.act, "dX", true}, {R_out, z.act, "R_out", true},
                    {Y, z.act, "Y", true}, {gate, z.gate, "gate", d->gate == LORA_GATE_ELEM},
                    {w_post, z.par, "w_post", false}, {w_pre, z.par, "w_pre", false}};
  const Buf out[] = {{dR, z.act, "dR", true}, {dY, z.act, "dY", true},
                     {grads->dgate, z.gate, "dgate", d->gate == LORA_GATE_ELEM}, {grads->dw_post, z.par, "dw_post", false},
                     {grads->dw_pre, z.par, "dw_pre", false}, {ws, bwd_bytes(d), "ws", false}};
  TRY(check_bufs(z, in, 7, out, 6));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t nb = rows ? bwd_blocks(d->T, d->H) : 0;
  NormGradArgs r{};
  r.H = (int32_t)d->H;
  r.nb = (int32_t)nb;
  float* part = static_cast<float*>(ws);
  const size_t slice = (size_t)nb * (size_t)((d->H + 63) / 64 * 64);
  NormArgs a = base_args(d);
  void* const dst[3] = {grads->dw_pre, grads->dw_post, d->gate == LORA_GATE_COL ? grads->dgate : nullptr};
  float** const slot[3] = {&a.p_pre, &a.p_post, &a.p_gate};
  for (int i = 0; i < 3; ++i) {
    if (dst[i] == nullptr) continue;
    if (rows) *slot[i] = part + i * slice;
    r.part[r.n] = *slot[i];
    r.dst[r.n++] = dst[i];
  }
  if (rows) {
    a.dR = dR_out;
    a.dX = dX;
    a.R = R_out;
    a.Y = Y;
    a.g = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.dR_out = dR;
    a.dY = dY;
    a.dg = d->gate == LORA_GATE_COL ? nullptr : grads->dgate;
    LAUNCHN("norm_bwd", st, launch_norm<true>(a, d->dtype, vec_ok(d, in, 7, out, 6), st));
  }
  if (r.n > 0) {
    const dim3 grid((unsigned)cdiv(d->H, 64), (unsigned)r.n);
    TraceScope ts("norm_grad", st);
    if (z.ps == 2) hipLaunchKernelGGL(norm_grad_kernel<uint16_t>, grid, dim3(1024), 0, st, r);
    else hipLaunchKernelGGL(norm_grad_kernel<float>, grid, dim3(1024), 0, st, r);
    LAUNCH(hipGetLastError());
  }
  return LORA_OK;
}

}  // extern "C"
