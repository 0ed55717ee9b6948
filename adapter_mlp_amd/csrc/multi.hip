// Low-rank adapters of many requests beside a shared projection:
//   Y[t] = X[t] W + s_i (X[t] A_i) B_i,   i = ids[t]
// (rows whose id lies outside [0, n) take the base alone).
#include <algorithm>

#include "abi.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "lds_dma.hpp"

namespace lora {
namespace {

struct MultiArgs {
  const void *X, *W, *A, *B;
  const float* scales;
  const int32_t* ids;
  void* Y;
  float* part;   // [ks, T, N] fp32 sums of X W over K ranges (nullptr: add to Y)
  float* upart;  // [kc, T, r] fp32 sums of X A_i over K ranges
  int64_t T, K, N, n;
  int32_t r, ks, kc, ntn, ntm;
};

// The adapter of a row, -1 for none.
__device__ __forceinline__ int row_id(const MultiArgs& a, int64_t t) {
  if (t >= a.T) return -1;
  const int i = a.ids[t];
  return i >= 0 && i < a.n ? i : -1;
}

template <int D, int K>
__device__ __forceinline__ void wait_stages(int after) {
  // vmcnt(D * after), after = 0 .. K (compile-time immediates)
  if constexpr (K > 0) {
    if (after >= K) {
      wait_vmcnt<D * K>();
      return;
    }
    wait_stages<D, K - 1>(after);
  } else {
    wait_vmcnt<0>();
  }
}

// ---------------------------------------------------------------------------
// X W for few rows (bf16): fp32 sums over one of ks K ranges.  Bound by
// streaming W once, so the work is split over K until the grid fills the
// chip, and every block keeps several 64-deep K stages in flight: W
// [64][128 columns] and X [16 MT rows][64] go from global memory straight into
// a ring of LDS slots.  Four wavefronts of 32 columns each; the weight is the
// MFMA's row operand, so a lane ends with four consecutive columns of a row.
// LDS layouts: W rows of 256 bytes, 16-byte chunk c of row k at c ^ 4 (k & 3),
// read with the transposing LDS read; X rows of 128 bytes, chunk c of row m at
// c ^ (m & 7).
// ---------------------------------------------------------------------------
template <int MT>
struct BaseCfg {
  static constexpr int WB = 64 * 256, XB = MT * 16 * 128, SB = WB + XB;
  static constexpr int NST = MT <= 4 ? 4 : 3;
  static constexpr int XPW = MT / 2;  // 1 KB loads of X per wavefront and stage
  static constexpr int D = 4 + XPW;
};

template <int MT>
__device__ __forceinline__ void base_block(const MultiArgs& a, char* ring, int bid) {
  using C = BaseCfg<MT>;
  lds_char* const lds = (lds_char*)ring;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // blocks b, b + 8, ... run on one XCD: the row tiles of one weight tile follow each other there
  const int units = a.ntn * a.ks;
  const int j = bid >> 3;
  const int u = (j / a.ntm) * 8 + (bid & 7), tm = j % a.ntm;
  if (u >= units) return;
  const int tn = u % a.ntn, part = u / a.ntn;
  const int steps = (int)(a.K / 64);
  const int s0 = (int)((int64_t)part * steps / a.ks), s1 = (int)((int64_t)(part + 1) * steps / a.ks);
  const int64_t m0 = (int64_t)tm * (16 * MT), n0 = (int64_t)tn * 128;
  const uint32_t ldw2 = (uint32_t)(a.N * 2), ldx2 = (uint32_t)(a.K * 2);
  const char* wp = static_cast<const char*>(a.W) + ((int64_t)s0 * 64 * a.N + n0) * 2;
  int64_t wn = ((a.K - (int64_t)s0 * 64) * a.N - n0) * 2;
  const char* xp = static_cast<const char*>(a.X) + (m0 * a.K + (int64_t)s0 * 64) * 2;
  int64_t xn = ((a.T - m0) * a.K - (int64_t)s0 * 64) * 2;
  const uint32_t woff = (uint32_t)(lane >> 4) * ldw2 + (uint32_t)(((lane & 15) ^ (4 * ((lane >> 4) & 3))) * 16);
  uint32_t xoff[C::XPW];  // rows past T read zero
#pragma unroll
  for (int i = 0; i < C::XPW; ++i) {
    const int row = 8 * (C::XPW * w + i) + (lane >> 3);
    xoff[i] = m0 + row < a.T ? (uint32_t)row * ldx2 + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16) : 0x80000000u;
  }
  auto issue = [&](int slot) {
    const uint32_t base = lds_addr(lds) + slot * C::SB;
    const i32x4 rw = rsrc_words(wp, wn), rx = rsrc_words(xp, xn);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma16(rw, woff, base + (4 * w + i) * 1024, (uint32_t)(4 * (4 * w + i)) * ldw2);
#pragma unroll
    for (int i = 0; i < C::XPW; ++i)
      dma16(rx, xoff[i], base + C::WB + (C::XPW * w + i) * 1024);
    wp += (int64_t)64 * a.N * 2;
    wn -= (int64_t)64 * a.N * 2;
    xp += 128;
    xn -= 128;
  };
  const int g = lane >> 4, c = lane & 15, jj = c >> 2;
  f32x4 acc[2][MT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  int wo[2];  // fragment offsets of the wavefront's two 16-column blocks
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = 32 * w + 16 * i + 4 * (lane & 3);
    wo[i] = (8 * g + jj) * 256 + (((col >> 3) ^ (4 * jj)) * 16) + (lane & 1) * 8;
  }
  const int n = s1 - s0;
  for (int s = 0; s < C::NST - 1 && s < n; ++s) issue(s);
  int slot = 0;
  for (int s = 0; s < n; ++s) {
    const int after = n - 1 - s < C::NST - 2 ? n - 1 - s : C::NST - 2;
    wait_stages<C::D, C::NST - 2>(after);
    __syncthreads();  // stage s is in for every wavefront, and stage s - 1 is no longer read
    if (s + C::NST - 1 < n) issue(slot == 0 ? C::NST - 1 : slot - 1);
    const lds_char* ws = lds + slot * C::SB;
    const lds_char* xs = ws + C::WB;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 fw[2], fx[MT];
#pragma unroll
      for (int i = 0; i < 2; ++i) fw[i] = lds_read_tr8(ws + wo[i] + 32 * k * 256, 4 * 256);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        fx[m] = __builtin_bit_cast(bf16x8, lds_read16(xs + (16 * m + c) * 128 + (((4 * k + g) ^ (c & 7)) * 16)));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fx[m], acc[i][m], 0, 0, 0);
    }
    slot = slot + 1 == C::NST ? 0 : slot + 1;
  }
  float* out = a.part + (int64_t)part * a.T * a.N;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t t = m0 + 16 * m + c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t col = n0 + 32 * w + 16 * i + 4 * g;
      if (t < a.T && col < a.N) *reinterpret_cast<f32x4*>(out + t * a.N + col) = acc[i][m];
    }
  }
}

template <int MT>
__global__ __launch_bounds__(256) void multi_base_kernel(const MultiArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[BaseCfg<MT>::NST * BaseCfg<MT>::SB];
  base_block<MT>(a, ring, blockIdx.x);
}

// ---------------------------------------------------------------------------
// U = X A_i (bf16): fp32 sums over K ranges of kShrinkK, for 16 RG rows a
// block.  Every wavefront takes a quarter of the range for all of the rows
// and walks the distinct adapters of the rows, each multiplied against all
// of them (the MFMA computes 16 rows at a time anyway) and kept where it is
// the row's own; rows of one request sit together, so that is one or two
// passes over rows that stay in cache.  A_i [K, r] is read as it lies: lane
// 16 q + c takes columns NJ c .. NJ c + NJ - 1 of 8 consecutive K rows, which
// after a transpose in registers are the operands of NJ tiles (tile t: rank
// index NJ c + t).
// ---------------------------------------------------------------------------
constexpr int kShrinkK = 1024;

template <int NJ>
__device__ __forceinline__ void load_a_frags(brsrc ra, uint32_t row0, int r, int c, bf16x8 (&f)[NJ]) {
  // row0: first of the lane's 8 K rows; rows past the end read zero
  const uint32_t ld = (uint32_t)r * 2;
  uint32_t off = row0 * ld + (uint32_t)(NJ * c) * 2;
  if (NJ * c >= r) off = 0x80000000u;  // columns past the rank read zero
  uint16_t x[8][NJ];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t o = off + (off < 0x80000000u ? (uint32_t)e * ld : 0u);
    if constexpr (NJ == 4) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(ra, o, 0, 0);
      x[e][0] = (uint16_t)v[0];
      x[e][1] = (uint16_t)(v[0] >> 16);
      x[e][2] = (uint16_t)v[1];
      x[e][3] = (uint16_t)(v[1] >> 16);
    } else if constexpr (NJ == 2) {
      const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(ra, o, 0, 0);
      x[e][0] = (uint16_t)v;
      x[e][1] = (uint16_t)(v >> 16);
    } else {
#pragma unroll
      for (int t = 0; t < NJ; ++t) x[e][t] = __builtin_amdgcn_raw_buffer_load_b16(ra, o + 2 * t, 0, 0);
    }
  }
#pragma unroll
  for (int t = 0; t < NJ; ++t) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (uint32_t)x[2 * e][t] | ((uint32_t)x[2 * e + 1][t] << 16);
    f[t] = __builtin_bit_cast(bf16x8, v);
  }
}

template <int RG, int NJ>
__global__ __launch_bounds__(256) void multi_shrink_kernel(const MultiArgs a) {
  __shared__ f32x4 red[3][RG * NJ][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * RG);
  const int kc = blockIdx.y;
  const int64_t k0 = (int64_t)kc * kShrinkK + w * (kShrinkK / 4);
  const int64_t klen = a.K - k0 < kShrinkK / 4 ? a.K - k0 : kShrinkK / 4;  // multiple of 64, may be <= 0
  const int my = lane < 16 * RG ? row_id(a, t0 + lane) : -1;               // id of row t0 + lane
  int rid[RG];                                                             // ids of this lane's MFMA rows
#pragma unroll
  for (int m = 0; m < RG; ++m) rid[m] = __shfl(my, 16 * m + c);
  uint32_t xrow[RG];  // rows past T read zero
#pragma unroll
  for (int m = 0; m < RG; ++m)
    xrow[m] = t0 + 16 * m + c < a.T ? (uint32_t)((16 * m + c) * a.K * 2) : 0x80000000u;
  const brsrc rx = make_rsrc(static_cast<const char*>(a.X) + (t0 * a.K + k0) * 2, ((a.T - t0) * a.K - k0) * 2);
  uint64_t todo = __ballot(my >= 0);
  while (todo != 0) {
    const int id = __builtin_amdgcn_readlane(my, __builtin_ctzll(todo));
    todo &= ~__ballot(my == id);
    const char* Ai = static_cast<const char*>(a.A) + (int64_t)id * a.K * a.r * 2;
    const brsrc ra = make_rsrc(Ai + k0 * a.r * 2, klen * a.r * 2);
    f32x4 acc[RG][NJ];
#pragma unroll
    for (int m = 0; m < RG; ++m)
#pragma unroll
      for (int t = 0; t < NJ; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
#pragma unroll 2
    for (int k = 0; k < (int)klen; k += 32) {
      bf16x8 fa[NJ], fx[RG];
      load_a_frags<NJ>(ra, (uint32_t)(k + 8 * g), a.r, c, fa);
#pragma unroll
      for (int m = 0; m < RG; ++m)
        fx[m] = __builtin_bit_cast(bf16x8, buf_load16(rx, xrow[m] + (xrow[m] < 0x80000000u ? (uint32_t)(k + 8 * g) * 2 : 0u)));
#pragma unroll
      for (int m = 0; m < RG; ++m)
#pragma unroll
        for (int t = 0; t < NJ; ++t) acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[t], fx[m], acc[m][t], 0, 0, 0);
    }
    // the four quarters of the K range, in ascending order
    if (w > 0)
#pragma unroll
      for (int m = 0; m < RG; ++m)
#pragma unroll
        for (int t = 0; t < NJ; ++t) red[w - 1][m * NJ + t][lane] = acc[m][t];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int m = 0; m < RG; ++m) {
        const int64_t t = t0 + 16 * m + c;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          f32x4 s = acc[m][j];
#pragma unroll
          for (int q = 0; q < 3; ++q) s += red[q][m * NJ + j][lane];
          // rank index NJ (4 g + v) + j
          float* u = a.upart + ((int64_t)kc * a.T + t) * a.r;
          if (rid[m] == id)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int i = NJ * (4 * g + v) + j;
              if (i < a.r) u[i] = s[v];
            }
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Y = sum of the K ranges' parts (or Y itself) + s_i U B_i, rounded once.
// 16 rows a block, one wavefront per 4 rows and 512 columns: a lane owns 8
// columns.  U of the block's rows is summed over its K ranges into LDS, times
// the adapter's scale.  Four rows of one adapter share the loads of B_i.
// ---------------------------------------------------------------------------
template <typename T>
struct Cols;
template <>
struct Cols<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[8]) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = lo_bf(v[k]);
      f[2 * k + 1] = hi_bf(v[k]);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    const u32x4 v = {pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])};
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = v;
  }
};
template <>
struct Cols<float> {
  static constexpr int N = 1;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[1]) { f[0] = static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[1]) { static_cast<float*>(p)[i] = f[0]; }
};

template <typename T>
__global__ __launch_bounds__(256) void multi_expand_kernel(const MultiArgs a) {
  constexpr int C = Cols<T>::N;
  __shared__ float us[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.y * 16;
  const int64_t col = ((int64_t)blockIdx.x * 64 + lane) * C;
  for (int e = threadIdx.x; e < 16 * a.r; e += 256) {
    const int row = e / a.r, j = e % a.r;
    const int64_t t = t0 + row;
    const int id = row_id(a, t);
    float s = 0.0f;
    if (id >= 0) {
      for (int k = 0; k < a.kc; ++k) s += a.upart[((int64_t)k * a.T + t) * a.r + j];
      s *= a.scales[id];
    }
    us[row][j] = s;
  }
  __syncthreads();
  if (col >= a.N) return;
  float y[4][C];
  int id[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + 4 * w + i;
    id[i] = __builtin_amdgcn_readfirstlane(row_id(a, t));
    if (t >= a.T) continue;
    if (a.part == nullptr) {
      Cols<T>::load(a.Y, t * a.N + col, y[i]);
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) y[i][j] = 0.0f;
      for (int k = 0; k < a.ks; ++k) {
        const float* p = a.part + ((int64_t)k * a.T + t) * a.N + col;
#pragma unroll
        for (int j = 0; j < C; ++j) y[i][j] += p[j];
      }
    }
  }
  const int64_t bs = (int64_t)a.r * a.N;
  if (id[0] == id[1] && id[0] == id[2] && id[0] == id[3]) {
    if (id[0] >= 0)
      for (int j = 0; j < a.r; ++j) {
        float b[C];
        Cols<T>::load(a.B, id[0] * bs + (int64_t)j * a.N + col, b);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < C; ++k) y[i][k] = fmaf(us[4 * w + i][j], b[k], y[i][k]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (id[i] < 0) continue;
      for (int j = 0; j < a.r; ++j) {
        float b[C];
        Cols<T>::load(a.B, id[i] * bs + (int64_t)j * a.N + col, b);
#pragma unroll
        for (int k = 0; k < C; ++k) y[i][k] = fmaf(us[4 * w + i][j], b[k], y[i][k]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + 4 * w + i < a.T) Cols<T>::store(a.Y, (t0 + 4 * w + i) * a.N + col, y[i]);
}

// U in fp32: one block per row; threads are (K slot, rank index), slots added in ascending order.
__global__ __launch_bounds__(256) void multi_shrink_f32_kernel(const MultiArgs a) {
  __shared__ float red[256];
  const int64_t t = blockIdx.x;
  const int id = row_id(a, t);
  if (id < 0) return;  // uniform
  const int slots = 256 / a.r, slot = threadIdx.x / a.r, j = threadIdx.x % a.r;
  const float* x = static_cast<const float*>(a.X) + t * a.K;
  const float* A = static_cast<const float*>(a.A) + (int64_t)id * a.K * a.r;
  float s = 0.0f;
  if (slot < slots)
    for (int64_t k = slot; k < a.K; k += slots) s = fmaf(x[k], A[k * a.r + j], s);
  red[threadIdx.x] = s;
  __syncthreads();
  if (slot == 0) {
    for (int q = 1; q < slots; ++q) s += red[q * a.r + j];
    a.upart[t * a.r + j] = s;
  }
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
// Row tiles of 32, 64 or 128: the smallest that hold all rows, 128 beyond.
int row_tiles(int64_t T) { return T <= 32 ? 2 : T <= 64 ? 4 : 8; }

// K ranges of X W: enough blocks to fill the chip twice, each with at least
// four K stages.
int base_ksplit(int64_t T, int64_t K, int64_t N) {
  const int64_t units = cdiv(N, 128) * cdiv(T, 16 * row_tiles(T));
  const int64_t want = cdiv(512, units), most = std::max<int64_t>(1, K / 256);
  return (int)std::max<int64_t>(1, std::min(want, most));
}

template <int MT>
hipError_t launch_base(const MultiArgs& a, hipStream_t st) {
  const int64_t nb = cdiv((int64_t)a.ntn * a.ks, 8) * 8 * a.ntm;
  hipLaunchKernelGGL(multi_base_kernel<MT>, dim3((unsigned)nb), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <int RG>
hipError_t launch_shrink(const MultiArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)cdiv(a.T, 16 * RG), (unsigned)a.kc);
  switch (cdiv(a.r, 16)) {
    case 1: hipLaunchKernelGGL((multi_shrink_kernel<RG, 1>), grid, dim3(256), 0, st, a); break;
    case 2: hipLaunchKernelGGL((multi_shrink_kernel<RG, 2>), grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((multi_shrink_kernel<RG, 3>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((multi_shrink_kernel<RG, 4>), grid, dim3(256), 0, st, a); break;
  }
  return hipGetLastError();
}

// Workspace of a call.
struct MultiPlan {
  int ks, kc;
  float *part, *upart;
  size_t bytes;
};
MultiPlan plan_multi(const lora_multi_desc& d, bool base, void* ws) {
  MultiPlan p{};
  const bool bf16 = d.dtype == LORA_BF16;
  p.ks = bf16 && base && d.T > 0 ? base_ksplit(d.T, d.K, d.N) : 1;
  p.kc = bf16 ? (int)cdiv(d.K, kShrinkK) : 1;
  Ws w(ws);
  p.upart = static_cast<float*>(w.take((size_t)p.kc * d.T * d.r * 4));
  if (bf16 && base) p.part = static_cast<float*>(w.take((size_t)p.ks * d.T * d.N * 4));
  p.bytes = w.off;
  return p;
}

lora_status check_multi(const lora_multi_desc* d) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16, LORA_EDTYPE, "dtype %d is not LORA_F32 or LORA_BF16", d->dtype);
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  const bool bf16 = d->dtype == LORA_BF16;
  const int64_t es = bf16 ? 2 : 4, lim = ((int64_t)1 << 31) - 4096;
  CHECK(d->T >= 0, LORA_ESHAPE, "T = %lld is negative", (long long)d->T);
  CHECK(d->K > 0 && d->N > 0, LORA_ESHAPE, "K = %lld and N = %lld must be positive", (long long)d->K, (long long)d->N);
  CHECK(d->r >= 1 && d->r <= 64, LORA_ESHAPE, "rank r = %lld must be in [1, 64]", (long long)d->r);
  CHECK(d->n >= 0 && d->n < ((int64_t)1 << 31), LORA_ESHAPE, "n = %lld adapters", (long long)d->n);
  if (bf16) {
    CHECK(d->K % 64 == 0 && d->N % 64 == 0, LORA_ESHAPE, "K = %lld and N = %lld must be multiples of 64 for bf16",
          (long long)d->K, (long long)d->N);
    CHECK(d->r % 8 == 0, LORA_ESHAPE, "rank r = %lld must be a multiple of 8 for bf16", (long long)d->r);
  }
  CHECK(d->K <= lim / es / d->N, LORA_ESHAPE, "W (%lld x %lld) exceeds 2 GiB", (long long)d->K, (long long)d->N);
  CHECK(std::max(d->K, d->N) <= lim / es / d->r, LORA_ESHAPE, "an adapter exceeds 2 GiB");
  CHECK(d->T <= lim / es / std::max(d->K, d->N), LORA_ESHAPE, "X or Y (%lld rows) exceeds 2 GiB", (long long)d->T);
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_multi_workspace_size(const lora_multi_desc* d, size_t* bytes) {
  TRY(check_multi(d));
  if (bytes) *bytes = plan_multi(*d, true, nullptr).bytes;
  return LORA_OK;
}

lora_status lora_multi_fwd(const lora_multi_desc* d, const void* X, const void* W, const void* A, const void* B,
                           const float* scales, const int32_t* ids, void* Y, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_multi(d));
  const bool bf16 = d->dtype == LORA_BF16;
  const size_t al = bf16 ? 16 : 4, es = bf16 ? 2 : 4;
  const size_t nx = (size_t)d->T * d->K * es, ny = (size_t)d->T * d->N * es, nw = (size_t)d->K * d->N * es;
  const size_t na = (size_t)d->n * d->K * d->r * es, nb = (size_t)d->n * d->N * d->r * es;
  const size_t need = plan_multi(*d, W != nullptr, nullptr).bytes;
  if (d->T == 0) return LORA_OK;
  CHECK(X && Y && ids, LORA_EINVAL, "X, ids or Y is NULL");
  CHECK(d->n == 0 || (A && B && scales), LORA_EINVAL, "A, B or scales is NULL");
  CHECK(aligned(X, al) && aligned(W, al) && aligned(A, al) && aligned(B, al) && aligned(Y, al), LORA_EALIGN,
        "X, W, A, B or Y is not %d-byte aligned", (int)al);
  CHECK(aligned(scales, 4) && aligned(ids, 4), LORA_EALIGN, "scales or ids is not 4-byte aligned");
  TRY(check_ws(ws, ws_bytes, need));
  const struct {
    const void* p;
    size_t bytes;
  } in[] = {{X, nx}, {W, W ? nw : 0}, {A, na}, {B, nb}, {scales, (size_t)d->n * 4}, {ids, (size_t)d->T * 4}};
  for (const auto& b : in)
    CHECK(b.bytes == 0 || (!overlaps(Y, ny, b.p, b.bytes) && !overlaps(ws, need, b.p, b.bytes)), LORA_EUNSUPPORTED,
          "Y or the workspace overlaps an input");
  CHECK(!overlaps(Y, ny, ws, need), LORA_EUNSUPPORTED, "Y overlaps the workspace");

  hipStream_t st = static_cast<hipStream_t>(stream);
  const MultiPlan p = plan_multi(*d, W != nullptr, ws);
  MultiArgs a{};
  a.X = X;
  a.W = W;
  a.A = A;
  a.B = B;
  a.scales = scales;
  a.ids = ids;
  a.Y = Y;
  a.part = p.part;
  a.upart = p.upart;
  a.T = d->T;
  a.K = d->K;
  a.N = d->N;
  a.n = d->n;
  a.r = (int32_t)d->r;
  a.ks = p.ks;
  a.kc = p.kc;
  const int mt = row_tiles(d->T);
  a.ntn = (int32_t)cdiv(d->N, 128);
  a.ntm = (int32_t)cdiv(d->T, 16 * mt);
  if (bf16) {
    if (d->n > 0) LAUNCHN("multi_shrink", st, d->T <= 64 ? launch_shrink<1>(a, st) : launch_shrink<4>(a, st));
    if (W)
      LAUNCHN("multi_base", st, mt == 2 ? launch_base<2>(a, st) : mt == 4 ? launch_base<4>(a, st) : launch_base<8>(a, st));
    TraceScope ts("multi_expand", st);
    hipLaunchKernelGGL(multi_expand_kernel<uint16_t>, dim3((unsigned)cdiv(d->N, 512), (unsigned)cdiv(d->T, 16)), dim3(256), 0,
                       st, a);
    LAUNCH(hipGetLastError());
    return LORA_OK;
  }
  if (W) {
    GemmArgs g{};
    g.M = d->T;
    g.nseg = 1;
    g.nreg = 1;
    g.epi = EPI_STORE;
    g.bkind = B_NN;
    g.seg[0].A = X;
    g.seg[0].lda = d->K;
    g.seg[0].K = d->K;
    g.seg[0].b[0][0].p = W;
    g.seg[0].b[0][0].ld = d->N;
    g.reg[0].N = d->N;
    g.reg[0].out = Y;
    g.reg[0].ldo = d->N;
    g.ksplit = 1;
    g.ntile_m = cdiv(d->T, gemm_tile_rows(false));
    g.ntile_n = cdiv(d->N, gemm_tile_cols(false, false));
    LAUNCHN("gemm_nn_store_f32", st, launch_gemm_f32(g, st));
  }
  if (d->n > 0) {
    {
      TraceScope ts("multi_shrink_f32", st);
      hipLaunchKernelGGL(multi_shrink_f32_kernel, dim3((unsigned)d->T), dim3(256), 0, st, a);
      LAUNCH(hipGetLastError());
    }
    TraceScope ts("multi_expand_f32", st);
    hipLaunchKernelGGL(multi_expand_kernel<float>, dim3((unsigned)cdiv(d->N, 64), (unsigned)cdiv(d->T, 16)), dim3(256), 0, st, a);
    LAUNCH(hipGetLastError());
  }
  return LORA_OK;
}

}  // extern "C"
