// MLP of routed experts for few tokens:
//   l = X router^T,  the top_k experts of each token by l (or by a score of l plus a bias),
//   Y[t] = sum_j w_j  down_e (phi(gate_e X[t]) * up_e X[t]),   e = ids[t, j]
// with shared experts, which every token takes with weight 1, behind the
// routed ones in the stacks.
//
// With few tokens a layer streams the weights of the experts that were
// chosen, once, from HBM, and the rest has to stay beside that: the experts'
// rows are [n_out, n_in], so that 16 bytes of a row are a lane's MFMA operand
// as they lie in memory.  Which experts are met is known on the device only:
// the grid has a place for every expert that could be met; a block lists the
// rows of its own from the table of choices and ends where there are none.
//
// Launches: logits, choice (in one with the logits for a small router, with gate / up for one token),
// gate / up with the activation, down, sum over a
// token's experts (in one with down where few experts can be met).  Nothing is
// accumulated across blocks out of order: each (token, choice) has a row of its
// own in h and in the products of down.
//
// Measured, in bf16, all launches (a read-only stream reaches 7.2 TB/s on this
// chip): 64 tokens, 8 of 128 experts of 2048 x 768: 205 us, 1.22 GB, of which gate / up
// 127 us and down 67 us at 6.3 TB/s; 33 tokens, 2 of 8 of 4096 x 14336: 458 us, 2.9 GB,
// 301 and 146 us at 6.3 and 6.9 TB/s; one token, 8 of 128: 25 us, 76 MB, three launches of which
// none is long enough to reach the rate (2.7, 16 and 8 us).
#include <algorithm>
#include <cmath>

#include "abi.hpp"
#include "common.hpp"
#include "lds_dma.hpp"
#include "vec.hpp"

namespace lora {
namespace {

constexpr int kMaxT = 256, kMaxE = 512, kMaxK = 16, kMaxShared = 16;
constexpr int kRows = 64;  // rows of an expert that a block takes at a time
// Tokens, and experts they could meet, of a call by 4 x 4 tiles.  Against the ring for all:
// one token on 2 of 8 experts of 4096 x 14336 118 and 139 us, 4 and 8 tokens 300 and 386 against 327
// and 417; one token on 8 of 128 of 2048 x 768 27 and 27; but 8 tokens on 50 of 5120 x 1536 414 and
// 362, where the 16 wavefronts of a block of down take turns at the experts.
constexpr int kFewT = 8, kFewUnits = 16;
constexpr int kSumSlots = kFewT * kFewUnits;

struct MoeArgs {
  const void *X, *router, *gate, *up, *down;
  const float* bias;
  void* Y;
  double* logits;  // [T, E]
  int32_t* ids;    // [T, kk], kk = top_k + shared
  float* w;        // [T, kk]
  uint8_t* place;  // [E, Tp]: 1 + j where expert e is choice j of token t, else 0
  void* h;         // [T kk][2][I] bf16 (high and low part) or [T kk][Ip] fp32
  float* part;     // [T kk][Hp]
  int64_t H, I, Hp, Ip;
  int32_t T, Tp, E, k, kk, shared;  // Tp: T rounded up to 4
  int32_t units, routed, by_slot;  // experts that may be met: routed ones (by choice or by expert), then shared
  int32_t cs, cr;                  // blocks that share a shared or routed expert's rows
  int32_t act, score, normalize;
  float scale;
};

// ---------------------------------------------------------------------------
// Logits: a wavefront has one expert and TW tokens, or where these are few
// (KW = 4) the block's four take turns at the inputs (calls on 128 experts of width 2048: 1 token 24.2 and without
// 25.8 us, 64 tokens 200.4 and 198.2).  The choice of experts hangs on the last bits of near ties, so
// products, which fp64 holds exactly for bf16 and fp32 inputs, and sums are fp64: off by a
// few 2^-53 of the terms, whichever lanes they fall to.  (Runs of V products in fp32, added up in fp64:
// 1 to 2 us less at 64 to 256 tokens on 64 to 128 experts, 8 of 327 us a call at 200 on 256 of 4096 x 256.)
// ---------------------------------------------------------------------------
template <typename TX, typename TR, int V, int TW, int KW>
__global__ __launch_bounds__(256) void moe_logits_kernel(const MoeArgs a) {
  __shared__ double part[4][TW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = min((int)blockIdx.x * (4 / KW) + (KW == 4 ? 0 : wave), a.E - 1), t0 = blockIdx.y * TW;
  const int64_t H = a.H, row = (int64_t)e * H;
  double acc[TW];
#pragma unroll
  for (int j = 0; j < TW; ++j) acc[j] = 0.0;
#pragma unroll(KW == 4 ? 2 : 4)
  for (int64_t k = (KW == 4 ? threadIdx.x : lane) * V; k < H; k += KW * 64 * V) {
    Vec<TR, V> w;
    w.load(a.router, row + k);
    Vec<TX, V> x[TW];
#pragma unroll
    for (int j = 0; j < TW; ++j) x[j].load(a.X, (int64_t)min(t0 + j, a.T - 1) * H + k);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < TW; ++j) acc[j] = fma((double)x[j][i], (double)w[i], acc[j]);
  }
#pragma unroll
  for (int j = 0; j < TW; ++j) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) acc[j] += __shfl_xor(acc[j], d);
    if (lane == 0) part[wave][j] = acc[j];
  }
  __syncthreads();
  const int j = KW == 4 ? threadIdx.x : lane, t = t0 + j;
  if (j < TW && t < a.T) {
    a.logits[(int64_t)t * a.E + e] = KW == 4 ? ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j] : part[wave][j];
    a.place[e * a.Tp + t] = 0;
  }
}

// ---------------------------------------------------------------------------
// Choice, a block a token.  Order: the larger key, then the lower index; NaN
// comes after every number.  An expert's place is the number of experts before
// it, counted by all threads at once: E^2 comparisons, but no chain of
// reductions.  (128 experts, 8 of them: 4 to 4.8 us, k rounds of a wavefront's argmax
// 9.4 us.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t order_key(double x) {
  if (x != x) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);  // -0 and 0 are equal
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// A sigmoid over exp(m), m = min(0, the largest logit that a token chose) where its weights are normalised, else 0:
// with 1 for the largest of small scores the quotient is what it is however far down the logits lie (in fp32, and
// undivided, scores were subnormal from logits of -88 on and all 0 from -104 on).
__device__ __forceinline__ double sigmoid_over(double l, double m) {
  return l > 0.0 ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / (1.0 + exp(l));
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

__device__ __forceinline__ void choose(const MoeArgs& a, int t, const double* l) {
  __shared__ uint64_t key[kMaxE];
  __shared__ int place[kMaxE];
  __shared__ double chosen_l[kMaxK];
  __shared__ int chosen[kMaxK];
  const int tid = threadIdx.x;
  const bool sig = a.score == LORA_SCORE_SIGMOID;
  double mine = 0.0;
  if (tid < a.E) {
    mine = l[tid];
    key[tid] = order_key(a.bias ? 1.0 / (1.0 + exp(-mine)) + (double)a.bias[tid] : mine);
    place[tid] = 0;
  }
  __syncthreads();
  // thread (e, part) counts over a part of the experts
  int per = 64;
  while (per < a.E) per *= 2;
  const int parts = kMaxE / per, part = tid / per, e = tid % per;
  if (e < a.E) {
    const int j0 = a.E * part / parts, j1 = a.E * (part + 1) / parts;
    const uint64_t k = key[e];
    int before = 0;
#pragma unroll 4
    for (int j = j0; j < j1; ++j) before += key[j] + (j < e) > k;  // no key is the largest integer
    if (parts > 1) atomicAdd(&place[e], before);
    else place[e] = before;
  }
  __syncthreads();
  if (tid < a.E && place[tid] < a.k) {
    chosen[place[tid]] = tid;
    chosen_l[place[tid]] = mine;
  }
  __syncthreads();
  if (tid >= 64) return;
  const bool routed = tid < a.k;
  float w;  // sigmoids and their quotient are fp64, rounded once
  if (sig) {
    double m = routed && a.normalize ? chosen_l[tid] : -INFINITY;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmax(m, __shfl_xor(m, d));
    const double s = routed ? sigmoid_over(chosen_l[tid], a.normalize ? fmin(m, 0.0) : 0.0) : 0.0;
    const double sum = a.normalize ? wave_sum(s) : 1.0;
    w = (float)(s / sum * (double)a.scale);
  } else {
    const double top = chosen_l[0];
    w = routed ? expf((float)(chosen_l[tid] - top)) : 0.0f;
    float sum = w;
    if (!a.normalize) {
      sum = 0.0f;
      for (int i = tid; i < a.E; i += 64) sum += expf((float)(l[i] - top));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    w = w / sum * a.scale;
  }
  if (tid < a.kk) {
    a.ids[t * a.kk + tid] = routed ? chosen[tid] : a.E + tid - a.k;
    if (routed) a.place[chosen[tid] * a.Tp + t] = (uint8_t)(tid + 1);
    a.w[t * a.kk + tid] = routed ? w : 1.0f;
  }
}
__global__ __launch_bounds__(kMaxE) void moe_select_kernel(const MoeArgs a) {
  choose(a, blockIdx.x, a.logits + (int64_t)blockIdx.x * a.E);
}

// Logits and choice of a token in one block, where the router is small and a launch costs more
// than every block's reading of it: a wavefront has four experts at a time, so 32 of them are a round trip.
// (GPU us a call, against two launches: 17 tokens, fp32 router of 10 x 250: 16.5 and 17.7; 160 tokens, 32 x 1024 in bf16,
// 33.9 and 35.6; 40 tokens, 100 x 1024, 61.4 and 59.2; 60 tokens in fp32, 64 x 128 17.5 and 18.7, 80 x 128 19.3 and 18.7,
// 256 x 64 31.5 and 24.8; in bf16, 512 x 64 59.8 and 40.7.)
constexpr int64_t kRouteBytes = 64 * 1024;
constexpr int kRouteE = 64;
template <typename TX, typename TR, int V>
__global__ __launch_bounds__(kMaxE) void moe_route_kernel(const MoeArgs a) {
  constexpr int EW = 4, WAVES = kMaxE / 64;
  __shared__ double l[kMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
  for (int e0 = wave * EW; e0 < a.E; e0 += WAVES * EW) {
    double acc[EW];
#pragma unroll
    for (int j = 0; j < EW; ++j) acc[j] = 0.0;
#pragma unroll 2
    for (int64_t k = lane * V; k < a.H; k += 64 * V) {
      Vec<TX, V> x;
      x.load(a.X, (int64_t)t * a.H + k);
      Vec<TR, V> w[EW];
#pragma unroll
      for (int j = 0; j < EW; ++j) w[j].load(a.router, (int64_t)min(e0 + j, a.E - 1) * a.H + k);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < EW; ++j) acc[j] = fma((double)x[i], (double)w[j][i], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < EW; ++j) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) acc[j] += __shfl_xor(acc[j], d);
      if (lane == 0 && e0 + j < a.E) l[e0 + j] = acc[j];
    }
  }
  if ((int)threadIdx.x < a.E) a.place[threadIdx.x * a.Tp + t] = 0;
  __syncthreads();
  choose(a, t, l);
}

// ---------------------------------------------------------------------------
// The expert of a block and its rows, as entries t kk + j of the choices in
// ascending order; every wavefront makes its own list.  Returns their number,
// 0 also where another block has the expert.  One line of the table of places
// is all it takes (lists made from ids, T kk of them, cost a block seven round
// trips at 160 tokens of 10, more than its products).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int list_rows(const MoeArgs& a, int unit, uint16_t* rows, int lane, int& expert) {
  uint32_t at = 0;  // places of tokens 4 lane .. 4 lane + 3, a byte each
  int self = 0;
  if (unit >= a.routed) {
    expert = a.E + unit - a.routed;
    at = 0x01010101u * (uint32_t)(a.k + unit - a.routed + 1);
  } else {
    expert = unit;
    if (a.by_slot) {  // an expert is left to the first token that chose it
      self = unit / a.k;
      expert = __builtin_amdgcn_readfirstlane(a.ids[self * a.kk + unit % a.k]);
    }
    if (4 * lane < a.T) at = *reinterpret_cast<const uint32_t*>(a.place + expert * a.Tp + 4 * lane);
  }
  uint64_t has[4];
  int before = 0, count = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    has[i] = __ballot(4 * lane + i < a.T && ((at >> (8 * i)) & 255) != 0);
    before += __builtin_popcountll(has[i] & ((1ull << lane) - 1));
    count += __builtin_popcountll(has[i]);
  }
  if (a.by_slot && unit < a.routed)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (has[i] != 0 && 4 * __builtin_ctzll(has[i]) + i < self) return 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((has[i] >> lane) & 1) rows[before++] = (uint16_t)((4 * lane + i) * a.kk + (int)((at >> (8 * i)) & 255) - 1);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return count;
}

// The unit of a block, the first of its rows and the way to the next, `rows` at a time.
// Shared experts, which have every row, come first (last: 160 tokens on 8 + 2 of 128 experts of
// 2048 x 768 274 against 239 us), blocks that may find no row of their expert last.
__device__ __forceinline__ int unit_of(const MoeArgs& a, int rows, int& first, int& step) {
  int y = blockIdx.y;
  const bool shared = y < a.shared * a.cs;
  if (!shared) y -= a.shared * a.cs;
  const int n = shared ? a.shared : a.routed;
  first = y / n * rows;
  step = (shared ? a.cs : a.cr) * rows;
  return y % n + (shared ? a.routed : 0);
}

// The same for calls of up to 8 tokens and 16 experts, from the choices
// themselves, at most 128: one round trip, where an expert named by a choice and
// its line of the table are two (0.7 us each).
__device__ __forceinline__ int list_rows_few(const MoeArgs& a, int unit, uint16_t* rows, int lane, int& expert) {
  const int n = a.T * a.kk;
  int id[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) id[q] = 64 * q + lane < n ? a.ids[64 * q + lane] : -1;
  int self = 0;
  expert = unit < a.routed ? unit : a.E + unit - a.routed;
  if (a.by_slot && unit < a.routed) {
    self = unit / a.k * a.kk + unit % a.k;
    expert = __builtin_amdgcn_readlane(self < 64 ? id[0] : id[1], self & 63);
  }
  const uint64_t m0 = __ballot(id[0] == expert), m1 = __ballot(id[1] == expert);
  if (a.by_slot && unit < a.routed && (m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(m1)) < self) return 0;
  const uint64_t below = (1ull << lane) - 1;
  if (id[0] == expert) rows[__builtin_popcountll(m0 & below)] = (uint16_t)lane;
  if (id[1] == expert) rows[__builtin_popcountll(m0) + __builtin_popcountll(m1 & below)] = (uint16_t)(64 + lane);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return __builtin_popcountll(m0) + __builtin_popcountll(m1);
}

// ---------------------------------------------------------------------------
// Products of up to 8 rows (bf16): the 4 x 4 x 4 MFMA, whose 16 blocks take 16
// runs of 8 inputs of the same 4 outputs and 4 rows.  A load is then 256
// consecutive bytes of each of 4 weight rows, which HBM and the vector cache
// like much better than the 64 bytes of each of 16 rows that a 16 x 16 tile
// takes from registers: reading alone 6.9 against 5.8 TB/s.  Weights pass the
// caches by (without the hint 6.3 TB/s); they are read once.
// A wavefront has NW such tiles of outputs and XT of rows (NX parts of each, by
// precision), U steps of 128 inputs in flight.
// ---------------------------------------------------------------------------
constexpr int kStep4 = 128;
typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mul4(u32x4 w, u32x4 x, f32x4 acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    acc = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4_t, u32x2{w[2 * i], w[2 * i + 1]}),
                                                 __builtin_bit_cast(s16x4_t, u32x2{x[2 * i], x[2 * i + 1]}), acc, 0, 0, 0);
  return acc;
}

// acc[i][m] += W_i X_m^T over the steps s0 .. s1 - 1 of K inputs.
template <int NW, int NX, int XT, int U>
__device__ __forceinline__ void products4(const uint16_t* const (&wp)[NW], const uint16_t* const (&xp)[NX][XT], const bool (&xin)[XT],
                                          int s0, int s1, int K, int lane, f32x4 (&acc)[NW][XT]) {
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int m = 0; m < XT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  for (int s = s0; s < s1; s += U) {
    u32x4 w[U][NW], x[U][NX][XT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && s + u >= s1) continue;  // uniform
      const int k = (s + u) * kStep4 + (lane >> 2) * 8;
      const bool in = k < K;  // K is a multiple of 64: the last step may be half
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        w[u][i] = u32x4{0, 0, 0, 0};
        if (in) w[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[i] + k));
      }
#pragma unroll
      for (int p = 0; p < NX; ++p)
#pragma unroll
        for (int m = 0; m < XT; ++m) {
          x[u][p][m] = u32x4{0, 0, 0, 0};
          if (in && xin[m]) x[u][p][m] = *reinterpret_cast<const u32x4*>(xp[p][m] + k);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && s + u >= s1) continue;
#pragma unroll
      for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int m = 0; m < XT; ++m)
#pragma unroll
          for (int p = 0; p < NX; ++p) acc[i][m] = mul4(w[u][i], x[u][p][m], acc[i][m]);
    }
  }
  // over the 16 blocks; every lane has the sums of 4 outputs of row lane % 4
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int m = 0; m < XT; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int d = 4; d < 64; d <<= 1) acc[i][m][v] += __shfl_xor(acc[i][m][v], d);
}

// ---------------------------------------------------------------------------
// Products in fp32 of more rows: 16 x 16 tiles from registers.  A lane has 4 consecutive
// inputs of an operand row; a step of 16 inputs is four MFMAs that take one of
// each lane's inputs (which input of a step is which K index does not matter,
// as long as both operands agree).  Rows begin at any 4-byte address, so the
// 16-byte loads ask for no more; only a last step of fewer than 16 inputs is
// loaded one by one (one by one throughout: 336 us for 160 tokens on 17 experts of
// 1001 x 999, 156 us so).
// ---------------------------------------------------------------------------
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
constexpr int kStepF = 16;

__device__ __forceinline__ f32x4 load4(const float* p, int64_t k, int64_t K, bool whole) {
  f32x4 v;
  if (whole) return *reinterpret_cast<const f32x4_u*>(p + k);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k + i < K ? p[k + i] : 0.0f;
  return v;
}

// acc[i][m] += W_i (16 rows) X_m^T (16 rows) over the steps s0 .. s1 - 1.  U steps
// of loads are in flight together.  A lane ends with outputs 4 g .. 4 g + 3 of
// row c (lane = 16 g + c).
template <int MT, int U, bool TAIL>
__device__ __forceinline__ void product_steps(const float* const (&wp)[2], const float* const (&xp)[MT], const bool (&xin)[MT], int s,
                                              int s1, int64_t K, int g, f32x4 (&acc)[2][MT]) {
  f32x4 w[U][2], x[U][MT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (TAIL && s + u >= s1) continue;  // uniform
    const int64_t k = (int64_t)(s + u) * kStepF + 4 * g;
    const bool whole = !TAIL || (int64_t)(s + u + 1) * kStepF <= K;  // uniform
#pragma unroll
    for (int i = 0; i < 2; ++i) w[u][i] = load4(wp[i], k, K, whole);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      x[u][m] = f32x4{0, 0, 0, 0};
      if (xin[m]) x[u][m] = load4(xp[m], k, K, whole);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (TAIL && s + u >= s1) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[u][i][j], x[u][m][j], acc[i][m], 0, 0, 0);
  }
}
template <int MT>
__device__ __forceinline__ void products(const float* const (&wp)[2], const float* const (&xp)[MT], const bool (&xin)[MT], int s0,
                                         int s1, int64_t K, int g, f32x4 (&acc)[2][MT]) {
  constexpr int U = MT == 2 ? 4 : 2;  // what the registers hold
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  const int whole = (int)std::min<int64_t>(s1, K / kStepF);
  int s = s0;
  for (; s + U <= whole; s += U) product_steps<MT, U, false>(wp, xp, xin, s, s1, K, g, acc);
  for (; s < s1; s += U) product_steps<MT, U, true>(wp, xp, xin, s, s1, K, g, acc);
}

// ---------------------------------------------------------------------------
// Products in fp32 of up to 16 rows: the 4 x 4 x 1 MFMA, whose 16 blocks take 16 runs of 4 inputs
// of the same 4 outputs and 4 rows; a step of 64 inputs is four of them for each
// tile of outputs and of rows.  A load is 256 bytes of each of 4 weight rows, not 64 of each of 16: 40 tokens
// on 4 + 1 of 60 experts of 700 x 900 107 against 131 us, 17 on 3 of 40 of 1001 x 1333 110 against 135;
// from 17 rows on the loads of X outnumber the weights' (fp32, 160 tokens on 2 + 1 of 16 of 1024 x 1024: 155 against
// 107 us).  Rows begin at any 4-byte address, so the 16-byte loads ask
// for no more (buffer loads, whose offsets cost one register a tile; rows that are not
// there lie past the buffer and read zero).  In a last step of fewer than 64
// inputs what is loaded past the row's end is cleared.
// ---------------------------------------------------------------------------
constexpr int kStepF4 = 64, kNt = 2;  // the streaming hint
constexpr uint32_t kNowhere = 0x80000000u;

// W tile i is at woff[i / NB] of wr[i % NB].  The lane's first input of step s is k = 64 s + 4 (lane / 4).
template <int NB, int NW, int XT, int U, bool TAIL>
__device__ __forceinline__ void steps_f32(const brsrc (&wr)[NB], const uint32_t (&woff)[NW / NB], brsrc xr, const uint32_t (&xoff)[XT], int s, int K,
                                          int lane, f32x4 (&acc)[NW][XT]) {
  f32x4 w[U][NW], x[U][XT];
  const int k = s * kStepF4 + (lane >> 2) * 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = (s + u) * kStepF4 * 4;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      w[u][i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(wr[i % NB], TAIL && k >= K ? kNowhere : woff[i / NB], at, kNt));
#pragma unroll
    for (int m = 0; m < XT; ++m)
      x[u][m] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, TAIL && k >= K ? kNowhere : xoff[m], at, 0));
  }
  if constexpr (TAIL) {
#pragma unroll
    for (int j = 1; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < NW; ++i) w[0][i][j] = k + j < K ? w[0][i][j] : 0.0f;
#pragma unroll
      for (int m = 0; m < XT; ++m) x[0][m][j] = k + j < K ? x[0][m][j] : 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int m = 0; m < XT; ++m) acc[i][m] = __builtin_amdgcn_mfma_f32_4x4x1f32(w[u][i][j], x[u][m][j], acc[i][m], 0, 0, 0);
}

// acc[i][m] = W_i X_m^T over the steps s0 .. s1 - 1 of K inputs; each row of 16 lanes has its own sums, of 4 outputs
// of row lane % 4.
template <int NB, int NW, int XT, int U>
__device__ __forceinline__ void products_f32(const brsrc (&wr)[NB], const uint32_t (&woff)[NW / NB], brsrc xr, const uint32_t (&xoff)[XT],
                                             int s0, int s1, int K, int lane, f32x4 (&acc)[NW][XT]) {
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int m = 0; m < XT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  const int whole = min(s1, K / kStepF4);
  int s = s0;
#pragma unroll 1
  for (; s + U <= whole; s += U) steps_f32<NB, NW, XT, U, false>(wr, woff, xr, xoff, s, K, lane, acc);
  if constexpr (U > 1)
#pragma unroll 1
    for (; s < whole; ++s) steps_f32<NB, NW, XT, 1, false>(wr, woff, xr, xoff, s, K, lane, acc);
  if (s < s1) steps_f32<NB, NW, XT, 1, true>(wr, woff, xr, xoff, s, K, lane, acc);
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int m = 0; m < XT; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float t = acc[i][m][v];
        t += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(t), 0x124, 0xf, 0xf, true));  // row_ror:4
        t += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(t), 0x128, 0xf, 0xf, true));  // row_ror:8
        acc[i][m][v] = t;
      }
}

// Sums over a block's four wavefronts, in ascending order, to the first; the
// first LANES lanes hold them.  True where the caller has the result.
template <int LANES, int NW, int MT>
__device__ __forceinline__ bool join(f32x4 (&acc)[NW][MT], f32x4* red, int wave, int lane) {
  if (wave > 0 && lane < LANES)
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) red[(((wave - 1) * NW + i) * MT + m) * LANES + lane] = acc[i][m];
  __syncthreads();
  if (wave > 0) return false;
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] += red[((q * NW + i) * MT + m) * LANES + lane % LANES];
  return true;
}

// Rows of a lane's tiles: row ROWS m + r of the block's list (entry of ids; in: there is one).
template <int MT, int ROWS>
__device__ __forceinline__ void tile_rows(const uint16_t* rows, int count, int r, bool (&in)[MT], int (&slot)[MT]) {
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    in[m] = ROWS * m + r < count;
    slot[m] = in[m] ? rows[ROWS * m + r] : 0;
  }
}

// h of four outputs from n on, of one row.
template <typename T>
__device__ __forceinline__ void store_h(const MoeArgs& a, int slot, int64_t n, f32x4 e, f32x4 u) {
  float h[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float phi;
    act_fwd<sizeof(T) == 4>(a.act, e[v], phi);
    h[v] = phi * u[v];
  }
  if constexpr (sizeof(T) == 2) {
    // Two bf16 parts keep 2^-16 of h, so that Y is rounded once in effect.  The high one is cut off and
    // the low one rounded, so that both have h's sign and an infinity in down is multiplied into the
    // same infinity twice.  That asks for a low part that is a normal number and not zero: where it
    // would be less, the high part goes down a step, which the low one then holds (2^-15 of h is kept where that
    // is below 2^-110); below 2^-118, where a step is less than the smallest normal number, it goes
    // down by that number (h is kept to 2^-134).  h below 2^-125 has no two such parts; its low one may be zero.
    uint32_t hi[4];
    float lo[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t bits = __float_as_uint(h[v]);
      hi[v] = bits & 0xffff0000u;
      if (fabsf(h[v] - __uint_as_float(hi[v])) < 0x1p-126f && fabsf(h[v]) >= 0x1p-125f)
        hi[v] = fabsf(h[v]) >= 0x1p-118f ? hi[v] - 0x10000u : __float_as_uint(h[v] - copysignf(0x1p-126f, h[v])) & 0xffff0000u;
      lo[v] = h[v] - __uint_as_float(hi[v]);
      if (!__builtin_isfinite(h[v])) {
        hi[v] = f2bf(h[v]) << 16;
        lo[v] = h[v];
      }
    }
    uint16_t* out = static_cast<uint16_t*>(a.h) + (int64_t)slot * 2 * a.I + n;
    *reinterpret_cast<u32x2*>(out) = u32x2{(hi[0] >> 16) | hi[1], (hi[2] >> 16) | hi[3]};
    *reinterpret_cast<u32x2*>(out + a.I) = u32x2{pack_bf2(lo[0], lo[1]), pack_bf2(lo[2], lo[3])};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.h) + (int64_t)slot * a.Ip + n) = f32x4{h[0], h[1], h[2], h[3]};
  }
}

// Gate and up by 4 x 4 tiles: a block has 8 outputs, its wavefronts a quarter of
// the inputs each (with 16 or 32 outputs and half or all of the inputs 8 and 11%
// more at one token, 7 and 14% at five).
template <int XT>
__device__ __forceinline__ void up4(const MoeArgs& a, int expert, int count, const uint16_t* rows, f32x4* red) {
  constexpr int G = 2, U = XT == 1 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * (4 * G);
  const int steps = (int)((a.H + kStep4 - 1) / kStep4);
  const uint16_t *wp[2 * G], *xp[1][XT];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int64_t row = (int64_t)expert * a.I + n0 + 4 * i + r;
    wp[2 * i] = static_cast<const uint16_t*>(a.gate) + row * a.H;
    wp[2 * i + 1] = static_cast<const uint16_t*>(a.up) + row * a.H;
  }
  bool in[XT];
  int slot[XT];
  tile_rows<XT, 4>(rows, count, r, in, slot);
#pragma unroll
  for (int m = 0; m < XT; ++m) xp[0][m] = static_cast<const uint16_t*>(a.X) + (int64_t)(slot[m] / a.kk) * a.H;
  f32x4 acc[2 * G][XT];
  products4<2 * G, 1, XT, U>(wp, xp, in, steps * wave / 4, steps * (wave + 1) / 4, (int)a.H, lane, acc);
  if (!join<4, 2 * G, XT>(acc, red, wave, lane) || lane >= 4) return;
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int m = 0; m < XT; ++m)
      if (in[m]) store_h<uint16_t>(a, slot[m], n0 + 4 * i, acc[2 * i][m], acc[2 * i + 1][m]);
}

// fp32, up to 16 rows: of a block's four wavefronts KS share the inputs of the same outputs, 8 of gate and up
// or 16 of down, and their sums meet in LDS.
constexpr int kFewF = 16;
constexpr int kRedF = 2 * 16 * 4 * 9;  // KS = 2: 2 sets of outputs, 16 tiles, 4 rows, 8 parts (KS = 4: 16 * 4 * 17)
template <int XT, bool UP, int KS>
__device__ __forceinline__ void f32_few(const MoeArgs& a, int expert, int count, const uint16_t* rows, f32x4* red) {
  constexpr int NW = 4, G = UP ? NW / 2 : NW, U = XT == 1 ? 4 : XT == 2 ? 3 : 1;  // what the registers hold
  constexpr int P = 4 * KS + 1;  // parts of a sum, and one to spread the banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 3;
  const int64_t K = UP ? a.H : a.I, N = UP ? a.I : a.H;
  const int64_t n0 = (int64_t)blockIdx.x * (4 * G * (4 / KS));
  uint32_t xoff[XT], woff[G];
#pragma unroll
  for (int m = 0; m < XT; ++m) {
    xoff[m] = kNowhere;
    if (4 * m + r < count) {
      const int slot = rows[4 * m + r];
      xoff[m] = (UP ? (uint32_t)(slot / a.kk) * (uint32_t)a.H : (uint32_t)slot * (uint32_t)a.Ip) * 4 + (lane >> 2) * 16;
    }
  }
  // outputs past the last one repeat it and are not stored
#pragma unroll
  for (int i = 0; i < G; ++i)
    woff[i] = (uint32_t)std::min(n0 + 4 * (G * (wave / KS) + i) + r, N - 1) * (uint32_t)K * 4 + (lane >> 2) * 16;
  const brsrc xr = UP ? make_rsrc(a.X, (int64_t)a.T * a.H * 4) : make_rsrc(a.h, (int64_t)a.T * a.kk * a.Ip * 4);
  constexpr int NB = UP ? 2 : 1;
  brsrc wr[NB];
  wr[0] = make_rsrc(static_cast<const float*>(UP ? a.gate : a.down) + (int64_t)expert * N * K, N * K * 4);
  if constexpr (UP) wr[1] = make_rsrc(static_cast<const float*>(a.up) + (int64_t)expert * N * K, N * K * 4);
  const int steps = (int)((K + kStepF4 - 1) / kStepF4), q = wave % KS;
  f32x4 acc[NW][XT];
  products_f32<NB, NW, XT, U>(wr, woff, xr, xoff, steps * q / KS, steps * (q + 1) / KS, (int)K, lane, acc);
  if ((lane & 15) < 4)
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int m = 0; m < XT; ++m) red[((wave / KS * NW + i) * XT * 4 + 4 * m + r) * P + 4 * q + (lane >> 4)] = acc[i][m];
  __syncthreads();
  auto sum = [&](int tile, int row) {
    const f32x4* part = red + (tile * XT * 4 + row) * P;
    f32x4 t = part[0];
#pragma unroll
    for (int j = 1; j < 4 * KS; ++j) t += part[j];
    return t;
  };
  const int i = (int)threadIdx.x / (4 * XT), row = (int)threadIdx.x % (4 * XT);
  const int64_t n = n0 + 4 * i;
  if (i >= G * (4 / KS) || row >= count || n >= N) return;
  if constexpr (UP) store_h<float>(a, rows[row], n, sum(2 * i, row), sum(2 * i + 1, row));
  else *reinterpret_cast<f32x4*>(a.part + (int64_t)rows[row] * a.Hp + n) = sum(i, row);
}

// fp32: a block has 16 outputs of gate and up or 32 of down, its wavefronts a
// quarter of the inputs each (twice the outputs and half the inputs: 5% less at
// 64 tokens on 64 experts of 1024 x 1024, elsewhere up to 47% more).
template <int MT, bool UP>
__device__ __forceinline__ void f32_block(const MoeArgs& a, int expert, int count, const uint16_t* rows, f32x4* red) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int64_t K = UP ? a.H : a.I, N = UP ? a.I : a.H;
  // outputs past the last one repeat it and are not stored
  const int64_t n0 = (int64_t)blockIdx.x * (UP ? 16 : 32);
  const int64_t row = (int64_t)expert * N + std::min(n0 + c, N - 1);
  const float* wp[2];
  if constexpr (UP) {
    wp[0] = static_cast<const float*>(a.gate) + row * K;
    wp[1] = static_cast<const float*>(a.up) + row * K;
  } else {
    wp[0] = static_cast<const float*>(a.down) + row * K;
    wp[1] = static_cast<const float*>(a.down) + ((int64_t)expert * N + std::min(n0 + 16 + c, N - 1)) * K;
  }
  const float* xp[MT];
  bool in[MT];
  int slot[MT];
  tile_rows<MT, 16>(rows, count, c, in, slot);
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = UP ? static_cast<const float*>(a.X) + (int64_t)(slot[m] / a.kk) * a.H : static_cast<const float*>(a.h) + (int64_t)slot[m] * a.Ip;
  const int steps = (int)((K + kStepF - 1) / kStepF);
  f32x4 acc[2][MT];
  products<MT>(wp, xp, in, steps * wave / 4, steps * (wave + 1) / 4, K, g, acc);
  if (!join<64, 2, MT>(acc, red, wave, lane)) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (!in[m]) continue;
    const int64_t n = n0 + 4 * g;
    if constexpr (UP) {
      if (n < N) store_h<float>(a, slot[m], n, acc[0][m], acc[1][m]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (n + 16 * i < N) *reinterpret_cast<f32x4*>(a.part + (int64_t)slot[m] * a.Hp + n + 16 * i) = acc[i][m];
    }
  }
}

// ---------------------------------------------------------------------------
// Products of more rows (bf16): 16 x 16 tiles through LDS.  Each of a block's
// NW wavefronts has 16 weight rows (8 of gate and 8 of up, or 16 of down), the
// block's rows of X are shared; from 33 rows on two wavefronts share their weights and
// halve the rows, so that LDS is read less.  Stages of 64 inputs go from global memory
// straight into a ring of LDS slots, 128 bytes of 8 rows a load: rows of 128
// bytes, 16-byte chunk j of row r at j ^ (r & 7).  A block begins at one of 32
// places of the inputs and goes round: all blocks at the same place of rows
// that lie a power of two apart load from few of HBM's channels (33 tokens on
// experts of 4096 x 14336: 508 us without, 447 us so).  Eight wavefronts take 128 rows at a time
// instead of 64 and load X half as often for the same outputs, four leave two blocks a CU
// that fill each other's gaps (256 tokens: on 2 of 8 of 4096 x 14336 680 against 870 us, on
// 6 + 2 of 64 of 4096 x 1408 457 against 483; 160 on 8 + 1 of 64 of 2048 x 1024, 22 rows an expert, 187
// against 174).
// ---------------------------------------------------------------------------
template <bool UP, int MT, int NW>
struct RingCfg {
  static constexpr int RING = NW == 4 ? 78 * 1024 : 152 * 1024;  // two blocks a CU, or one
  static constexpr int NX = UP ? 1 : 2;                          // h comes in two parts
  static constexpr int WB = NW * 2048, XB = NX * MT * 2048, SB = WB + XB;
  static constexpr int NST = RING / SB;
  static constexpr int XL = XB / NW >= 1024 ? XB / NW / 1024 : 1;     // loads of X a wavefront makes for a stage
  static constexpr int LANES = XB / NW >= 1024 ? 64 : XB / NW / 16;   // with so many lanes
  static constexpr int WR = MT >= 4 ? 2 : 1;  // tiles of weights a wavefront multiplies, by MT / WR of X
};

template <bool UP, int MT, int NW>
__device__ __forceinline__ void ring_block(const MoeArgs& a, int expert, int count, const uint16_t* rows, char* ring) {
  using C = RingCfg<UP, MT, NW>;
  constexpr int NX = C::NX, NST = C::NST, WR = C::WR, M = MT / WR;
  lds_char* const lds = (lds_char*)ring;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t K = UP ? a.H : a.I, N = UP ? a.I : a.H;
  // rows past the last one are not stored
  const int64_t n0 = std::min(((int64_t)blockIdx.x * NW + wave) * (UP ? 8 : 16), N - (UP ? 8 : 16));
  const uint32_t pitch = (uint32_t)(K * 2);
  const int n = (int)(K / 64);
  const int off = n * (int)(blockIdx.x % 32) / 32;
  const int r8 = lane >> 3, chunk = (lane & 7) ^ r8;  // row of 8 and chunk that a lane loads
  const uint32_t woff = (uint32_t)r8 * pitch + (uint32_t)chunk * 16;
  const char *w0, *w1;
  if constexpr (UP) {
    w0 = static_cast<const char*>(a.gate) + ((int64_t)expert * N + n0) * K * 2;
    w1 = static_cast<const char*>(a.up) + ((int64_t)expert * N + n0) * K * 2;
  } else {
    w0 = static_cast<const char*>(a.down) + ((int64_t)expert * N + n0) * K * 2;
    w1 = w0 + 8 * K * 2;
  }
  const i32x4 r0 = rsrc_words(w0, 8 * K * 2), r1 = rsrc_words(w1, 8 * K * 2);
  const i32x4 rx = UP ? rsrc_words(a.X, (int64_t)a.T * a.H * 2) : rsrc_words(a.h, (int64_t)a.T * a.kk * 2 * a.I * 2);
  // The wavefronts share the stage's rows of X (or of its parts one after the other); rows that are not
  // there read zero.
  uint32_t xoff[C::XL], xlds[C::XL];
#pragma unroll
  for (int j = 0; j < C::XL; ++j) {
    const int p0 = (wave * C::XL + j) * C::LANES, row = (p0 + lane) >> 3;  // 16-byte chunks of X before
    const int part = row / (16 * MT), i = row % (16 * MT);
    const int at = (lane & 7) ^ (row & 7);
    xlds[j] = (uint32_t)(C::WB + p0 * 16);
    xoff[j] = 0x80000000u;
    if (i < count) {
      const int slot = rows[i];
      xoff[j] = (UP ? (uint32_t)(slot / a.kk) * pitch : (uint32_t)(2 * slot + part) * pitch) + (uint32_t)at * 16;
    }
  }
  auto issue = [&](int s, int slot) {
    s += off;
    if (s >= n) s -= n;
    const uint32_t base = lds_addr(lds) + slot * C::SB, at = (uint32_t)s * 128;
    dma16_once(r0, woff, base + wave * 2048, at);
    dma16_once(r1, woff, base + wave * 2048 + 1024, at);
    if (C::LANES == 64 || lane < C::LANES)
#pragma unroll
      for (int j = 0; j < C::XL; ++j) dma16(rx, xoff[j], base + xlds[j], at);
  };
  const int g = lane >> 4, c = lane & 15;
  const int wt = wave / WR * WR, mt = wave % WR * M;  // first tiles of weights and of X
  f32x4 acc[WR][M];
#pragma unroll
  for (int i = 0; i < WR; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  for (int s = 0; s < NST - 1 && s < n; ++s) issue(s, s);
  int slot = 0;
  for (int s = 0; s < n; ++s) {
    const int after = n - 1 - s < NST - 2 ? n - 1 - s : NST - 2;
    wait_stages<2 + C::XL, NST - 2>(after);
    __syncthreads();  // stage s is in for every wavefront, and stage s - 1 is no longer read
    if (s + NST - 1 < n) issue(s + NST - 1, slot == 0 ? NST - 1 : slot - 1);
    const lds_char* ws = lds + slot * C::SB + wt * 2048;
    const lds_char* xs = lds + slot * C::SB + C::WB + mt * 2048;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int at = c * 128 + (((4 * q + g) ^ (c & 7)) * 16);
      bf16x8 w[WR];
#pragma unroll
      for (int i = 0; i < WR; ++i) w[i] = __builtin_bit_cast(bf16x8, lds_read16(ws + i * 2048 + at));
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int p = 0; p < NX; ++p) {
          const bf16x8 x = __builtin_bit_cast(bf16x8, lds_read16(xs + (p * MT + m) * 2048 + at));
#pragma unroll
          for (int i = 0; i < WR; ++i) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], x, acc[i][m], 0, 0, 0);
        }
    }
    slot = slot + 1 == NST ? 0 : slot + 1;
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const bool in = 16 * (mt + m) + c < count;
    const int at = in ? rows[16 * (mt + m) + c] : 0;
#pragma unroll
    for (int i = 0; i < WR; ++i) {
      const int64_t n1 = ((int64_t)blockIdx.x * NW + wt + i) * (UP ? 8 : 16) + 4 * g;
      if constexpr (UP) {
        f32x4 u;  // outputs 0 .. 7 are gate's, 8 .. 15 up's
#pragma unroll
        for (int v = 0; v < 4; ++v) u[v] = __shfl_xor(acc[i][m][v], 32);
        if (in && g < 2 && n1 < N) store_h<uint16_t>(a, at, n1, acc[i][m], u);
      } else if (in && n1 < N) {
        *reinterpret_cast<f32x4*>(a.part + (int64_t)at * a.Hp + n1) = acc[i][m];
      }
    }
  }
}

template <bool UP, int NW>
__global__ __launch_bounds__(64 * NW, 2) void moe_ring_kernel(const MoeArgs a) {
  __shared__ __attribute__((aligned(1024))) char ring[RingCfg<UP, 1, NW>::RING];
  __shared__ uint16_t lists[NW][kMaxT];
  constexpr int ROWS = 16 * NW;  // at a time
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int expert;
  int first, step;
  const int count = list_rows(a, unit_of(a, ROWS, first, step), lists[wave], lane, expert);
  for (int row0 = first; row0 < count; row0 += step) {  // the same in every wavefront
    const uint16_t* rows = lists[wave] + row0;
    const int n = min(count - row0, ROWS);
    if (row0 > first) __syncthreads();  // the ring is no longer read
    if (n <= 16) ring_block<UP, 1, NW>(a, expert, n, rows, ring);
    else if (n <= 32) ring_block<UP, 2, NW>(a, expert, n, rows, ring);
    else if (NW == 4 || n <= 64) ring_block<UP, 4, NW>(a, expert, n, rows, ring);
    else if constexpr (NW == 8) ring_block<UP, 8, NW>(a, expert, n, rows, ring);
  }
}

// The choice for one token of up to 128 experts (without a selection bias) by
// every block of gate and up for itself, instead of a launch in between; the first
// block leaves it for the later launch.  Each wavefront counts over a quarter
// of the experts, two a lane.  Returns the expert of this block.  (GPU us a call against
// a launch for it: 8 of 128 experts of 2048 x 768 24.2 and 24.5, 8 + 2 of 64 of 1024 x 256 15.4 and 16.6, 2 of 8 of
// 512 x 256 11.5 and 12.6, from Python 17.5 and 20.8.)
__device__ __forceinline__ int choose_one(const MoeArgs& a, int (*part)[128], int unit, int wave, int lane) {
  const bool sig = a.score == LORA_SCORE_SIGMOID;
  double l[2];
  uint64_t key[2];
  int before[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 64 * i + lane;
    l[i] = e < a.E ? a.logits[e] : 0.0;
    key[i] = e < a.E ? order_key(l[i]) : 0;
  }
  const int j1 = a.E * (wave + 1) / 4;
  for (int j = a.E * wave / 4; j < j1; ++j) {
    const uint64_t of = j < 64 ? key[0] : key[1];
    const uint64_t k = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(of >> 32), j & 63) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int)of, j & 63);
    before[0] += k + (j < lane) > key[0];  // no key is the largest integer
    before[1] += k + (j < 64 + lane) > key[1];
  }
  part[wave][lane] = before[0];
  part[wave][64 + lane] = before[1];
  __syncthreads();
  int place[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 64 * i + lane;
    place[i] = e < a.E ? part[0][e] + part[1][e] + part[2][e] + part[3][e] : a.E;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {
    const uint64_t m = __ballot(place[0] == 0);
    const int at = __builtin_ctzll(m ? m : __ballot(place[1] == 0));
    const double top = __shfl(m ? l[0] : l[1], at);
    float w[2];
    if (sig) {
      double s[2], sum = 0.0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i] = sigmoid_over(l[i], a.normalize ? fmin(top, 0.0) : 0.0);
        if (place[i] < a.k) sum += s[i];
      }
      sum = a.normalize ? wave_sum(sum) : 1.0;
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = (float)(s[i] / sum * (double)a.scale);
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = expf((float)(l[i] - top));
        if (place[i] < (a.normalize ? a.k : a.E)) sum += w[i];
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = w[i] / sum * a.scale;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (place[i] < a.k) {
        a.ids[place[i]] = 64 * i + lane;
        a.w[place[i]] = w[i];
      }
    if (lane < a.shared) {
      a.ids[a.k + lane] = a.E + lane;
      a.w[a.k + lane] = 1.0f;
    }
  }
  if (unit >= a.k) return a.E + unit - a.k;
  const uint64_t m0 = __ballot(place[0] == unit);
  return m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(__ballot(place[1] == unit));
}
__global__ __launch_bounds__(256, 4) void moe_up_one_kernel(const MoeArgs a) {
  __shared__ int part[4][128];
  __shared__ uint16_t rows[4];
  __shared__ f32x4 red[3 * 4 * 4];  // of three wavefronts: 4 tiles, 4 lanes
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (lane == 0) rows[wave] = (uint16_t)blockIdx.y;  // choices and shared experts in order
  const int expert = choose_one(a, part, blockIdx.y, wave, lane);
  up4<1>(a, expert, 1, rows + wave, red);
}

// Gate and up of bf16 calls of up to 8 tokens.
__global__ __launch_bounds__(256, 4) void moe_up_few_kernel(const MoeArgs a) {
  __shared__ uint16_t rows[4][kFewT];
  __shared__ f32x4 red[3 * 4 * 2 * 4];  // of three wavefronts: 4 x 2 tiles, 4 lanes
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int expert;
  const int count = list_rows_few(a, blockIdx.y, rows[wave], lane, expert);
  if (count == 0) return;  // the same in every wavefront
  if (count <= 4) up4<1>(a, expert, count, rows[wave], red);
  else up4<2>(a, expert, count, rows[wave], red);
}

// fp32 calls of up to 16 tokens: blocks of half the outputs (700 x 900: 1 token on 4 of 40 experts 24 against 27 us
// a call, 4 on 4 + 1 of 40 44 against 46).
template <bool UP>
__global__ __launch_bounds__(256, 4) void moe_f32_few_kernel(const MoeArgs a) {
  __shared__ uint16_t lists[4][kMaxT];
  __shared__ f32x4 red[kRedF];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int expert;
  const int n = list_rows(a, blockIdx.y, lists[wave], lane, expert);
  if (n == 0) return;  // the same in every wavefront
  if (n <= 4) f32_few<1, UP, 4>(a, expert, n, lists[wave], red);
  else if (n <= 8) f32_few<2, UP, 4>(a, expert, n, lists[wave], red);
  else f32_few<4, UP, 4>(a, expert, n, lists[wave], red);
}

// fp32 calls of more.
template <bool UP>
__global__ __launch_bounds__(256, 3) void moe_f32_kernel(const MoeArgs a) {
  __shared__ uint16_t lists[4][kMaxT];
  __shared__ f32x4 red[3 * 2 * 4 * 64];
  static_assert(kRedF <= 3 * 2 * 4 * 64);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int expert;
  int first, step;
  const int count = list_rows(a, unit_of(a, kRows, first, step), lists[wave], lane, expert);
  for (int row0 = first; row0 < count; row0 += step) {  // the same in every wavefront
    const uint16_t* rows = lists[wave] + row0;
    const int n = min(count - row0, kRows);
    if (row0 > first) __syncthreads();  // red is no longer read
    if (n <= 4) f32_few<1, UP, 2>(a, expert, n, rows, red);
    else if (n <= 8) f32_few<2, UP, 2>(a, expert, n, rows, red);
    else if (n <= 16) f32_few<4, UP, 2>(a, expert, n, rows, red);
    else if (n <= 32) f32_block<2, UP>(a, expert, n, rows, red);
    else f32_block<4, UP>(a, expert, n, rows, red);
  }
}

// Down and the sum in one, for bf16 calls of up to 8 tokens: a block has 4 NW
// outputs of every token, its 16 wavefronts share the experts and, where there
// are fewer experts than wavefronts, their inputs; the products meet in LDS.
template <int NW>
__global__ __launch_bounds__(1024) void moe_down_sum_kernel(const MoeArgs a) {
  __shared__ uint16_t rows[16][kFewT];
  __shared__ f32x4 prod[kSumSlots * NW];  // by part of the inputs, entry of ids, tile
  __shared__ float weight[kSumSlots];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 3;
  const int slots = a.T * a.kk;
  if (threadIdx.x < slots) weight[threadIdx.x] = a.w[threadIdx.x];
  int kp = 1;  // of units <= 16 / kp, and no token has more choices: kp slots <= kSumSlots
  while (kp < 4 && 2 * kp * a.units <= kFewUnits) kp *= 2;
  const int part = wave % kp, steps = (int)((a.I + kStep4 - 1) / kStep4);
  const int64_t n0 = (int64_t)blockIdx.x * (4 * NW);
  if (const int unit = wave / kp; unit < a.units) {
    int expert;
    const int count = list_rows_few(a, unit, rows[wave], lane, expert);
    const uint16_t* wp[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) wp[i] = static_cast<const uint16_t*>(a.down) + ((int64_t)expert * a.H + n0 + 4 * i + r) * a.I;
    auto run = [&](auto xt) {
      constexpr int XT = decltype(xt)::value;
      const uint16_t* xp[2][XT];
      bool in[XT];
      int slot[XT];
      tile_rows<XT, 4>(rows[wave], count, r, in, slot);
#pragma unroll
      for (int m = 0; m < XT; ++m)
#pragma unroll
        for (int p = 0; p < 2; ++p) xp[p][m] = static_cast<const uint16_t*>(a.h) + (int64_t)(2 * slot[m] + p) * a.I;
      f32x4 acc[NW][XT];
      products4<NW, 2, XT, XT == 1 ? 16 / (NW + 2) : 2>(wp, xp, in, steps * part / kp, steps * (part + 1) / kp, (int)a.I, lane, acc);
#pragma unroll
      for (int m = 0; m < XT; ++m)
        if (in[m] && lane < 4)
#pragma unroll
          for (int i = 0; i < NW; ++i) prod[(part * slots + slot[m]) * NW + i] = acc[i][m];
    };
    if (count > 4) run(std::integral_constant<int, 2>());
    else if (count > 0) run(std::integral_constant<int, 1>());
  }
  __syncthreads();
  if (threadIdx.x < a.T * NW) {
    const int t = threadIdx.x / NW, i = threadIdx.x % NW;
    f32x4 y = {0, 0, 0, 0};
    for (int j = 0; j < a.kk; ++j) {
      const int at = t * a.kk + j;
      f32x4 p = prod[at * NW + i];
      for (int q = 1; q < kp; ++q) p += prod[(q * slots + at) * NW + i];
      y += weight[at] * p;
    }
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.Y) + t * a.H + n0 + 4 * i) = u32x2{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
  }
}

// Y[t] = sum over j of w[t, j] part[t, j], in ascending order; four columns a thread.
template <typename T>
__global__ __launch_bounds__(64) void moe_sum_kernel(const MoeArgs a) {
  const int t = blockIdx.y;
  const int64_t n = ((int64_t)blockIdx.x * 64 + threadIdx.x) * 4;
  if (n >= a.H) return;
  constexpr int AHEAD = 8;  // loaded together (past the last one it is read again)
  f32x4 y = {0, 0, 0, 0};
  for (int j0 = 0; j0 < a.kk; j0 += AHEAD) {
    f32x4 p[AHEAD];
    float w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int at = t * a.kk + min(j0 + i, a.kk - 1);
      w[i] = a.w[at];
      p[i] = *reinterpret_cast<const f32x4*>(a.part + (int64_t)at * a.Hp + n);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (j0 + i < a.kk) y += w[i] * p[i];
  }
  T* out = static_cast<T*>(a.Y) + t * a.H + n;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < a.H) out[v] = y[v];
  }
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
template <typename TX, typename TR, int V>
hipError_t launch_route(const MoeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((moe_route_kernel<TX, TR, V>), dim3((unsigned)a.T), dim3(kMaxE), 0, st, a);
  return hipGetLastError();
}
template <typename TX, typename TR, int V>
hipError_t launch_logits(const MoeArgs& a, hipStream_t st) {
  const unsigned y = (unsigned)cdiv(a.T, 4), four = (unsigned)cdiv(a.E, 4);
  if (a.T <= 2) hipLaunchKernelGGL((moe_logits_kernel<TX, TR, V, 1, 4>), dim3((unsigned)a.E, (unsigned)a.T), dim3(256), 0, st, a);
  else if (a.E * y < 1024) hipLaunchKernelGGL((moe_logits_kernel<TX, TR, V, 4, 4>), dim3((unsigned)a.E, y), dim3(256), 0, st, a);
  else hipLaunchKernelGGL((moe_logits_kernel<TX, TR, V, 4, 1>), dim3(four, y), dim3(256), 0, st, a);
  return hipGetLastError();
}

// Several blocks share an expert's rows where there are few blocks otherwise (n for each expert): a
// shared expert's all, a routed one's twice what falls to it if experts are chosen evenly (rows past
// that are done in turn).  160 tokens: on 2 + 1 of 4 of 1024 x 512 29 against 48 us; fp32, on 2 + 1 of 16 of
// 1024 x 1024, 105 against 144; without the limit on n no gain, and up to 3 us of empty blocks.
void split_rows(MoeArgs& a, int64_t n, int64_t at_once) {
  a.cs = a.cr = 1;
  if (n * a.units >= 2048) return;
  a.cs = (int32_t)cdiv(a.T, at_once);
  a.cr = (int32_t)cdiv(std::min(a.T, std::max(1, 2 * a.T * a.k / a.E)), at_once);
}
// Eight wavefronts where experts have many rows and there are blocks enough.
template <bool UP>
hipError_t launch_ring(MoeArgs a, hipStream_t st) {
  const int64_t N = UP ? a.I : a.H, n = N / (UP ? 32 : 64);
  const bool wide = a.T > kRows && a.T * a.kk >= 30 * a.units && n * a.units >= 512;
  split_rows(a, n, wide ? 2 * kRows : kRows);
  if (wide) {
    const dim3 grid((unsigned)cdiv(N, UP ? 64 : 128), (unsigned)(a.shared * a.cs + a.routed * a.cr));
    hipLaunchKernelGGL((moe_ring_kernel<UP, 8>), grid, dim3(512), 0, st, a);
  } else {
    const dim3 grid((unsigned)n, (unsigned)(a.shared * a.cs + a.routed * a.cr));
    hipLaunchKernelGGL((moe_ring_kernel<UP, 4>), grid, dim3(256), 0, st, a);
  }
  return hipGetLastError();
}
bool choose_in_up(const MoeArgs& a) { return a.T == 1 && a.units <= kFewUnits && a.k < a.E && a.E <= 128 && a.bias == nullptr; }
hipError_t launch_up_one(const MoeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(moe_up_one_kernel, dim3((unsigned)(a.I / 8), (unsigned)a.units), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_up_few(const MoeArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(moe_up_few_kernel, dim3((unsigned)(a.I / 8), (unsigned)a.units), dim3(256), 0, st, a);
  return hipGetLastError();
}
// 16 outputs a block where that makes a block for every CU, else 8 (2048 outputs: 28 against 31 us a
// call, 4096: 175 against 163).
hipError_t launch_down_sum(const MoeArgs& a, hipStream_t st) {
  if (a.H >= 4096) hipLaunchKernelGGL(moe_down_sum_kernel<4>, dim3((unsigned)(a.H / 16)), dim3(1024), 0, st, a);
  else hipLaunchKernelGGL(moe_down_sum_kernel<2>, dim3((unsigned)(a.H / 8)), dim3(1024), 0, st, a);
  return hipGetLastError();
}
template <bool UP>
hipError_t launch_f32(MoeArgs a, hipStream_t st) {
  const int64_t N = UP ? a.I : a.H, n = cdiv(N, UP ? 16 : 32);
  if (a.T <= kFewF) {
    hipLaunchKernelGGL(moe_f32_few_kernel<UP>, dim3((unsigned)cdiv(N, UP ? 8 : 16), (unsigned)a.units), dim3(256), 0, st, a);
    return hipGetLastError();
  }
  split_rows(a, n, kRows);
  hipLaunchKernelGGL(moe_f32_kernel<UP>, dim3((unsigned)n, (unsigned)(a.shared * a.cs + a.routed * a.cr)), dim3(256), 0, st, a);
  return hipGetLastError();
}

struct MoePlan {
  double* logits;
  int32_t* ids;
  float* w;
  uint8_t* place;
  void* h;
  float* part;
  size_t bytes;
};
MoePlan plan_moe(const lora_moe_desc& d, void* ws) {
  MoePlan p{};
  if (d.T == 0) return p;
  const size_t slots = (size_t)d.T * (size_t)(d.top_k + d.shared);
  Ws w(ws);
  p.logits = static_cast<double*>(w.take((size_t)d.T * d.E * 8));
  p.ids = static_cast<int32_t*>(w.take(slots * 4));
  p.w = static_cast<float*>(w.take(slots * 4));
  p.place = static_cast<uint8_t*>(w.take((size_t)d.E * (size_t)(cdiv(d.T, 4) * 4)));
  p.h = w.take(slots * (size_t)(cdiv(d.I, 4) * 4) * 4);
  p.part = static_cast<float*>(w.take(slots * (size_t)(cdiv(d.H, 4) * 4) * 4));
  p.bytes = w.off;
  return p;
}

lora_status check_moe(const lora_moe_desc* d) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16 || d->dtype == LORA_BF16_F32LORA, LORA_EDTYPE, "unknown dtype %d",
        d->dtype);
  CHECK(d->act == LORA_ACT_SWIGLU || d->act == LORA_ACT_GEGLU_TANH, LORA_EINVAL, "unknown activation %d", d->act);
  CHECK(d->score == LORA_SCORE_SOFTMAX || d->score == LORA_SCORE_SIGMOID, LORA_EINVAL, "unknown score %d", d->score);
  CHECK(d->normalize == 0 || d->normalize == 1, LORA_EINVAL, "normalize = %d is not 0 or 1", d->normalize);
  CHECK(std::isfinite(d->scale), LORA_EINVAL, "scale is not finite");
  CHECK(d->T >= 0 && d->T <= kMaxT, LORA_ESHAPE, "T = %lld must be in [0, %d]", (long long)d->T, kMaxT);
  CHECK(d->E > 0 && d->E <= kMaxE, LORA_ESHAPE, "E = %lld must be in [1, %d]", (long long)d->E, kMaxE);
  CHECK(d->shared >= 0 && d->shared <= kMaxShared, LORA_ESHAPE, "shared = %lld must be in [0, %d]", (long long)d->shared,
        kMaxShared);
  CHECK(d->top_k >= 1 && d->top_k <= kMaxK && d->top_k <= d->E, LORA_ESHAPE, "top_k = %d must be in [1, %d] and at most E",
        d->top_k, kMaxK);
  const bool bf16 = d->dtype != LORA_F32;
  CHECK(d->H > 0 && d->I > 0 && d->H <= (1 << 22) && d->I <= (1 << 22), LORA_ESHAPE, "H = %lld and I = %lld must be in [1, %d]",
        (long long)d->H, (long long)d->I, 1 << 22);
  if (bf16)
    CHECK(d->H % 64 == 0 && d->I % 64 == 0, LORA_ESHAPE, "H = %lld and I = %lld must be multiples of 64 for bf16",
          (long long)d->H, (long long)d->I);
  CHECK(d->H <= (((int64_t)1 << 31) - 4096) / (bf16 ? 2 : 4) / d->I, LORA_ESHAPE, "an expert's weight (%lld x %lld) exceeds 2 GiB",
        (long long)d->H, (long long)d->I);
  // loads of X and h through 32-bit byte offsets
  const int64_t lim = ((int64_t)1 << 31) - 4096;
  CHECK(d->T * d->H <= lim / 4 && d->T * (d->top_k + d->shared) * (cdiv(d->I, 4) * 4) <= lim / 4, LORA_ESHAPE,
        "X (%lld rows) or its experts' h (%lld rows) exceeds 2 GiB", (long long)d->T, (long long)(d->T * (d->top_k + d->shared)));
  return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_moe_workspace_size(const lora_moe_desc* d, size_t* bytes) {
  TRY(check_moe(d));
  if (bytes) *bytes = plan_moe(*d, nullptr).bytes;
  return LORA_OK;
}

lora_status lora_moe_fwd(const lora_moe_desc* d, const void* X, const void* router, const float* bias, const void* gate,
                         const void* up, const void* down, void* Y, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_moe(d));
  const bool bf16 = d->dtype != LORA_F32, sig = d->score == LORA_SCORE_SIGMOID;
  if (d->T == 0) return LORA_OK;
  const size_t es = bf16 ? 2 : 4, al = bf16 ? 16 : 4, rs = d->dtype == LORA_BF16 ? 2 : 4;
  const size_t nx = (size_t)d->T * d->H * es, nw = (size_t)(d->E + d->shared) * d->H * d->I * es;
  const size_t need = plan_moe(*d, nullptr).bytes;
  CHECK(X && router && gate && up && down && Y, LORA_EINVAL, "X, router, gate, up, down or Y is NULL");
  CHECK(bias == nullptr || sig, LORA_EINVAL, "a selection bias needs sigmoid scores");
  CHECK(aligned(X, al) && aligned(router, al) && aligned(gate, al) && aligned(up, al) && aligned(down, al) && aligned(Y, al),
        LORA_EALIGN, "X, router, gate, up, down or Y is not %d-byte aligned", (int)al);
  CHECK(aligned(bias, 4), LORA_EALIGN, "bias is not 4-byte aligned");
  TRY(check_ws(ws, ws_bytes, need));
  const struct {
    const void* p;
    size_t bytes;
  } in[] = {{X, nx}, {router, (size_t)d->E * d->H * rs}, {bias, bias ? (size_t)d->E * 4 : 0}, {gate, nw}, {up, nw}, {down, nw}};
  for (const auto& b : in)
    CHECK(b.bytes == 0 || (!overlaps(Y, nx, b.p, b.bytes) && !overlaps(ws, need, b.p, b.bytes)), LORA_EUNSUPPORTED,
          "Y or the workspace overlaps an input");
  CHECK(!overlaps(Y, nx, ws, need), LORA_EUNSUPPORTED, "Y overlaps the workspace");

  hipStream_t st = static_cast<hipStream_t>(stream);
  const MoePlan p = plan_moe(*d, ws);
  MoeArgs a{};
  a.X = X;
  a.router = router;
  a.gate = gate;
  a.up = up;
  a.down = down;
  a.bias = bias;
  a.Y = Y;
  a.logits = p.logits;
  a.ids = p.ids;
  a.w = p.w;
  a.place = p.place;
  a.h = p.h;
  a.part = p.part;
  a.H = d->H;
  a.I = d->I;
  a.Hp = cdiv(d->H, 4) * 4;
  a.Ip = cdiv(d->I, 4) * 4;
  a.T = (int32_t)d->T;
  a.Tp = (int32_t)(cdiv(d->T, 4) * 4);
  a.E = (int32_t)d->E;
  a.k = d->top_k;
  a.kk = d->top_k + (int32_t)d->shared;
  a.shared = (int32_t)d->shared;
  a.by_slot = d->T * d->top_k < d->E;
  a.routed = a.by_slot ? a.T * a.k : a.E;
  a.units = a.routed + a.shared;
  a.act = d->act;
  a.score = d->score;
  a.normalize = d->normalize;
  a.scale = d->scale;
  // the router's 16-byte loads in fp32: whole vectors in every row, at aligned addresses
  const bool vx = d->H % 4 == 0 && aligned(X, 16) && aligned(router, 16);
  const bool one = bf16 && choose_in_up(a);
  const bool route = !one && d->E <= kRouteE && d->E * d->H * (int64_t)rs <= kRouteBytes;
  if (route) {
    if (d->dtype == LORA_BF16) LAUNCHN("moe_route", st, (launch_route<uint16_t, uint16_t, 8>(a, st)));
    else if (bf16) LAUNCHN("moe_route", st, (launch_route<uint16_t, float, 8>(a, st)));
    else if (vx) LAUNCHN("moe_route", st, (launch_route<float, float, 4>(a, st)));
    else LAUNCHN("moe_route", st, (launch_route<float, float, 1>(a, st)));
  } else if (d->dtype == LORA_BF16) LAUNCHN("moe_logits", st, (launch_logits<uint16_t, uint16_t, 8>(a, st)));
  else if (bf16) LAUNCHN("moe_logits", st, (launch_logits<uint16_t, float, 8>(a, st)));
  else if (vx) LAUNCHN("moe_logits", st, (launch_logits<float, float, 4>(a, st)));
  else LAUNCHN("moe_logits", st, (launch_logits<float, float, 1>(a, st)));
  if (one) {
    LAUNCHN("moe_up_one", st, launch_up_one(a, st));
    LAUNCHN("moe_down_sum", st, launch_down_sum(a, st));
    return LORA_OK;
  }
  if (!route) {
    TraceScope ts("moe_select", st);
    hipLaunchKernelGGL(moe_select_kernel, dim3((unsigned)a.T), dim3(kMaxE), 0, st, a);
    LAUNCH(hipGetLastError());
  }
  if (bf16 && a.T <= kFewT && a.units <= kFewUnits) {
    LAUNCHN("moe_up_few", st, launch_up_few(a, st));
    LAUNCHN("moe_down_sum", st, launch_down_sum(a, st));
    return LORA_OK;
  }
  if (bf16) LAUNCHN("moe_up", st, launch_ring<true>(a, st));
  else LAUNCHN("moe_up_f32", st, launch_f32<true>(a, st));
  if (bf16) LAUNCHN("moe_down", st, launch_ring<false>(a, st));
  else LAUNCHN("moe_down_f32", st, launch_f32<false>(a, st));
  TraceScope ts("moe_sum", st);
  const dim3 grid((unsigned)cdiv(d->H, 256), (unsigned)a.T);
  if (bf16) hipLaunchKernelGGL(moe_sum_kernel<uint16_t>, grid, dim3(64), 0, st, a);
  else hipLaunchKernelGGL(moe_sum_kernel<float>, grid, dim3(64), 0, st, a);
  LAUNCH(hipGetLastError());
  return LORA_OK;
}

}  // extern "C"
