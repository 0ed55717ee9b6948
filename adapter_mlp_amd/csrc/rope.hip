// Norms of queries and keys for each head with the rotation by position in
// the same pass, between the Q/K/V projections and attention:
//   n = v rms(v)^-1 (o + w)           rms(v)^2 = mean(v^2) + eps over a head (or n = v)
//   (x, y) -> m (x cos a - y sin a, x sin a + y cos a)     for rot / 2 pairs of n,
//   a = pos[t, axis[i]] freq[i]
// and the gradients of both.
//
// HBM-bound: a head is read and written once (backward: also its gradient
// read), some 15 operations an element.  A lane owns V pairs of a head, both
// elements of each, so that the rotation stays within the lane and the sum of
// the squares is the only exchange: d / 2V lanes of a wavefront hold a head,
// and a wavefront works on 64 / lanes heads of one token at a time, all of
// which share the angles.  Those are formed once for a token (and head chunk),
// one pair a lane, and handed to the owners through LDS.
#include <algorithm>
#include <cmath>

#include "abi.hpp"
#include "common.hpp"
#include "vec.hpp"

namespace lora {
namespace {

constexpr int kMaxD = 512;       // head width
// Blocks side by side: what the registers let run at once, with as many tokens
// for each (a block for every four tokens: 4099 tokens 20.3 us, so 18.1; 8192: 40.6
// and 38.6).
constexpr int kFwdBlocks = 1024;
constexpr int kBwdBlocks = 768;  // of a backward pass with a norm

// One of q and k: rows (t, h) of d elements at p + t st + h sh.
struct HeadSet {
  const void *v, *dv;  // input and (backward) the gradient of the output
  void* out;           // output, or the input's gradient
  const void* w;       // norm weight, nullptr: no norm
  float* part;         // backward: [blocks, d] sums of the weight's gradient
  int64_t v_st, v_sh, dv_st, dv_sh, out_st, out_sh;
  int32_t h, iters;    // heads, and wavefront steps that they take
  // backward: the blocks from block0 on work on this set, gx of them side by side on every chunk of `steps`
  int32_t block0, gx, steps;
};
struct RopeArgs {
  HeadSet set[2];
  int64_t T;
  const int32_t *pos, *axis;
  const float* freq;
  int64_t pos_st, pos_sa;
  int32_t d, rot, axes;
  int32_t lanes;          // lanes of a head (a power of two)
  int32_t steps;          // forward, blockIdx.y: a token's wavefront steps are cut into chunks of `steps`
  float scale, eps, offset;
};

// cos and sin of a position's angle, times scale; per = quarter turns a
// position.  The angle is reduced to x, an eighth of a turn at most, in fp64: at
// position 2^31 the product holds the angle to 2^-19, the reduction here to
// 2^-24.  There the Taylor series of sin and cos of pi / 2 x end: the next terms are
// below 2e-9 and 2e-10.
__device__ __forceinline__ float2 turn(int pos, double per, float scale) {
  const double quarters = (double)pos * per;
  const double q = rint(quarters);
  const float x = (float)(quarters - q), z = x * x;
  const float s = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.6044118e-4f, -4.6817541e-3f), 7.9692626e-2f), -6.4596410e-1f), 1.5707963f);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.5202042e-5f, 9.1926027e-4f), -2.0863481e-2f), 2.5366951e-1f), -1.2337006f), 1.0f);
  const int k = (int)(q - 4.0 * floor(q * 0.25));
  const float u = (k & 1) ? s : c, v = (k & 1) ? c : s;
  return float2{(k == 1 || k == 2) ? -scale * u : scale * u, k >= 2 ? -scale * v : scale * v};
}

// The pair that a lane forms the angles of: of every 64 the one at its place.
struct Pair {
  double per;
  int64_t at;  // of its axis in a token's positions; < 0: not turned
  __device__ __forceinline__ Pair(const RopeArgs& a, int i) {
    per = 0.0;
    at = -1;
    if (i >= a.rot / 2) return;
    const int ax = a.axis ? a.axis[i] : 0;
    if (ax < 0 || ax >= a.axes) return;
    at = ax * a.pos_sa;
    per = (double)a.freq[i] * 0.63661977236758134308;
  }
  __device__ __forceinline__ int pos(const RopeArgs& a, int64_t t) const { return at >= 0 && t < a.T ? a.pos[t * a.pos_st + at] : 0; }
};

// The wavefront's table of a token: entry i = (cos, sin) of pair i.  The first
// 64 pairs' constants and position are at hand.
__device__ __forceinline__ void fill_turns(const RopeArgs& a, int64_t t, float2* table, int lane, const Pair& own, int pos) {
  __builtin_amdgcn_wave_barrier();  // the table's last readers are done
  if (lane < a.rot / 2) table[lane] = turn(pos, own.per, a.scale);
  for (int i = lane + 64; i < a.rot / 2; i += 64) {
    const Pair p(a, i);
    table[i] = turn(p.pos(a, t), p.per, a.scale);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// What a lane owns of a head: unit u holds the elements e[0 .. V-1] at `first`
// and e[V .. 2V-1] at `second`; its pair j is (e[j], e[V + j]), or with PAIRS
// (e[2j], e[2j + 1]).  Units past the rotated ones pass through.
template <int V>
struct Unit {
  int first, second, pair;  // pair < 0: not turned
  bool ok;
  __device__ __forceinline__ void set(const RopeArgs& a, int u, bool interleaved) {
    const int turned = a.rot / (2 * V);
    ok = u < a.d / (2 * V);
    pair = u < turned ? u * V : -1;
    if (u < turned && !interleaved) {
      first = u * V;
      second = a.rot / 2 + u * V;
    } else {
      first = u * 2 * V;
      second = first + V;
    }
  }
};

template <int V, bool PAIRS>
__device__ __forceinline__ void rotate(float (&e)[2 * V], const float2 (&cs)[V], float sign) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int x = PAIRS ? 2 * j : j, y = PAIRS ? 2 * j + 1 : V + j;
    const float c = cs[j].x, s = sign * cs[j].y, ex = e[x], ey = e[y];
    e[x] = fmaf(ex, c, -ey * s);
    e[y] = fmaf(ex, s, ey * c);
  }
}

template <typename TA, int V, int NU>
struct Raw {
  Vec<TA, V> v[NU][2];
  __device__ __forceinline__ void load(const void* p, int64_t at, const Unit<V> (&u)[NU], bool in) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      v[i][0].zero();
      v[i][1].zero();
      if (in && u[i].ok) {
        v[i][0].load(p, at + u[i].first);
        v[i][1].load(p, at + u[i].second);
      }
    }
  }
  __device__ __forceinline__ float at(int i, int e) const { return v[i][e / V][e % V]; }
};

// Sum over the lanes of a head (a power of two), the same in all of them.  Up to
// 16 lanes by DPP: neighbours, pairs, then mirrored halves and rows, whose lanes
// hold equal sums by then.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
  if (lanes > 1) x += dpp<0xB1>(x);
  if (lanes > 2) x += dpp<0x4E>(x);
  if (lanes > 4) x += dpp<0x141>(x);
  if (lanes > 8) x += dpp<0x140>(x);
  if (lanes > 16) x += __shfl_xor(x, 16);
  if (lanes > 32) x += __shfl_xor(x, 32);
  return x;
}

// A lane's weights, 0 where the set has none.
template <typename TP, int V, int NU>
struct Weights {
  Vec<TP, V> v[NU][2];
  __device__ __forceinline__ void load(const void* w, const Unit<V> (&u)[NU]) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      v[i][0].zero();
      v[i][1].zero();
      if (w && u[i].ok) {
        v[i][0].load(w, u[i].first);
        v[i][1].load(w, u[i].second);
      }
    }
  }
  __device__ __forceinline__ float at(int i, int e) const { return v[i][e / V][e % V]; }
};

// Where a wavefront's step `it` of a token works: the set, and the lane's head.
__device__ __forceinline__ bool place(const RopeArgs& a, int it, int lane, int& k, int& head) {
  k = it >= a.set[0].iters;
  const int per = 64 / a.lanes;
  head = (it - (k ? a.set[0].iters : 0)) * per + lane / a.lanes;
  return head < a.set[k].h;
}

// The angles of a lane's units.
template <int V, int NU>
__device__ __forceinline__ void lane_turns(const RopeArgs& a, const float2* table, const Unit<V> (&u)[NU], float2 (&cs)[NU][V]) {
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) cs[i][j] = u[i].pair >= 0 && u[i].ok ? table[u[i].pair + j] : float2{1.0f, 0.0f};
}

// sign -1: the rotation's inverse of dv (the backward pass without a norm).
// Measured: 8192 tokens of 32 + 8 heads of 128 in bf16, 168 MB: 32 us, 5.3 TB/s (a large
// copy: 4.85, from HBM throughout); one token 4 us, the round trips of its
// loads.  Streaming hints on the stores are 2 us faster here and 4 us slower in
// what reads the heads next, so there are none.  fp32 heads whose width is no
// multiple of eight go one pair a lane, with lanes idle in most heads: 8192 tokens of
// 10 + 2 of 66, 52 MB, 34.6 us (of 64: 50 MB, 17.5).
template <typename TA, typename TP, int V, int NU, bool PAIRS>
__global__ __launch_bounds__(256) void rope_fwd_kernel(const RopeArgs a, const float sign) {
  __shared__ float2 tables[4][kMaxD / 2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2* const table = tables[wave];
  Unit<V> u[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) u[i].set(a, (lane & (a.lanes - 1)) + i * a.lanes, PAIRS);
  const float inv_d = 1.0f / (float)a.d;
  const int i0 = blockIdx.y * a.steps, i1 = min(i0 + a.steps, a.set[0].iters + a.set[1].iters);
  const Pair own(a, lane);
  int of = -1;  // whose weights the lane holds
  Weights<TP, V, NU> w;
  int64_t t = (int64_t)blockIdx.x * 4 + wave;
  int pos = own.pos(a, t);
  for (; t < a.T; t += (int64_t)gridDim.x * 4) {
    Raw<TA, V, NU> next;
    auto fetch = [&](int it) {
      int k, head;
      const bool in = place(a, it, lane, k, head);
      const HeadSet& s = a.set[k];
      next.load(s.v, t * s.v_st + head * s.v_sh, u, in);
    };
    fetch(i0);
    fill_turns(a, t, table, lane, own, pos);
    pos = own.pos(a, t + (int64_t)gridDim.x * 4);
    float2 cs[NU][V];
    lane_turns<V, NU>(a, table, u, cs);
    for (int it = i0; it < i1; ++it) {
      const Raw<TA, V, NU> x = next;
      if (it + 1 < i1) fetch(it + 1);
      int k, head;
      const bool in = place(a, it, lane, k, head);
      const HeadSet& s = a.set[k];
      if (k != of) w.load(a.set[of = k].w, u);
      float r = 1.0f;
      if (s.w) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) q = fmaf(x.at(i, e), x.at(i, e), q);
        r = rsqrtf(fmaf(lanes_sum(q, a.lanes), inv_d, a.eps));
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (!in || !u[i].ok) continue;
        float e[2 * V];
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) e[j] = x.at(i, j);
        if (s.w)
#pragma unroll
          for (int j = 0; j < 2 * V; ++j) e[j] *= r * (a.offset + w.at(i, j));
        if (u[i].pair >= 0) rotate<V, PAIRS>(e, cs[i], sign);
        const int64_t at = t * s.out_st + head * s.out_sh;
        Vec<TA, V>::store(s.out, at + u[i].first, e);
        Vec<TA, V>::store(s.out, at + u[i].second, e + V);
      }
    }
  }
}

// With g the inverse rotation of the output's gradient and n = v / rms(v):
//   dw = sum over tokens and heads of g n
//   dv = (g (o + w) - n mean(g (o + w) n)) / rms(v)       (dv = g without a norm)
// The sums of dw gather in the registers of the lane that owns the element,
// one slice a block, and rope_grad_kernel adds the slices in a fixed order.
// A block works on q or on k, so that a lane holds the sums of one weight; each has
// its share of the blocks.
// Measured: the tokens above with fp32 weights, 252 MB: 49 us, 5.2 TB/s, and 4.7 us to
// add the slices.  (q and k in one block, 157 registers: 83 us at four blocks a CU,
// of which three run, 72 at three; four at 128 registers, which spill: 84.)
template <typename TA, typename TP, int V, int NU, bool PAIRS>
__global__ __launch_bounds__(256, V == 8 ? 3 : 1) void rope_bwd_kernel(const RopeArgs a) {
  __shared__ float2 tables[4][kMaxD / 2];
  __shared__ float sums[4][kMaxD];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2* const table = tables[wave];
  const HeadSet& s = a.set[a.set[1].gx > 0 && (int)blockIdx.x >= a.set[1].block0];
  const int block = (int)blockIdx.x - s.block0;
  Unit<V> u[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) u[i].set(a, (lane & (a.lanes - 1)) + i * a.lanes, PAIRS);
  const float inv_d = 1.0f / (float)a.d;
  const int per = 64 / a.lanes, i0 = block / s.gx * s.steps, i1 = min(i0 + s.steps, s.iters);
  const bool norm = s.w != nullptr;
  Weights<TP, V, NU> w;
  w.load(s.w, u);
  float acc[NU][2 * V];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) acc[i][e] = 0.0f;
  const Pair own(a, lane);
  int64_t t = (int64_t)(block % s.gx) * 4 + wave;
  int pos = own.pos(a, t);
  for (; t < a.T; t += (int64_t)s.gx * 4) {
    Raw<TA, V, NU> nx, nd;
    auto fetch = [&](int it) {
      const int head = it * per + lane / a.lanes;
      const bool in = head < s.h;
      nx.load(s.v, t * s.v_st + head * s.v_sh, u, in && norm);
      nd.load(s.dv, t * s.dv_st + head * s.dv_sh, u, in);
    };
    fetch(i0);
    fill_turns(a, t, table, lane, own, pos);
    pos = own.pos(a, t + (int64_t)s.gx * 4);
    float2 cs[NU][V];
    lane_turns<V, NU>(a, table, u, cs);
    for (int it = i0; it < i1; ++it) {
      const Raw<TA, V, NU> x = nx, dd = nd;
      if (it + 1 < i1) fetch(it + 1);
      const int head = it * per + lane / a.lanes;
      const bool in = head < s.h;
      float g[NU][2 * V];
#pragma unroll
      for (int i = 0; i < NU; ++i) {
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) g[i][e] = dd.at(i, e);
        if (u[i].pair >= 0) rotate<V, PAIRS>(g[i], cs[i], -1.0f);
      }
      if (norm) {
        float q = 0.0f, m = 0.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            q = fmaf(x.at(i, e), x.at(i, e), q);
            m = fmaf(g[i][e] * (a.offset + w.at(i, e)), x.at(i, e), m);
          }
        const float r = rsqrtf(fmaf(lanes_sum(q, a.lanes), inv_d, a.eps));
        m = lanes_sum(m, a.lanes) * inv_d * r * r;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            const float n = x.at(i, e) * r, ge = g[i][e];
            // lanes without a head hold zeros, whose row factors may be infinite
            acc[i][e] += in && u[i].ok ? ge * n : 0.0f;
            g[i][e] = r * fmaf(-x.at(i, e), m, ge * (a.offset + w.at(i, e)));
          }
      }
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (in && u[i].ok) {
          const int64_t at = t * s.out_st + head * s.out_sh;
          Vec<TA, V>::store(s.out, at + u[i].first, g[i]);
          Vec<TA, V>::store(s.out, at + u[i].second, g[i] + V);
        }
    }
  }
  if (s.part == nullptr) return;  // uniform
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
      float x = acc[i][e];  // over the heads that the wavefront holds side by side
      for (int b = a.lanes; b < 64; b <<= 1) x += __shfl_xor(x, b);
      if (lane < a.lanes && u[i].ok) sums[wave][(e < V ? u[i].first : u[i].second) + e % V] = x;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += 256) s.part[(int64_t)block * a.d + c] = ((sums[0][c] + sums[1][c]) + sums[2][c]) + sums[3][c];
}

// dst[c] = sum over the nb slices of part [nb, d]: 64 runs of every 64th slice in
// ascending order, their sums added in a fixed order.  nb = 0 writes zeros.
struct RopeGradArgs {
  const float* part[2];
  void* dst[2];
  int32_t nb[2];
  int32_t d;
};
template <typename TP>
__global__ __launch_bounds__(1024) void rope_grad_kernel(const RopeGradArgs a) {
  constexpr int AHEAD = 16;  // slices a thread loads together (past the last one it is read again)
  __shared__ float run[16][16];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4, nb = a.nb[blockIdx.y];
  const float* p = a.part[blockIdx.y];
  float s = 0.0f;
  if (c < a.d)
    for (int b0 = k; b0 < nb; b0 += 64 * AHEAD) {
      float x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) x[i] = p[(int64_t)min(b0 + 64 * i, nb - 1) * a.d + c];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s = b0 + 64 * i < nb ? s + x[i] : s;
    }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if ((threadIdx.x & 63) < 16) run[threadIdx.x >> 6][threadIdx.x & 15] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < a.d) {
    s = run[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 16; ++i) s += run[i][threadIdx.x];
    store1(static_cast<TP*>(a.dst[blockIdx.y]) + c, s);
  }
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------

// Pairs a lane owns: 8 in bf16, 4 in fp32 where every access can be 16 bytes, else 1.
int lane_pairs(const lora_rope_desc* d, bool vec) { return d->dtype != LORA_F32 ? 8 : vec ? 4 : 1; }

// Lanes of a head, and how many steps the heads of a token take.
void set_lanes(RopeArgs& a, int V) {
  const int units = a.d / (2 * V);
  a.lanes = 1;
  while (a.lanes < 64 && a.lanes < units) a.lanes *= 2;
  for (HeadSet& s : a.set) s.iters = (int)cdiv(s.h, 64 / a.lanes);
}
// Blocks for n groups of tokens, at most `most`: as many groups for each.
int even_blocks(int64_t n, int64_t most) { return (int)cdiv(n, cdiv(n, most)); }
// Forward: blocks of four tokens along x, chunks of a token's steps along y
// while the tokens alone do not fill the chip.
dim3 forward_grid(RopeArgs& a) {
  const int64_t all = a.set[0].iters + a.set[1].iters;
  a.steps = (int32_t)cdiv(all, std::min(all, cdiv(8192, a.T)));
  return dim3((unsigned)even_blocks(cdiv(a.T, 4), kFwdBlocks), (unsigned)cdiv(all, a.steps));
}
// Backward with a norm: q's blocks, then k's, each with a share of the
// kBwdBlocks slices as it has of the work: a token's steps, and its angles,
// which take about as long as one and a half.
dim3 backward_grid(RopeArgs& a) {
  int64_t all = 0, steps = a.set[0].iters + a.set[1].iters;
  for (const HeadSet& s : a.set) all += s.h ? 2 * s.iters + 3 : 0;
  int block0 = 0;
  for (HeadSet& s : a.set) {
    s.block0 = block0;
    if (s.h == 0) continue;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kBwdBlocks * (2 * (int64_t)s.iters + 3) / all, kBwdBlocks - 1));
    const int64_t want = std::min(std::min<int64_t>(s.iters, most), cdiv(8192 * (int64_t)s.iters, a.T * steps));
    s.steps = (int32_t)cdiv(s.iters, want);
    const int64_t chunks = cdiv(s.iters, s.steps);
    s.gx = even_blocks(cdiv(a.T, 4), std::max<int64_t>(1, most / chunks));
    block0 += s.gx * (int)chunks;
  }
  return dim3((unsigned)block0);
}
int set_blocks(const HeadSet& s) { return s.h ? s.gx * (int)cdiv(s.iters, s.steps) : 0; }

template <typename TA, typename TP, int V, int NU, bool PAIRS>
hipError_t launch_one(const RopeArgs& a, dim3 grid, int what, hipStream_t st) {
  if (what == 2) hipLaunchKernelGGL((rope_bwd_kernel<TA, TP, V, NU, PAIRS>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((rope_fwd_kernel<TA, TP, V, NU, PAIRS>), grid, dim3(256), 0, st, a, what == 0 ? 1.0f : -1.0f);
  return hipGetLastError();
}
// what: 0 forward, 1 the inverse rotation alone, 2 backward with a norm
hipError_t launch_rope(const RopeArgs& a, dim3 grid, int32_t dtype, int V, bool pairs, int what, hipStream_t st) {
  if (dtype == LORA_BF16)
    return pairs ? launch_one<uint16_t, uint16_t, 8, 1, true>(a, grid, what, st) : launch_one<uint16_t, uint16_t, 8, 1, false>(a, grid, what, st);
  if (dtype == LORA_BF16_F32LORA)
    return pairs ? launch_one<uint16_t, float, 8, 1, true>(a, grid, what, st) : launch_one<uint16_t, float, 8, 1, false>(a, grid, what, st);
  if (V == 4) return pairs ? launch_one<float, float, 4, 1, true>(a, grid, what, st) : launch_one<float, float, 4, 1, false>(a, grid, what, st);
  // one pair a lane: up to 64, 128 or 256 pairs a head
  const int nu = a.d <= 128 ? 1 : a.d <= 256 ? 2 : 4;
  if (nu == 1) return pairs ? launch_one<float, float, 1, 1, true>(a, grid, what, st) : launch_one<float, float, 1, 1, false>(a, grid, what, st);
  if (nu == 2) return pairs ? launch_one<float, float, 1, 2, true>(a, grid, what, st) : launch_one<float, float, 1, 2, false>(a, grid, what, st);
  return pairs ? launch_one<float, float, 1, 4, true>(a, grid, what, st) : launch_one<float, float, 1, 4, false>(a, grid, what, st);
}

// ---------------------------------------------------------------------------
// Checks of the entry points.
// ---------------------------------------------------------------------------
struct RopeSizes {
  int64_t es, ps;
  size_t align;
  int64_t unit;  // bf16: strides and widths are multiples of this
};

lora_status check_desc(const lora_rope_desc* d, RopeSizes& z) {
  CHECK(d != nullptr, LORA_EINVAL, "desc is NULL");
  CHECK(d->dtype == LORA_F32 || d->dtype == LORA_BF16 || d->dtype == LORA_BF16_F32LORA, LORA_EDTYPE, "unknown dtype %d",
        d->dtype);
  CHECK(d->interleaved == 0 || d->interleaved == 1, LORA_EINVAL, "interleaved = %d is not 0 or 1", d->interleaved);
  CHECK(d->unit_offset == 0 || d->unit_offset == 1, LORA_EINVAL, "unit_offset = %d is not 0 or 1", d->unit_offset);
  CHECK(d->reserved == 0, LORA_EINVAL, "reserved must be 0");
  CHECK(std::isfinite(d->eps) && d->eps >= 0.0f, LORA_EINVAL, "eps must be finite and not negative");
  CHECK(std::isfinite(d->scale), LORA_EINVAL, "scale is not finite");
  CHECK(d->T >= 0 && d->T < ((int64_t)1 << 40), LORA_ESHAPE, "T = %lld is negative or too large", (long long)d->T);
  CHECK(d->hq > 0 && d->hq <= 65536 && d->hk >= 0 && d->hk <= 65536, LORA_ESHAPE, "hq = %lld must be in [1, 65536], hk = %lld in [0, 65536]",
        (long long)d->hq, (long long)d->hk);
  const int64_t unit = d->dtype == LORA_F32 ? 2 : 16;
  CHECK(d->d > 0 && d->d <= kMaxD && d->d % unit == 0, LORA_ESHAPE, "d = %lld must be a multiple of %d in [1, %d]",
        (long long)d->d, (int)unit, kMaxD);
  CHECK(d->rot >= 0 && d->rot <= d->d && d->rot % unit == 0, LORA_ESHAPE, "rot = %lld must be a multiple of %d in [0, d]",
        (long long)d->rot, (int)unit);
  CHECK(d->axes >= 1 && d->axes <= 16, LORA_ESHAPE, "axes = %d must be in [1, 16]", d->axes);
  z.es = d->dtype == LORA_F32 ? 4 : 2;
  z.ps = d->dtype == LORA_BF16 ? 2 : 4;
  z.align = d->dtype == LORA_F32 ? 4 : 16;
  z.unit = d->dtype == LORA_F32 ? 1 : 8;
  return LORA_OK;
}

// A tensor of a call: rows heads [T, h, d] with strides, or plain bytes.
struct Ext {
  const void* p;
  const char* name;
  int64_t T, h, st, sh, d;  // in bytes; plain: T = h = 1
  int64_t bytes() const { return T > 0 && h > 0 ? (T - 1) * st + (h - 1) * sh + d : 0; }
};

Ext plain(const void* p, size_t bytes, const char* name) { return {p, name, 1, 1, 0, 0, p ? (int64_t)bytes : 0}; }

// No two of a tensor's rows share memory.
bool rows_apart(const Ext& e) {
  if (e.T > 1 && e.h > 1) return (e.sh >= e.d && e.st >= (e.h - 1) * e.sh + e.d) || (e.st >= e.d && e.sh >= (e.T - 1) * e.st + e.d);
  return (e.T <= 1 || e.st >= e.d) && (e.h <= 1 || e.sh >= e.d);
}

// Parts of one buffer (q, k and v of a fused projection) interleave: with
// one period S in both, each tensor's part of a period must end before the
// other's begins.
bool period_apart(const Ext& a, const Ext& b, int64_t Sa, int64_t span_a, int64_t Sb, int64_t span_b) {
  if (Sa != Sb || span_a > Sa || span_b > Sa) return false;
  int64_t delta = (int64_t)(((intptr_t)b.p - (intptr_t)a.p) % Sa);
  if (delta < 0) delta += Sa;
  return delta >= span_a && delta + span_b <= Sa;
}
// Rows that lie between each other's along both the tokens and the heads (q, k and v head by head,
// [T, h, 3, d]).  With the same strides in both, rows (t, i) of a and (t', i') of b begin
// a - b + (t - t') st + (i - i') sh apart, and meet where that is in (-a.d, b.d): for every i - i' the
// t - t' that do so are a range.  A stride of a single token or head is the other's.
bool lattice_apart(const Ext& a, const Ext& b) {
  if ((a.T > 1 && b.T > 1 && a.st != b.st) || (a.h > 1 && b.h > 1 && a.sh != b.sh)) return false;
  const int64_t st = a.T > 1 ? a.st : b.T > 1 ? b.st : 0, sh = a.h > 1 ? a.sh : b.h > 1 ? b.sh : 0;
  const int64_t base = (int64_t)((intptr_t)a.p - (intptr_t)b.p);
  for (int64_t i = 1 - b.h; i < a.h; ++i) {
    const int64_t lo = -a.d - (base + i * sh), hi = b.d - (base + i * sh);  // of (t - t') st, both ends out
    if (st == 0) {
      if (lo < 0 && hi > 0) return false;
      continue;
    }
    // floor(lo / st) + 1 .. ceil(hi / st) - 1
    const int64_t first = (lo >= 0 ? lo / st : -((st - 1 - lo) / st)) + 1, last = (hi > 0 ? (hi - 1) / st : -((st - hi) / st));
    if (std::max(first, 1 - b.T) <= std::min(last, a.T - 1)) return false;
  }
  return true;
}
bool apart(const Ext& a, const Ext& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes() == 0 || b.bytes() == 0) return true;
  if (!overlaps(a.p, (size_t)a.bytes(), b.p, (size_t)b.bytes())) return true;
  return (a.st > 0 && period_apart(a, b, a.st, (a.h - 1) * a.sh + a.d, b.st, (b.h - 1) * b.sh + b.d)) ||
         (a.sh > 0 && period_apart(a, b, a.sh, (a.T - 1) * a.st + a.d, b.sh, (b.T - 1) * b.st + b.d)) || lattice_apart(a, b);
}
bool same(const Ext& a, const Ext& b) {
  return a.p == b.p && a.T == b.T && a.h == b.h && a.d == b.d && (a.T <= 1 || a.st == b.st) && (a.h <= 1 || a.sh == b.sh);
}

lora_status check_heads(const lora_rope_desc* d, const RopeSizes& z, const lora_heads* x, int64_t h, const char* name,
                        bool out, Ext& e) {
  e = Ext{nullptr, name, 0, 0, 0, 0, 0};
  if (h == 0 || d->T == 0) return LORA_OK;
  CHECK(x != nullptr && x->p != nullptr, LORA_EINVAL, "%s is NULL", name);
  CHECK(aligned(x->p, z.align), LORA_EALIGN, "%s is not %d-byte aligned", name, (int)z.align);
  // the stride of a single token or head means nothing
  const int64_t st = d->T > 1 ? x->stride_t : 0, sh = h > 1 ? x->stride_h : 0;
  CHECK(st >= 0 && sh >= 0 && st % z.unit == 0 && sh % z.unit == 0, LORA_EALIGN,
        "%s: strides %lld and %lld must not be negative and multiples of %d", name, (long long)st, (long long)sh, (int)z.unit);
  const int64_t most = (int64_t)1 << 45;  // elements, so that no offset leaves 64 bits
  CHECK(st <= most / d->T && sh <= most / h, LORA_ESHAPE, "%s is too large", name);
  e = Ext{x->p, name, d->T, h, st * z.es, sh * z.es, d->d * z.es};
  CHECK(!out || rows_apart(e), LORA_EUNSUPPORTED, "%s: rows of an output overlap", name);
  return LORA_OK;
}

// An output may be exactly an input of the same heads; nothing else overlaps.
// kin[i]: which of q (0) and k (1) tensor i belongs to, -1 neither.
lora_status check_overlap(const Ext* in, const int* in_kin, int ni, const Ext* out, const int* out_kin, int no) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      CHECK((in_kin[j] >= 0 && in_kin[j] == out_kin[i] && same(out[i], in[j])) || apart(out[i], in[j]), LORA_EUNSUPPORTED,
            "%s overlaps %s", out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      CHECK(apart(out[i], out[j]), LORA_EUNSUPPORTED, "%s overlaps %s", out[i].name, out[j].name);
  }
  return LORA_OK;
}

bool vec_heads(const Ext& e) {
  return e.p == nullptr || (aligned(e.p, 16) && e.st % 16 == 0 && e.sh % 16 == 0);
}

lora_status check_common(const lora_rope_desc* d, const RopeSizes& z, const int32_t* pos, const float* freq,
                         const int32_t* axis, const void* w_q, const void* w_k) {
  CHECK(d->hk > 0 || w_k == nullptr, LORA_EINVAL, "w_k without heads of k");
  CHECK(d->rot == 0 || (pos != nullptr && freq != nullptr), LORA_EINVAL, "pos or inv_freq is NULL");
  CHECK(d->axes == 1 || axis != nullptr || d->rot == 0, LORA_EINVAL, "positions of several axes need axis");
  CHECK(aligned(pos, 4) && aligned(freq, 4) && aligned(axis, 4), LORA_EALIGN, "pos, inv_freq or axis is not 4-byte aligned");
  CHECK(aligned(w_q, z.align) && aligned(w_k, z.align), LORA_EALIGN, "w_q or w_k is not %d-byte aligned", (int)z.align);
  const int64_t most = (int64_t)1 << 45;
  CHECK(d->pos_stride_t >= 0 && d->pos_stride_a >= 0 && (d->T <= 1 || d->pos_stride_t <= most / d->T) &&
            d->pos_stride_a <= most / d->axes, LORA_ESHAPE, "strides %lld and %lld of pos", (long long)d->pos_stride_t,
        (long long)d->pos_stride_a);
  return LORA_OK;
}

size_t pos_bytes(const lora_rope_desc* d) {
  return (size_t)((d->T - 1) * d->pos_stride_t + (d->axes - 1) * d->pos_stride_a + 1) * 4;
}

RopeArgs base_args(const lora_rope_desc* d, const int32_t* pos, const float* freq, const int32_t* axis, const void* w_q,
                   const void* w_k) {
  RopeArgs a{};
  a.T = d->T;
  a.pos = pos;
  a.axis = axis;
  a.freq = freq;
  a.pos_st = d->pos_stride_t;
  a.pos_sa = d->pos_stride_a;
  a.d = (int32_t)d->d;
  a.rot = (int32_t)d->rot;
  a.axes = d->axes;
  a.scale = d->scale;
  a.eps = d->eps;
  a.offset = d->unit_offset ? 1.0f : 0.0f;
  a.set[0].h = (int32_t)d->hq;
  a.set[1].h = (int32_t)d->hk;
  a.set[0].w = w_q;
  a.set[1].w = w_k;
  return a;
}

// Slices of both weights' gradients; an upper bound over the ways to split the work.
size_t bwd_bytes(const lora_rope_desc* d) { return d->T == 0 ? 0 : (size_t)kBwdBlocks * (size_t)d->d * 4; }

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status lora_qk_norm_rope_workspace_size(const lora_rope_desc* d, size_t* bwd) {
  RopeSizes z;
  TRY(check_desc(d, z));
  if (bwd) *bwd = bwd_bytes(d);
  return LORA_OK;
}

lora_status lora_qk_norm_rope_fwd(const lora_rope_desc* d, const lora_heads* Q, const lora_heads* K, const int32_t* pos,
                                  const float* inv_freq, const int32_t* axis, const void* w_q, const void* w_k,
                                  const lora_heads* Q_out, const lora_heads* K_out, void* stream) {
  RopeSizes z;
  TRY(check_desc(d, z));
  if (d->T == 0) return LORA_OK;
  TRY(check_common(d, z, pos, inv_freq, axis, w_q, w_k));
  const size_t wb = (size_t)(d->d * z.ps), half = (size_t)d->rot / 2 * 4;
  Ext in[7], out[2];
  TRY(check_heads(d, z, Q, d->hq, "Q", false, in[0]));
  TRY(check_heads(d, z, K, d->hk, "K", false, in[1]));
  TRY(check_heads(d, z, Q_out, d->hq, "Q_out", true, out[0]));
  TRY(check_heads(d, z, K_out, d->hk, "K_out", true, out[1]));
  in[2] = plain(pos, pos_bytes(d), "pos");
  in[3] = plain(inv_freq, half, "inv_freq");
  in[4] = plain(axis, half, "axis");
  in[5] = plain(w_q, wb, "w_q");
  in[6] = plain(w_k, wb, "w_k");
  const int in_kin[] = {0, 1, -1, -1, -1, -1, -1}, out_kin[] = {0, 1};
  TRY(check_overlap(in, in_kin, 7, out, out_kin, 2));
  RopeArgs a = base_args(d, pos, inv_freq, axis, w_q, w_k);
  bool vec = d->d % 8 == 0 && d->rot % 8 == 0 && aligned(w_q, 16) && aligned(w_k, 16);
  for (int k = 0; k < 2; ++k) {
    if (a.set[k].h == 0) continue;
    a.set[k].v = in[k].p;
    a.set[k].v_st = in[k].st / z.es;
    a.set[k].v_sh = in[k].sh / z.es;
    a.set[k].out = const_cast<void*>(out[k].p);
    a.set[k].out_st = out[k].st / z.es;
    a.set[k].out_sh = out[k].sh / z.es;
    vec = vec && vec_heads(in[k]) && vec_heads(out[k]);
  }
  const int V = lane_pairs(d, vec);
  set_lanes(a, V);
  const dim3 grid = forward_grid(a);
  hipStream_t st = static_cast<hipStream_t>(stream);
  LAUNCHN("qk_norm_rope_fwd", st, launch_rope(a, grid, d->dtype, V, d->interleaved != 0, 0, st));
  return LORA_OK;
}

lora_status lora_qk_norm_rope_bwd(const lora_rope_desc* d, const lora_heads* dQ_out, const lora_heads* dK_out,
                                  const lora_heads* Q, const lora_heads* K, const int32_t* pos, const float* inv_freq,
                                  const int32_t* axis, const void* w_q, const void* w_k, const lora_heads* dQ,
                                  const lora_heads* dK, void* dw_q, void* dw_k, void* ws, size_t ws_bytes, void* stream) {
  RopeSizes z;
  TRY(check_desc(d, z));
  CHECK((w_q != nullptr) == (dw_q != nullptr) && (w_k != nullptr) == (dw_k != nullptr), LORA_EINVAL,
        "a weight and its gradient are given together");
  const bool rows = d->T > 0, norm = w_q != nullptr || w_k != nullptr;
  CHECK(aligned(dw_q, z.ps) && aligned(dw_k, z.ps), LORA_EALIGN, "dw_q or dw_k is not aligned to its type");
  if (rows) TRY(check_common(d, z, pos, inv_freq, axis, w_q, w_k));
  else CHECK(d->hk > 0 || w_k == nullptr, LORA_EINVAL, "w_k without heads of k");
  const size_t need = norm ? bwd_bytes(d) : 0;
  TRY(check_ws(ws, ws_bytes, need));
  const size_t wb = (size_t)(d->d * z.ps), half = (size_t)d->rot / 2 * 4;
  Ext in[9], out[5];
  TRY(check_heads(d, z, dQ_out, d->hq, "dQ_out", false, in[0]));
  TRY(check_heads(d, z, dK_out, d->hk, "dK_out", false, in[1]));
  TRY(check_heads(d, z, Q, w_q ? d->hq : 0, "Q", false, in[2]));
  TRY(check_heads(d, z, K, w_k ? d->hk : 0, "K", false, in[3]));
  TRY(check_heads(d, z, dQ, d->hq, "dQ", true, out[0]));
  TRY(check_heads(d, z, dK, d->hk, "dK", true, out[1]));
  in[4] = plain(pos, rows ? pos_bytes(d) : 0, "pos");
  in[5] = plain(inv_freq, half, "inv_freq");
  in[6] = plain(axis, half, "axis");
  in[7] = plain(w_q, wb, "w_q");
  in[8] = plain(w_k, wb, "w_k");
  out[2] = plain(dw_q, wb, "dw_q");
  out[3] = plain(dw_k, wb, "dw_k");
  out[4] = plain(need ? ws : nullptr, need, "ws");
  const int in_kin[] = {0, 1, 0, 1, -1, -1, -1, -1, -1}, out_kin[] = {0, 1, -1, -1, -1};
  TRY(check_overlap(in, in_kin, 9, out, out_kin, 5));
  hipStream_t st = static_cast<hipStream_t>(stream);
  RopeGradArgs r{};
  r.d = (int32_t)d->d;
  int n = 0;
  if (rows) {
    RopeArgs a = base_args(d, pos, inv_freq, axis, w_q, w_k);
    bool vec = d->d % 8 == 0 && d->rot % 8 == 0 && aligned(w_q, 16) && aligned(w_k, 16);
    for (int k = 0; k < 2; ++k) {
      if (a.set[k].h == 0) continue;
      HeadSet& s = a.set[k];
      const Ext& v = norm ? in[2 + k] : in[k];  // the rotation alone runs the forward kernel on the gradient
      s.v = v.p;
      s.v_st = v.st / z.es;
      s.v_sh = v.sh / z.es;
      s.dv = in[k].p;
      s.dv_st = in[k].st / z.es;
      s.dv_sh = in[k].sh / z.es;
      s.out = const_cast<void*>(out[k].p);
      s.out_st = out[k].st / z.es;
      s.out_sh = out[k].sh / z.es;
      vec = vec && vec_heads(in[k]) && vec_heads(in[2 + k]) && vec_heads(out[k]);
    }
    const int V = lane_pairs(d, vec);
    set_lanes(a, V);
    const dim3 grid = norm ? backward_grid(a) : forward_grid(a);
    float* part = static_cast<float*>(ws);
    if (w_q) a.set[0].part = part;
    if (w_k) a.set[1].part = part + (w_q ? (size_t)set_blocks(a.set[0]) * d->d : 0);
    void* const dst[2] = {dw_q, dw_k};
    for (int k = 0; k < 2; ++k) {
      if (dst[k] == nullptr) continue;
      r.part[n] = a.set[k].part;
      r.nb[n] = set_blocks(a.set[k]);
      r.dst[n++] = dst[k];
    }
    if (norm) LAUNCHN("qk_norm_rope_bwd", st, launch_rope(a, grid, d->dtype, V, d->interleaved != 0, 2, st));
    else LAUNCHN("qk_norm_rope_inv", st, launch_rope(a, grid, d->dtype, V, d->interleaved != 0, 1, st));
  } else {
    if (w_q) r.dst[n++] = dw_q;
    if (w_k) r.dst[n++] = dw_k;
  }
  if (n > 0) {
    const dim3 grid((unsigned)cdiv(d->d, 16), (unsigned)n);
    TraceScope ts("qk_norm_rope_grad", st);
    if (z.ps == 2) hipLaunchKernelGGL(rope_grad_kernel<uint16_t>, grid, dim3(1024), 0, st, r);
    else hipLaunchKernelGGL(rope_grad_kernel<float>, grid, dim3(1024), 0, st, r);
    LAUNCH(hipGetLastError());
  }
  return LORA_OK;
}

}  // extern "C"
