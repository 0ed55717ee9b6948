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
  int32_t nshrink, nz;  // few rows: blocks of the shrink, and how many share the adapters of 16 rows
  uint16_t* u;          // scaled U in two bf16 parts, as GemmArgs::mt_u (many rows)
  MultiTile* plan;      // adapters of every 256-row tile (many rows)
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
// a ring of LDS slots.  Wavefront (h, k) of four takes column half h and
// K half k of every stage (no operand is read from LDS more often than it
// must for 64 x 16 MT sums a wavefront), and the two K halves meet at the
// end.  The weight is the MFMA's row operand, so a lane ends with four
// consecutive columns of a row.
// LDS layouts: W rows of 256 bytes, 16-byte chunk c of row k at c ^ 4 (k & 3),
// read with the transposing LDS read; X rows of 128 bytes, chunk c of row m at
// c ^ (m & 7).
// Measured, U beside it: one row of 4096 x 4096 8.2 us (4.1 TB/s over W), 67
// rows of 4096 x 14336 27 us (117 MB of W: 4.3 TB/s, a large copy 4.85).
// ---------------------------------------------------------------------------
template <int MT>
struct BaseCfg {
  static constexpr int WB = 64 * 256, XB = MT * 16 * 128, SB = WB + XB;
  // two blocks a CU while three stages fit half of its LDS, else one with five
  static constexpr int PER_CU = 3 * SB <= 81920 ? 2 : 1;
  static constexpr int NST = PER_CU == 2 ? (4 * SB <= 81920 ? 4 : 3) : 5;
  static constexpr int SMEM = NST * SB > 2 * MT * 4096 ? NST * SB : 2 * MT * 4096;
  static_assert(SMEM * PER_CU <= 163840, "LDS of a CU");
};

template <int MT>
__device__ __forceinline__ void base_block(const MultiArgs& a, char* ring, int bid) {
  using C = BaseCfg<MT>;
  lds_char* const lds = (lds_char*)ring;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = w & 1, kh = w >> 1;
  // blocks b, b + 8, ... run on one XCD: the row tiles of one part of W follow each other there
  const int j = bid >> 3, unit = (j / a.ntm) * 8 + (bid & 7), tm = j % a.ntm;
  if (unit >= a.ntn * a.ks) return;
  const int tn = unit % a.ntn, part = unit / a.ntn;
  const int steps = (int)(a.K / 64);
  const int s0 = (int)((int64_t)part * steps / a.ks), s1 = (int)((int64_t)(part + 1) * steps / a.ks);
  const int64_t n0 = (int64_t)tn * 128;
  const uint32_t ldw2 = (uint32_t)(a.N * 2), ldx2 = (uint32_t)(a.K * 2);
  const char* wp = static_cast<const char*>(a.W) + ((int64_t)s0 * 64 * a.N + n0) * 2;
  int64_t wn = ((a.K - (int64_t)s0 * 64) * a.N - n0) * 2;
  const int64_t m0 = (int64_t)tm * (16 * MT);
  const char* xp = static_cast<const char*>(a.X) + (m0 * a.K + (int64_t)s0 * 64) * 2;
  int64_t xn = ((a.T - m0) * a.K - (int64_t)s0 * 64) * 2;
  const uint32_t woff = (uint32_t)(lane >> 4) * ldw2 + (uint32_t)(((lane & 15) ^ (4 * ((lane >> 4) & 3))) * 16);
  // X block b of 1 KB holds rows 8 b .. 8 b + 7; wavefront w loads blocks w, w + 4, ... of 2 MT
  constexpr int XP = (2 * MT + 3) / 4;
  uint32_t xoff[XP];  // rows past T read zero
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int row = 8 * (w + 4 * i) + (lane >> 3);
    xoff[i] = m0 + row < a.T ? (uint32_t)row * ldx2 + (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16) : 0x80000000u;
  }
  auto issue = [&](int slot) {
    const uint32_t base = lds_addr(lds) + slot * C::SB;
    const i32x4 rw = rsrc_words(wp, wn), rx = rsrc_words(xp, xn);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma16(rw, woff, base + (4 * w + i) * 1024, (uint32_t)(4 * (4 * w + i)) * ldw2);
#pragma unroll
    for (int i = 0; i < XP; ++i)
      if (w + 4 * i < 2 * MT) dma16(rx, xoff[i], base + C::WB + (w + 4 * i) * 1024);
    wp += (int64_t)64 * a.N * 2;
    wn -= (int64_t)64 * a.N * 2;
    xp += 128;
    xn -= 128;
  };
  // an odd MT leaves the last X load to wavefronts 0 and 1
  const bool fewer = (2 * MT) % 4 != 0 && w >= 2;
  const int g = lane >> 4, c = lane & 15, jj = c >> 2;
  f32x4 acc[4][MT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0, 0, 0, 0};
  // fragment offsets of 16-column blocks 2 i and 2 i + 1 (bit 1 of the chunk index is clear in the
  // first and in the swizzle, so the second is 32 bytes on)
  int wo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = 64 * h + 32 * i + 4 * (lane & 3);
    wo[i] = (32 * kh + 8 * g + jj) * 256 + (((col >> 3) ^ (4 * jj)) * 16) + (lane & 1) * 8;
  }
  const int xo = c * 128 + (((4 * kh + g) ^ (c & 7)) * 16);
  const int n = s1 - s0;
  for (int s = 0; s < C::NST - 1 && s < n; ++s) issue(s);
  int slot = 0;
  for (int s = 0; s < n; ++s) {
    const int after = n - 1 - s < C::NST - 2 ? n - 1 - s : C::NST - 2;
    if (fewer) wait_stages<4 + XP - 1, C::NST - 2>(after);
    else wait_stages<4 + XP, C::NST - 2>(after);
    __syncthreads();  // stage s is in for every wavefront, and stage s - 1 is no longer read
    if (s + C::NST - 1 < n) issue(slot == 0 ? C::NST - 1 : slot - 1);
    const lds_char* ws = lds + slot * C::SB;
    const lds_char* xs = ws + C::WB;
    bf16x8 fw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fw[i] = lds_read_tr8(ws + wo[i >> 1] + 32 * (i & 1), 4 * 256);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bf16x8 fx = __builtin_bit_cast(bf16x8, lds_read16(xs + xo + m * 2048));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[i], fx, acc[i][m], 0, 0, 0);
    }
    slot = slot + 1 == C::NST ? 0 : slot + 1;
  }
  __syncthreads();  // the ring becomes the exchange of the K halves
  f32x4* ex = reinterpret_cast<f32x4*>(ring) + h * (4 * MT * 64);
  if (kh == 1)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) ex[(m * 4 + i) * 64 + lane] = acc[i][m];
  __syncthreads();
  if (kh == 0) {
    float* out = a.part + (int64_t)part * a.T * a.N;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t t = m0 + 16 * m + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t col = n0 + 64 * h + 16 * i + 4 * g;
        const f32x4 v = acc[i][m] + ex[(m * 4 + i) * 64 + lane];
        if (t < a.T && col < a.N) *reinterpret_cast<f32x4*>(out + t * a.N + col) = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// U = X A_i for few rows (bf16): fp32 sums over K ranges of 1024.  A block has
// 16 rows; its four wavefronts take 256 K each, hold X of them in registers,
// and walk the distinct adapters of the rows, each multiplied against all of
// them (the MFMA computes 16 rows at a time anyway) and kept where it is the
// row's own; gridDim.z blocks share the walk, so that as a rule a block meets
// one adapter.  A_i [K, r] is read as it lies: lane 16 q + c takes columns
// NJ c .. NJ c + NJ - 1 of 8 consecutive K rows, which after a transpose in
// registers are the operands of NJ tiles (tile t: rank index NJ c + t).
// ---------------------------------------------------------------------------
constexpr int kShrinkK = 256;  // per wavefront

template <int NJ>
struct AFrags {
  uint32_t x[8][NJ];
  // rows row0 .. row0 + 7 of A_i; rows past the end and columns past the rank read zero
  __device__ __forceinline__ void load(brsrc ra, uint32_t row0, int r, int c) {
    const uint32_t ld = (uint32_t)r * 2;
    const bool in = NJ * c < r;
    const uint32_t off = row0 * ld + (uint32_t)(NJ * c) * 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t o = in ? off + (uint32_t)e * ld : 0x80000000u;
      if constexpr (NJ == 4) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(ra, o, 0, 0);
        x[e][0] = v[0];
        x[e][1] = v[1];
      } else if constexpr (NJ == 2) {
        x[e][0] = __builtin_amdgcn_raw_buffer_load_b32(ra, o, 0, 0);
      } else {
#pragma unroll
        for (int t = 0; t < NJ; ++t) x[e][t] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ra, o + 2 * t, 0, 0);
      }
    }
  }
  // operand of tile t: element e of the lane is row row0 + e
  __device__ __forceinline__ bf16x8 frag(int t) const {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (NJ == 1 || NJ == 3) v[e] = x[2 * e][t] | (x[2 * e + 1][t] << 16);
      else v[e] = __builtin_amdgcn_perm(x[2 * e + 1][t >> 1], x[2 * e][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
    }
    return __builtin_bit_cast(bf16x8, v);
  }
};

template <int NJ>
__device__ __forceinline__ void shrink_few_block(const MultiArgs& a, char* lds, int bx, int kc, int bz, int nz) {
  constexpr int STEPS = kShrinkK / 32;                // K steps of a wavefront
  constexpr int FLY = NJ == 3 ? 2 : NJ == 4 ? 4 : 8;  // of A_i, loaded at a time
  f32x4(*red)[NJ][64] = reinterpret_cast<f32x4(*)[NJ][64]>(lds);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int64_t k0 = (int64_t)(4 * kc + w) * kShrinkK;
  const int64_t klen = a.K - k0 < kShrinkK ? a.K - k0 : kShrinkK;  // multiple of 64, may be <= 0
  const int64_t t0 = (int64_t)bx * 16;
  const int my = lane < 16 ? row_id(a, t0 + lane) : -1;
  uint64_t todo = __ballot(my >= 0);
  if (todo == 0) return;  // uniform over the block
  const int rid = __shfl(my, c);  // adapter of the lane's MFMA row
  const brsrc rx = make_rsrc(static_cast<const char*>(a.X) + (t0 * a.K + k0) * 2, ((a.T - t0) * a.K - k0) * 2);
  u32x4 fx[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)  // rows past T and K past the range read zero
    fx[s] = buf_load16(rx, t0 + c < a.T && 32 * s < klen ? (uint32_t)((c * a.K + 32 * s + 8 * g) * 2) : 0x80000000u);
  for (int turn = 0; todo != 0; turn = turn + 1 == nz ? 0 : turn + 1) {
    const int id = __builtin_amdgcn_readlane(my, __builtin_ctzll(todo));
    todo &= ~__ballot(my == id);
    if (turn != bz) continue;
    const char* Ai = static_cast<const char*>(a.A) + (int64_t)id * a.K * a.r * 2;
    const brsrc ra = make_rsrc(Ai + k0 * a.r * 2, klen * a.r * 2);
    f32x4 acc[NJ];
#pragma unroll
    for (int t = 0; t < NJ; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s0 = 0; s0 < STEPS; s0 += FLY) {
      AFrags<NJ> fa[FLY];
#pragma unroll
      for (int s = 0; s < FLY; ++s) fa[s].load(ra, (uint32_t)(32 * (s0 + s) + 8 * g), a.r, c);
#pragma unroll
      for (int s = 0; s < FLY; ++s)
#pragma unroll
        for (int t = 0; t < NJ; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s].frag(t), __builtin_bit_cast(bf16x8, fx[s0 + s]), acc[t], 0, 0, 0);
    }
    // the four quarters of the K range, in ascending order
    if (w > 0)
#pragma unroll
      for (int t = 0; t < NJ; ++t) red[w - 1][t][lane] = acc[t];
    __syncthreads();
    if (w == 0) {
      float* u = a.upart + ((int64_t)kc * a.T + t0 + c) * a.r;
#pragma unroll
      for (int t = 0; t < NJ; ++t) {
#pragma unroll
        for (int q = 0; q < 3; ++q) acc[t] += red[q][t][lane];
        if (rid == id)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int i = NJ * (4 * g + v) + t;  // rank index
            if (i < a.r) u[i] = acc[t][v];
          }
      }
    }
    __syncthreads();
  }
}

template <int NJ>
__global__ __launch_bounds__(256) void multi_shrink_few_kernel(const MultiArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[3 * NJ * 1024];
  const int b = blockIdx.x, kz = b % (a.kc * a.nz);
  shrink_few_block<NJ>(a, lds, b / (a.kc * a.nz), kz / a.nz, kz % a.nz, a.nz);
}

// X W, and where nshrink > 0 U beside it in the same launch, neither waiting
// for the other.
// The nshrink blocks that form U come last: the others, which take longer, are
// then spread evenly over the CUs (in front, the shrink left some CUs two of
// them and others none: 46 against 38 us at 67 rows of 4096 x 14336).
template <int MT>
__global__ __launch_bounds__(256, BaseCfg<MT>::PER_CU) void multi_few_kernel(const MultiArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[BaseCfg<MT>::SMEM];
  static_assert(BaseCfg<MT>::SMEM >= 3 * 4 * 1024, "the shrink's exchange");
  const int b = (int)blockIdx.x - ((int)gridDim.x - a.nshrink);
  if (b < 0) {
    base_block<MT>(a, lds, blockIdx.x);
    return;
  }
  const int bx = b / (a.kc * a.nz), kz = b % (a.kc * a.nz);
  switch ((a.r + 15) / 16) {
    case 1: shrink_few_block<1>(a, lds, bx, kz / a.nz, kz % a.nz, a.nz); break;
    case 2: shrink_few_block<2>(a, lds, bx, kz / a.nz, kz % a.nz, a.nz); break;
    case 3: shrink_few_block<3>(a, lds, bx, kz / a.nz, kz % a.nz, a.nz); break;
    default: shrink_few_block<4>(a, lds, bx, kz / a.nz, kz % a.nz, a.nz); break;
  }
  // the compiler joins both ways before the other's loop, where loads that it holds pending from here
  // would make it wait for all loads in every step
  wait_vmcnt<0>();
}

// ---------------------------------------------------------------------------
// U = X A_i for many rows (bf16): fp32 sums over K ranges of 256.  A block has
// a 256-row tile, whose rows it first puts in the order of their adapters, and
// a wavefront holds X of 64 of those, by 256 K, in registers: read once, all
// loads in flight together.  The block then walks the tile's adapters: the
// [256, r] slice of A_i, contiguous in memory, is copied to LDS one adapter
// ahead and read with the transposing read (tile t: rank index 16 t + c), and
// a wavefront multiplies it where its rows have that adapter.  The first
// block of a tile also lists its adapters for the GEMM.  (Blocks of 32 or 64
// rows, each sorting the tile for itself, took longer to sort than to read X,
// and A_i by loads into registers left each adapter a chain of latencies.)
// Measured: 8192 rows of 4096 at rank 16, 67 MB of X: 23 us (2.9 TB/s); 777
// rows of 14336 at rank 64 with 12 adapters: 18 to 22 us, the walk over the
// adapters, which two blocks share (20 to 24 when both read the rows of the other).
// ---------------------------------------------------------------------------
// Rows of a 256-row tile in the order of their adapters (rows without one
// last), by 256 threads: id_of and row_of hold the sorted ids and rows.
__device__ __forceinline__ void sort_tile(int id, int* keys, int* id_of, int* row_of) {
  const int i = threadIdx.x;
  const int key = id < 0 ? 0x7fffffff : id;
  keys[i] = key;
  __syncthreads();
  // keys before this one, equal keys in the order of their rows: smaller or equal among the
  // wavefronts before, smaller among those after, and by row within its own
  int rank = 0;
  const int4* k4 = reinterpret_cast<const int4*>(keys);
  const int w = __builtin_amdgcn_readfirstlane(i >> 6);
#pragma unroll 16
  for (int j = 0; j < 16 * w; ++j) {
    const int4 k = k4[j];
    rank += (int)(k.x <= key) + (int)(k.y <= key) + (int)(k.z <= key) + (int)(k.w <= key);
  }
#pragma unroll
  for (int j = 16 * w; j < 16 * w + 16; ++j) {
    const int4 k = k4[j];
    rank += (int)(k.x < key) + (int)(k.y < key) + (int)(k.z < key) + (int)(k.w < key);
    rank += ((int)(k.x == key) & (int)(4 * j < i)) + ((int)(k.y == key) & (int)(4 * j + 1 < i)) +
            ((int)(k.z == key) & (int)(4 * j + 2 < i)) + ((int)(k.w == key) & (int)(4 * j + 3 < i));
  }
#pragma unroll 16
  for (int j = 16 * w + 16; j < 64; ++j) {
    const int4 k = k4[j];
    rank += (int)(k.x < key) + (int)(k.y < key) + (int)(k.z < key) + (int)(k.w < key);
  }
  id_of[rank] = id;
  row_of[rank] = i;
  __syncthreads();
}

// Slots of a sorted tile: `slot` of this thread's row (-1: none), the adapter
// of each slot in ids, and their number.
__device__ __forceinline__ void slots_of_tile(const int* id_of, int* heads, int* ids, int& slot, int& count) {
  const int i = threadIdx.x, lane = i & 63, w = i >> 6;
  const int id = id_of[i];
  const bool first = id >= 0 && (i == 0 || id_of[i - 1] != id);
  const uint64_t m = __ballot(first);
  if (lane == 0) heads[w] = __popcll(m);
  __syncthreads();
  int n = __popcll(m & ((2ull << lane) - 1)) - 1;  // firsts up to here, in this wavefront and those before
  for (int k = 0; k < w; ++k) n += heads[k];
  if (first) ids[n] = id;
  slot = id >= 0 ? n : -1;
  count = __builtin_amdgcn_readfirstlane(heads[0] + heads[1] + heads[2] + heads[3]);
  __syncthreads();
}

// The GEMM's list of the tile (blocks: 256 ints).
__device__ __forceinline__ void list_tile(MultiTile& p, const int* id_of, const int* row_of, const int* ids, int slot,
                                          int count, int* blocks) {
  const int i = threadIdx.x;
  blocks[i] = 0;
  __syncthreads();
  if (slot >= 0) atomicOr(&blocks[slot], 1 << (row_of[i] >> 4));
  p.slot[row_of[i]] = slot;
  p.id[i] = i < count ? ids[i] : 0;
  if (i == 0) p.count = count;
  __syncthreads();
  p.blocks[i] = (uint32_t)blocks[i];
}

template <int NJ>
__global__ __launch_bounds__(256) void multi_shrink_kernel(const MultiArgs a) {
  constexpr int RG = 4, STEPS = kShrinkK / 32;
  constexpr int SLICE = kShrinkK * NJ * 32 + 128;  // bytes of a slice; fragments of the last row may reach past it
  __shared__ __attribute__((aligned(1024))) char slices[2 * SLICE];
  __shared__ __attribute__((aligned(16))) int keys[256];
  __shared__ int id_of[256], row_of[256], heads[4], ids[256];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int kc = blockIdx.y;
  const int64_t k0 = (int64_t)kc * kShrinkK;
  const int64_t klen = a.K - k0 < kShrinkK ? a.K - k0 : kShrinkK;  // multiple of 64
  const int64_t t0 = (int64_t)blockIdx.x * 256;
  int slot, count;
  sort_tile(row_id(a, t0 + threadIdx.x), keys, id_of, row_of);
  slots_of_tile(id_of, heads, ids, slot, count);
  if (kc == 0 && blockIdx.z == 0) list_tile(a.plan[blockIdx.x], id_of, row_of, ids, slot, count, keys);
  const int first = blockIdx.z, every = gridDim.z;  // this block's share of the adapters: 1 or 2 blocks
  if (first >= count) return;                       // uniform over the block
  lds_char* const lds = (lds_char*)slices;
  auto issue = [&](int s, int buf) {
    const int64_t id = __builtin_amdgcn_readfirstlane(ids[s]);
    const i32x4 ra = rsrc_words(static_cast<const char*>(a.A) + (id * a.K + k0) * a.r * 2, klen * a.r * 2);
    for (int b = w; b < a.r / 2; b += 4)  // 1 KB each
      dma16(ra, (uint32_t)(b * 1024 + lane * 16), lds_addr(lds) + buf * SLICE + b * 1024);
  };
  const int my = slot, myrow = row_of[threadIdx.x];
  const brsrc rx = make_rsrc(static_cast<const char*>(a.X) + (t0 * a.K + k0) * 2, ((a.T - t0) * a.K - k0) * 2);
  int rslot[RG], row[RG];  // of this lane's MFMA rows
  u32x4 fx[RG][STEPS];
  // rows of this block's share (every is 1 or 2)
  const bool any = __ballot(my >= 0 && (my & (every - 1)) == first) != 0;
#pragma unroll
  for (int m = 0; m < RG; ++m) {
    rslot[m] = __shfl(my, 16 * m + c);
    row[m] = __shfl(myrow, 16 * m + c);
    const uint32_t at = (uint32_t)(row[m] * a.K * 2);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)  // other rows (past T, without an adapter too) and K past the range read zero
      fx[m][s] = buf_load16(rx, any && rslot[m] >= 0 && (rslot[m] & (every - 1)) == first && 32 * s < klen ? at + (uint32_t)(32 * s + 8 * g) * 2 : 0x80000000u);
  }
  issue(first, 0);
  int buf = 0;
  for (int s = first; s < count; s += every, buf ^= 1) {
    wait_vmcnt<0>();
    __syncthreads();  // slice s is in for every wavefront, and the one before is no longer read
    if (s + every < count) issue(s + every, buf ^ 1);
    if (__ballot(my == s) == 0) continue;  // no row of this wavefront
    f32x4 acc[RG][NJ];
#pragma unroll
    for (int m = 0; m < RG; ++m)
#pragma unroll
      for (int t = 0; t < NJ; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
    const uint32_t ld = (uint32_t)a.r * 2;
    const lds_char* const at = lds + buf * SLICE + (8 * g + (c >> 2)) * ld + (lane & 3) * 8;
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
#pragma unroll
      for (int t = 0; t < NJ; ++t) {
        const bf16x8 f = lds_read_tr8(at + 32 * k * ld + 32 * t, (int)(4 * ld));
#pragma unroll
        for (int m = 0; m < RG; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, fx[m][k]), acc[m][t], 0, 0, 0);
      }
#pragma unroll
    for (int m = 0; m < RG; ++m) {
      float* u = a.upart + ((int64_t)kc * a.T + t0 + row[m]) * a.r + 4 * g;
      if (rslot[m] == s)
#pragma unroll
        for (int t = 0; t < NJ; ++t)  // rank indices 16 t + 4 g .. + 3 (the rank is a multiple of 8)
          if (16 * t + 4 * g < a.r) *reinterpret_cast<f32x4*>(u + 16 * t) = acc[m][t];
    }
  }
}

// U of many rows as the GEMM reads it: summed over the K ranges, scaled, and
// split into two bf16 parts, u = hi + lo + e with |e| <= 2^-16 |u|: the matrix
// cores take bf16, and one part alone would make a row's result depend on how
// many rows share its batch by half a bf16 step of U (the few-rows path keeps
// U in fp32); what two parts leave is 1/256 of the output's own rounding.
// hi is cut off and lo rounded, so that both have u's sign and an infinity in B_i
// is multiplied into the same infinity twice; a low part of zero, which would give
// NaN there, is the smallest normal number instead, 2^-16 of u at most.
// Four rows a block: lane 8 k +
// j of a wavefront adds columns 8 j .. 8 j + 7 over every eighth K range from k,
// and the eight sums of a column meet by a butterfly, so that the loads of 56
// ranges (K = 14336) are two round trips.  6 to 7 us at both sizes above.
__global__ __launch_bounds__(256) void multi_u_kernel(const MultiArgs a) {
  constexpr int AHEAD = 4;  // ranges a lane loads together (past the last one it is read again)
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int k0 = lane >> 3, j0 = (lane & 7) * 8;
  const int id = row_id(a, t);
  if (t >= a.T) return;
  f32x4 s0 = f32x4{0, 0, 0, 0}, s1 = s0;
  if (id >= 0 && j0 < a.r) {  // the rank is a multiple of 8
    const float* u = a.upart + t * a.r + j0;
    for (int k = k0; k < a.kc; k += 8 * AHEAD) {
      f32x4 x[AHEAD][2];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const f32x4* p = reinterpret_cast<const f32x4*>(u + (int64_t)min(k + 8 * i, a.kc - 1) * a.T * a.r);
        x[i][0] = p[0];
        x[i][1] = p[1];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        s0 = k + 8 * i < a.kc ? s0 + x[i][0] : s0;
        s1 = k + 8 * i < a.kc ? s1 + x[i][1] : s1;
      }
    }
    const float s = a.scales[id];
    s0 *= s;
    s1 *= s;
  }
#pragma unroll
  for (int d = 8; d < 64; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s0[i] += __shfl_xor(s0[i], d);
      s1[i] += __shfl_xor(s1[i], d);
    }
  if (k0 == 0 && (a.r > 32 || j0 < 32)) {
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float l[2];
      uint32_t h[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = i < 2 ? s0[2 * i + k] : s1[2 * i - 4 + k];
        h[k] = __float_as_uint(x) & 0xffff0000u;
        const float d = x - __uint_as_float(h[k]);
        l[k] = d == 0.0f && fabsf(x) >= 0x1p-110f ? copysignf(0x1p-126f, x) : d;
        if (!__builtin_isfinite(x)) {
          h[k] = f2bf(x) << 16;
          l[k] = x;
        }
      }
      hi[i] = (h[0] >> 16) | h[1];
      lo[i] = pack_bf2(l[0], l[1]);
    }
    *reinterpret_cast<u32x4*>(a.u + t * 64 + j0) = hi;
    *reinterpret_cast<u32x4*>(a.u + (a.r > 32 ? (a.T + t) * 64 : t * 64 + 32) + j0) = lo;
  }
}

// ---------------------------------------------------------------------------
// Y = sum of the K ranges' parts (or Y itself) + s_i U B_i, rounded once.
// A block has four rows and 512 columns (a lane owns 8 of them); its four
// wavefronts share the K parts and the ranks of all four rows, so that few
// rows still have enough loads in flight, and meet in LDS, where wavefront w
// adds them in ascending order for row w.
// Measured: one row of 4096 5 us, 67 rows of 14336 at rank 16 8.7 us (7.7 MB of
// parts, 14.7 MB of B_i): latency, with the launch that precedes it.
// ---------------------------------------------------------------------------
// Eight columns of a row.
struct Cols {
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
  static __device__ __forceinline__ void add(const float* p, float (&f)[8]) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] += x[k];
      f[4 + k] += y[k];
    }
  }
};

__global__ __launch_bounds__(256) void multi_expand_kernel(const MultiArgs a) {
  constexpr int C = 8;
  __shared__ float us[4][64];
  __shared__ float sum[4][4][64 * C];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int cols = (int)((a.N + 64 * C - 1) / (64 * C));
  const int64_t t0 = (int64_t)(blockIdx.x / cols) * 4;
  const int64_t col = ((int64_t)(blockIdx.x % cols) * 64 + lane) * C;
  const bool in = col < a.N;
  const int rows = a.T - t0 < 4 ? (int)(a.T - t0) : 4;
  int id[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) id[i] = __builtin_amdgcn_readfirstlane(row_id(a, t0 + i));
  if (id[w] >= 0 && lane < a.r) {
    float s = 0.0f;
    const float* u = a.upart + (t0 + w) * a.r + lane;
#pragma unroll 4
    for (int k = 0; k < a.kc; ++k) s += u[(int64_t)k * a.T * a.r];
    us[w][lane] = s * a.scales[id[w]];
  }
  float y[4][C];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) y[i][j] = 0.0f;
  if (in) {
    if (a.part == nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i == w && i < rows) Cols::load(a.Y, (t0 + i) * a.N + col, y[i]);
    } else {
      const int64_t stride = a.T * a.N;
      for (int k = w; k < a.ks; k += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < rows) Cols::add(a.part + k * stride + (t0 + i) * a.N + col, y[i]);
    }
  }
  __syncthreads();
  if (in) {
    const int64_t bs = (int64_t)a.r * a.N;
    auto rank = [&](int id_, int j, float (&b)[C]) { Cols::load(a.B, id_ * bs + (int64_t)j * a.N + col, b); };
    if (id[0] >= 0 && id[0] == id[1] && id[0] == id[2] && id[0] == id[3]) {
#pragma unroll 4
      for (int j = w; j < a.r; j += 4) {
        float b[C];
        rank(id[0], j, b);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < C; ++k) y[i][k] = fmaf(us[i][j], b[k], y[i][k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (id[i] < 0) continue;
#pragma unroll 4
        for (int j = w; j < a.r; j += 4) {
          float b[C];
          rank(id[i], j, b);
#pragma unroll
          for (int k = 0; k < C; ++k) y[i][k] = fmaf(us[i][j], b[k], y[i][k]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) sum[w][i][j * 64 + lane] = y[i][j];
  __syncthreads();
  if (in && w < rows) {
    float o[C];
#pragma unroll
    for (int j = 0; j < C; ++j)
      o[j] = sum[0][w][j * 64 + lane] + sum[1][w][j * 64 + lane] + sum[2][w][j * 64 + lane] + sum[3][w][j * 64 + lane];
    Cols::store(a.Y, (t0 + w) * a.N + col, o);
  }
}

// U in fp32: one block per row (x, then y); threads are (K slot, rank index), slots added in ascending order.
// A thread's chain of round trips is the bound, so a rank above 16 gets 1024
// threads (65 rows of 1500 at rank 64: 14 us, 28 with 256) and a lower one,
// whose slots are many already, 256 (128 rows of 256 at rank 8: 3.7 us).
template <int THREADS>
__global__ __launch_bounds__(THREADS) void multi_shrink_f32_kernel(const MultiArgs a) {
  constexpr int AHEAD = THREADS > 256 ? 16 : 8;  // K a thread loads together (past the last one it is read again)
  __shared__ float red[THREADS];
  const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int id = row_id(a, t);
  if (id < 0) return;  // uniform
  const int slots = THREADS / a.r, slot = threadIdx.x / a.r, j = threadIdx.x % a.r;
  const float* x = static_cast<const float*>(a.X) + t * a.K;
  const float* A = static_cast<const float*>(a.A) + (int64_t)id * a.K * a.r;
  float s = 0.0f;
  if (slot < slots)
    for (int64_t k0 = slot; k0 < a.K; k0 += AHEAD * slots) {
      float xs[AHEAD], as[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int64_t k = min(k0 + i * slots, a.K - 1);
        xs[i] = x[k];
        as[i] = A[k * a.r + j];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) s = k0 + i * slots < a.K ? fmaf(xs[i], as[i], s) : s;
    }
  red[threadIdx.x] = s;
  __syncthreads();
  if (slot == 0) {
    for (int q = 1; q < slots; ++q) s += red[q * a.r + j];
    a.upart[t * a.r + j] = s;
  }
}

// ---------------------------------------------------------------------------
// Y in fp32: v_mfma_f32_16x16x4 straight from global memory, 32 x 32 outputs a
// wavefront, any widths.  A step is 16 K: lane 16 q + c holds K 4 q .. 4 q + 3
// of row c (X, one 16-byte load) and of column c (W), and gives one of the
// four to each MFMA, which takes any K as long as both operands agree.
//   KSPLIT: the block is one 32 x 32 tile and its wavefronts quarter K: few
//   tiles still fill the chip, and the chain of loads is a quarter as long.
//   Else 64 x 64 a block, a quadrant a wavefront: half the traffic.
// The adapter's term joins in the epilogue, from U of the tile's rows in LDS.
// Measured: 128 rows of 256 x 704 7.2 us: a chain of loads and products too short
// to fill the chip, not the 0.9 MB that it moves.  4096 rows of 1024 x 1024 138
// us, 62 TFLOP/s of the 152 a library product reaches: no operand is shared
// through LDS.
// ---------------------------------------------------------------------------
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

template <bool KSPLIT>
__global__ __launch_bounds__(256) void multi_f32_kernel(const MultiArgs a) {
  constexpr int TILE = KSPLIT ? 32 : 64, DEPTH = 4;  // DEPTH steps of loads in flight
  __shared__ f32x4 red[KSPLIT ? 4 : 1][KSPLIT ? 4 : 1][64];
  __shared__ float us[TILE][65];
  __shared__ int ids[TILE];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int tiles_n = (int)((a.N + TILE - 1) / TILE);
  const int64_t mt = (int64_t)(blockIdx.x / tiles_n) * TILE, nt = (int64_t)(blockIdx.x % tiles_n) * TILE;
  const int64_t m0 = KSPLIT ? mt : mt + 32 * (w & 1), n0 = KSPLIT ? nt : nt + 32 * (w >> 1);
  for (int i = threadIdx.x; i < TILE; i += 256) ids[i] = row_id(a, mt + i);
  __syncthreads();
  for (int e = threadIdx.x; e < TILE * a.r; e += 256) {
    const int row = e / a.r, j = e % a.r, id = ids[row];
    us[row][j] = id >= 0 ? a.upart[(mt + row) * a.r + j] * a.scales[id] : 0.0f;
  }
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  if (a.W != nullptr) {
    const int64_t quarter = (a.K + 63) / 64 * 16;
    const int64_t k0 = KSPLIT ? w * quarter : 0;
    const int64_t k1 = KSPLIT && k0 + quarter < a.K ? k0 + quarter : a.K;
    const float *X = static_cast<const float*>(a.X), *W = static_cast<const float*>(a.W);
    // Rows and columns past the end read the last one, whose sums are not stored: no load is guarded.
    const float *xr[2], *wc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xr[i] = X + min(m0 + 16 * i + c, a.T - 1) * a.K + 4 * g;
      wc[i] = W + min(n0 + 16 * i + c, a.N - 1) + 4 * g * a.N;
    }
    f32x4 x[DEPTH][2];
    float wv[DEPTH][2][4];
    auto load = [&](int s, int64_t k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[s][i] = *reinterpret_cast<const f32x4u*>(xr[i] + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) wv[s][i][q] = wc[i][(k + q) * a.N];
      }
    };
    auto mma = [&](int s) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[s][i][q], wv[s][j][q], acc[i][j], 0, 0, 0);
    };
    int64_t k = k0;
    if (k0 + 16 * DEPTH <= k1) {
#pragma unroll
      for (int s = 0; s < DEPTH; ++s) load(s, k0 + 16 * s);
      for (; k + 32 * DEPTH <= k1; k += 16 * DEPTH)
#pragma unroll
        for (int s = 0; s < DEPTH; ++s) {
          mma(s);
          load(s, k + 16 * (DEPTH + s));
        }
#pragma unroll
      for (int s = 0; s < DEPTH; ++s) mma(s);
      k += 16 * DEPTH;
    }
    for (; k + 16 <= k1; k += 16) {
      load(0, k);
      mma(0);
    }
    if (k < k1) {  // fewer than 16 K: zeros past them on both sides
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t kk = k + 4 * g + q, kc = min(kk, a.K - 1) - 4 * g;
          const float xv = xr[i][kc], v = wc[i][kc * a.N];
          x[0][i][q] = kk < k1 ? xv : 0.0f;
          wv[0][i][q] = kk < k1 ? v : 0.0f;
        }
      mma(0);
    }
  }
  if constexpr (KSPLIT) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) red[w][2 * i + j][lane] = acc[i][j];
  }
  __syncthreads();
  // tile (i, j) of the wavefront: rows m0 + 16 i + 4 g + v, column n0 + 16 j + c
  auto finish = [&](int i, int j, f32x4 y) {
    const int64_t n = n0 + 16 * j + c;
    if (n >= a.N) return;
    const int row = (int)(m0 - mt) + 16 * i + 4 * g;
    int id[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      id[v] = ids[row + v];
      if (a.W == nullptr && mt + row + v < a.T) y[v] = static_cast<const float*>(a.Y)[(mt + row + v) * a.N + n];
    }
    const float* B = static_cast<const float*>(a.B) + n;
    const int64_t bs = (int64_t)a.r * a.N;
    if (id[0] == id[1] && id[0] == id[2] && id[0] == id[3]) {
      if (id[0] >= 0)
        for (int k0 = 0; k0 < a.r; k0 += 8) {
          float b[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] = B[id[0] * bs + (int64_t)min(k0 + k, a.r - 1) * a.N];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int v = 0; v < 4; ++v) y[v] = k0 + k < a.r ? fmaf(us[row + v][min(k0 + k, a.r - 1)], b[k], y[v]) : y[v];
        }
    } else {  // at least one of the four has an adapter: a row without one reads that one's ranks
      const int top = max(max(id[0], id[1]), max(id[2], id[3]));
      for (int k0 = 0; k0 < a.r; k0 += 8) {
        float b[4][8];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int k = 0; k < 8; ++k) b[v][k] = B[(id[v] < 0 ? top : id[v]) * bs + (int64_t)min(k0 + k, a.r - 1) * a.N];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            y[v] = id[v] >= 0 && k0 + k < a.r ? fmaf(us[row + v][min(k0 + k, a.r - 1)], b[v][k], y[v]) : y[v];
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (mt + row + v < a.T) static_cast<float*>(a.Y)[(mt + row + v) * a.N + n] = y[v];
  };
  if constexpr (KSPLIT) {
    finish(w >> 1, w & 1, ((red[0][w][lane] + red[1][w][lane]) + red[2][w][lane]) + red[3][w][lane]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) finish(i, j, acc[i][j]);
  }
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
// Which path a bf16 call takes.  Few rows: W is streamed through 128-column
// tiles with K split over the grid, and the adapters join the fp32 sums as
// those are added up.  Many: the 256 x 256 tiles of the GEMM, with the adapters
// in its epilogue.  The rule compares models of both, fitted to 900 shapes of
// 136 to 3600 rows, 64 to 14336 wide, with 2 to 60 adapters of rank 16 to 64
// (us; the choice is 3% from the faster of the two in the mean).  Few: X W, the
// shrink of 16-row blocks that min(16, n) share, the parts' sum and U B. Many:
// a longer start, the GEMM, and the walk over the adapters a 256-row tile
// meets, counted as if the rows of all n came in runs, and at most 16: n is
// what is loaded, not what the batch uses.  Measured, few / many:
//    4096 x 4096, 12 of rank 32: 71 / 60 at 562 rows
//    1664 x 192, 2 of rank 16: 17 / 46 at 1100, 33 / 50 at 4096
//    1472 x 704, 2 of rank 16: 25 / 45 at 1536;  60 of rank 64: 69 / 64
//    14336 x 4096, 2 of rank 16: 79 / 90 at 300, 125 / 97 at 562
//    128 x 1664, 2 of rank 16: 23 / 25 at 1536, 32 / 25 at 2304
// (the many side with U in one bf16 part; two add 1 to 4% to it)
// Up to kFewRows rows always few, past kManyRows always many.
constexpr int64_t kFewRows = 128, kManyRows = 4096;
int shrink_share(int64_t n);
bool few_rows(const lora_multi_desc& d) {
  if (d.T <= kFewRows || d.T > kManyRows) return d.T <= kFewRows;
  const double t = (double)d.T, k = (double)d.K, n = (double)d.N, r = d.n ? (double)d.r : 0.0, z = shrink_share(d.n);
  const double met = std::min(std::min((double)d.n, 16.0), 256.0 * (double)d.n / t + 1);
  const double few = 15 + t / 1e6 * (k * (3.2e-3 * n + 1.35e-2 * z * r) + n * (2.1 + 3.2e-2 * r) + r * (29 + 8.8 * z));
  const double many = 23 + k / 250 + t / 1e6 * (1.33e-3 * k * n + 35 * r) + met * (0.9 + r / 85);
  return few < many;
}

// Row tiles of at most 128 rows, and the 16-row blocks of each.
int row_tiles(int64_t T) { return (int)cdiv(T, 128); }
int row_blocks(int64_t T) { return (int)cdiv(cdiv(T, 16), row_tiles(T)); }

// K ranges of the shrink.
int shrink_ranges(bool few, int64_t K) { return (int)cdiv(K, few ? 4 * kShrinkK : kShrinkK); }
// Few rows: 16 of them meet at most 16 adapters, each in a block of its own.
int shrink_share(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(16, n)); }
int shrink_blocks(int64_t T, int64_t K, int64_t n) {
  return n == 0 ? 0 : (int)cdiv(T, 16) * shrink_ranges(true, K) * shrink_share(n);
}

// K ranges of X W for few rows, by a model of what grows with them: the K
// stages of the fullest CU, 0.3 to 0.6 us each with 16 to 128 rows, against the
// fp32 parts, written and read again at some 3 TB/s.  (67 rows of 14336 x 4096:
// 76 us with 2 ranges, 41 with 8, 47 with 16; 32 rows of 4096 x 4096: 33 us with
// 1, 17 with 4, 21 with 16.)
int base_ksplit(int64_t T, int64_t K, int64_t N) {
  const int64_t units = cdiv(N, 128) * row_tiles(T), steps = K / 64;
  double best = 0.0;
  int bs = 1;
  for (int s = 1; s <= 32 && (s == 1 || steps / s >= 4); ++s) {
    const double t = (0.3 + 0.04 * row_blocks(T)) * (double)(cdiv(units * s, 256) * cdiv(steps, s)) + (double)s * T * N * 8 / 3e6;
    if (s == 1 || t < best * 0.98) {
      best = t;
      bs = s;
    }
  }
  return bs;
}

// The shrink joins the launch of X W up to this many blocks: it then starts at
// once and fills what the others leave free, but takes their amount of LDS
// (20 blocks to 1536: 2 to 12 us less joined; 2048 and more: 3 to 30 us more).
constexpr int kJoin = 1536;

hipError_t launch_shrink_few(const MultiArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.nshrink);
  switch (cdiv(a.r, 16)) {
    case 1: hipLaunchKernelGGL(multi_shrink_few_kernel<1>, grid, dim3(256), 0, st, a); break;
    case 2: hipLaunchKernelGGL(multi_shrink_few_kernel<2>, grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL(multi_shrink_few_kernel<3>, grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL(multi_shrink_few_kernel<4>, grid, dim3(256), 0, st, a); break;
  }
  return hipGetLastError();
}
template <int MT>
hipError_t launch_few(const MultiArgs& a, hipStream_t st) {
  const int blocks = a.nshrink + (a.W ? (int)cdiv(a.ntn * a.ks, 8) * 8 * a.ntm : 0);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(multi_few_kernel<MT>, dim3((unsigned)blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_few_mt(const MultiArgs& a, hipStream_t st) {
  switch (row_blocks(a.T)) {
    case 1: return launch_few<1>(a, st);
    case 2: return launch_few<2>(a, st);
    case 3: return launch_few<3>(a, st);
    case 4: return launch_few<4>(a, st);
    case 5: return launch_few<5>(a, st);
    case 6: return launch_few<6>(a, st);
    case 7: return launch_few<7>(a, st);
    default: return launch_few<8>(a, st);
  }
}
// Two blocks share the adapters of a tile where the grid leaves room.
hipError_t launch_shrink(const MultiArgs& a, hipStream_t st) {
  const int64_t x = cdiv(a.T, 256);
  const dim3 grid((unsigned)x, (unsigned)a.kc, x * a.kc < 512 && a.n > 1 ? 2 : 1);
  switch (cdiv(a.r, 16)) {
    case 1: hipLaunchKernelGGL(multi_shrink_kernel<1>, grid, dim3(256), 0, st, a); break;
    case 2: hipLaunchKernelGGL(multi_shrink_kernel<2>, grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL(multi_shrink_kernel<3>, grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL(multi_shrink_kernel<4>, grid, dim3(256), 0, st, a); break;
  }
  return hipGetLastError();
}

// Workspace of a call.
struct MultiPlan {
  bool few;    // the path of few rows
  bool tiles;  // the GEMM path
  int ks, kc;
  float *part, *upart;
  uint16_t* u;
  MultiTile* plan;
  size_t bytes;
};
MultiPlan plan_multi(const lora_multi_desc& d, bool base, void* ws) {
  MultiPlan p{};
  const bool bf16 = d.dtype == LORA_BF16;
  p.few = base ? few_rows(d) : d.T <= kFewRows;
  p.tiles = bf16 && base && !p.few;
  p.ks = !bf16 || !base || d.T == 0 ? 1 : p.tiles ? store_gemm_ksplit(d.T, d.N, d.K)
                                              : base_ksplit(d.T, d.K, d.N);
  p.kc = bf16 ? shrink_ranges(p.few, d.K) : 1;
  Ws w(ws);
  p.upart = static_cast<float*>(w.take((size_t)p.kc * d.T * d.r * 4));
  if (p.tiles) p.u = static_cast<uint16_t*>(w.take((size_t)d.T * (d.r > 32 ? 256 : 128)));
  if (bf16 && !p.few) p.plan = static_cast<MultiTile*>(w.take((size_t)cdiv(d.T, 256) * sizeof(MultiTile)));
  if (bf16 && base && (!p.tiles || p.ks > 1)) p.part = static_cast<float*>(w.take((size_t)p.ks * d.T * d.N * 4));
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
  CHECK(d->K <= (1 << 22) && d->N <= (1 << 22), LORA_ESHAPE, "K = %lld and N = %lld must be at most %d", (long long)d->K,
        (long long)d->N, 1 << 22);
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
  // with W or without, the larger
  if (bytes) *bytes = std::max(plan_multi(*d, true, nullptr).bytes, plan_multi(*d, false, nullptr).bytes);
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
  a.ntn = (int32_t)cdiv(d->N, 128);
  a.u = p.u;
  a.plan = p.plan;
  if (bf16) {
    if (p.few) {
      a.ntm = row_tiles(d->T);
      a.nz = shrink_share(d->n);
      a.nshrink = shrink_blocks(d->T, d->K, d->n);
      if (a.nshrink > kJoin) {
        LAUNCHN("multi_shrink_few", st, launch_shrink_few(a, st));
        a.nshrink = 0;
      }
      LAUNCHN("multi_few", st, launch_few_mt(a, st));
    } else if (p.tiles || d->n > 0) {  // without adapters the GEMM's tiles are still listed, as empty
      LAUNCHN("multi_shrink", st, launch_shrink(a, st));
    }
    if (p.tiles) {
      {
        TraceScope ts("multi_u", st);
        hipLaunchKernelGGL(multi_u_kernel, dim3((unsigned)cdiv(d->T, 4)), dim3(256), 0, st, a);
        LAUNCH(hipGetLastError());
      }
      GemmArgs g{};
      g.M = d->T;
      g.nseg = 1;
      g.nreg = 1;
      g.epi = EPI_STORE;
      g.bkind = B_NN;
      g.group = 8;
      g.seg[0].A = X;
      g.seg[0].lda = d->K;
      g.seg[0].K = d->K;
      g.seg[0].b[0][0].p = W;
      g.seg[0].b[0][0].ld = d->N;
      g.reg[0].N = d->N;
      g.reg[0].out = Y;
      g.reg[0].ldo = d->N;
      g.ntile_m = cdiv(d->T, gemm_tile_rows(true));
      g.ntile_n = cdiv(d->N, gemm_tile_cols(true, false));
      g.ksplit = p.ks;
      g.ksplit_t0 = (int32_t)store_gemm_split_from(g.ntile_m * g.ntile_n, p.ks);
      g.kpart = p.part;
      g.mt_u = p.u;
      g.mt_b = B;
      g.mt_plan = p.plan;
      g.mt_r = (int32_t)d->r;
      LAUNCHN("gemm_nn_store_multi", st, launch_gemm_bf16(g, st));
      if (p.ks > 1) LAUNCHN("ksplit_reduce", st, launch_ksplit_reduce(g, st));
      return LORA_OK;
    }
    TraceScope ts("multi_expand", st);
    hipLaunchKernelGGL(multi_expand_kernel, dim3((unsigned)(cdiv(d->N, 512) * cdiv(d->T, 4))), dim3(256), 0, st, a);
    LAUNCH(hipGetLastError());
    return LORA_OK;
  }
  if (d->n > 0) {
    TraceScope ts("multi_shrink_f32", st);
    // a launch may have 2^32 - 1 threads along x
    const int64_t gx = std::min<int64_t>(d->T, 1 << 20);
    const dim3 rows((unsigned)gx, (unsigned)cdiv(d->T, gx));
    if (d->r > 16) hipLaunchKernelGGL(multi_shrink_f32_kernel<1024>, rows, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(multi_shrink_f32_kernel<256>, rows, dim3(256), 0, st, a);
    LAUNCH(hipGetLastError());
  } else if (W == nullptr) {
    return LORA_OK;
  }
  TraceScope ts("multi_f32", st);
  const int64_t big = cdiv(d->T, 64) * cdiv(d->N, 64), small = cdiv(d->T, 32) * cdiv(d->N, 32);
  if (big >= 512) hipLaunchKernelGGL(multi_f32_kernel<false>, dim3((unsigned)big), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(multi_f32_kernel<true>, dim3((unsigned)small), dim3(256), 0, st, a);
  LAUNCH(hipGetLastError());
  return LORA_OK;
}

}  // extern "C"
