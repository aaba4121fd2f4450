// Sparse attention over the 8-bit latent cache (the attention of the decode
// step, model.py 596-605 of the atlas page "Query-key similarity", on cached
// rows held as E4M3 codes; the pages keep them in bf16).
//
// Cache: codes e4m3 [slots, S_max, 512], rotary keys bf16 [slots, S_max, 64]
// and one f32 scale for each block of `block` positions; position t stands for
// the latent s * code_t and the rotary key s * pe_t, s = scale[t / block], so
//   score_t,h = scale * s_t * (q_lat_h . code_t + q_pe_h . pe_t)
//   O_h       = sum_t p_t,h s_t code_t / sum_t p_t,h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "kernels.cuh"
#include "ptx.cuh"

namespace mla {

// ---------------------------------------------------------------- E4M3 limbs
// A factor kept as two E4M3 numbers has nine significant bits (four, four and
// the second's sign), one more than bf16's, and 8-bit products run at twice the
// rate of bf16 products: two of them cost what one bf16 product costs, and the
// codes go to the tensor cores as they lie in the cache, with no conversion and
// at half of bf16's shared memory.  (The softmax weights' second number is E5M2,
// for its range: eight bits.)
//
// An fp16 number f of magnitude below 1.8 has E4M3's exponent field for the
// value 2^8 f, subnormals included, so rounding 2^8 f to E4M3 is rounding f's
// bits to a multiple of 2^7 and taking seven of them.  (The conversion
// instructions do a quarter of the integer units' rate: a tile's P took 1020
// cycles with them, 600 so.)  Ties go away from zero.
//
// Two fp16 numbers: their first limbs as fp16 values, and what those leave.
__device__ __forceinline__ uint32_t limb_first(uint32_t f16x2) { return f16x2 + 0x00400040u; }  // bits 7.. are the limb
__device__ __forceinline__ __half2 limb_rest(uint32_t f16x2, uint32_t first) {
  const uint32_t cut = first & 0xbf80bf80u;
  return __hsub2(*reinterpret_cast<const __half2*>(&f16x2), *reinterpret_cast<const __half2*>(&cut));
}
// The E4M3 bytes of four rounded fp16 numbers (sign, then bits 13..7 of each:
// the magnitude, below 2^14, is doubled under the sign).
__device__ __forceinline__ uint32_t limb_bytes(uint32_t a, uint32_t b) {
  return __byte_perm(a + (a & 0x7fff7fffu), b + (b & 0x7fff7fffu), 0x7531);
}
__device__ __forceinline__ uint32_t limb_bytes_positive(uint32_t a, uint32_t b) {
  return __byte_perm(a << 1, b << 1, 0x7531);
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
// The E5M2 bytes of 2^8 times four fp16 numbers (below 2^7): an E5M2 number is
// the upper byte of an fp16 one.  Ties go away from zero.
__device__ __forceinline__ uint32_t limb_bytes_e5m2(__half2 a, __half2 b) {
  const __half2 up = __float2half2_rn(256.f);
  return __byte_perm(half2_bits(__hmul2(a, up)) + 0x00800080u, half2_bits(__hmul2(b, up)) + 0x00800080u, 0x7531);
}

// Exponent e with |amax| 2^e in (224, 448] (0 for amax = 0).
__device__ __forceinline__ int limb_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int k;
  const float m = frexpf(amax, &k);          // amax = m 2^k, m in [1/2, 1)
  const int e = (m <= 0.875f ? 9 : 8) - k;   // 448 = 0.875 2^9
  return e < -118 ? -118 : (e > 118 ? 118 : e);  // 2^(e - 8) and 2^-e are normal
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 126

// Four query factors x as limbs, from fp16 numbers 2^(e - 8) x: x 2^e = hi + lo /
// lo_scale.  A second limb that is scaled up by 16 keeps its bits however small
// x is: a bf16 x is met exactly (4 + 4 signed bits) down to 2^-17 of the
// largest; one that is not, down to 2^-10, and to 2^-19 of the largest below.
constexpr float kLimbLo = 1.f / 16.f;
__device__ __forceinline__ void limbs4_half(uint32_t f01, uint32_t f23, float lo_scale, uint32_t* hi, uint32_t* lo) {
  uint32_t first[2], rest[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t f = i ? f23 : f01;
    first[i] = limb_first(f);
    rest[i] = limb_first(half2_bits(__hmul2(limb_rest(f, first[i]), __float2half2_rn(lo_scale))));
  }
  *hi = limb_bytes(first[0], first[1]);
  *lo = limb_bytes(rest[0], rest[1]);
}
// The same from bf16 numbers x, `mul` = 2^(e - 8).
__device__ __forceinline__ uint32_t half2_of_bf16(uint32_t x, float mul) {
  return half2_bits(__floats2half2_rn(__uint_as_float(x << 16) * mul, __uint_as_float(x & 0xffff0000u) * mul));
}
__device__ __forceinline__ void limbs4(uint32_t x01, uint32_t x23, float mul, float lo_scale, uint32_t* hi, uint32_t* lo) {
  limbs4_half(half2_of_bf16(x01, mul), half2_of_bf16(x23, mul), lo_scale, hi, lo);
}
// 2^x as two fp16 numbers (0 below 2^-24, 2^15 above it).
__device__ __forceinline__ __half2 half2_power(int x) {
  const uint32_t b = x >= -14 ? (uint32_t)(min(x, 15) + 15) << 10 : (x >= -24 ? 1u << (x + 24) : 0u);
  const uint32_t w = b | (b << 16);
  return *reinterpret_cast<const __half2*>(&w);
}

// The magnitudes' bits of two bf16 numbers, each the larger of m's and x's.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x) { return __vmaxu2(m, x & 0x7fff7fffu); }

// The largest finite magnitude of a thread's 32 rotary factors (one that holds an
// infinity or NaN counts none: its head's scores are NaN anyway).
__device__ __forceinline__ float rotary_top(const uint4 (&r)[4]) {
  uint32_t m2 = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) m2 = amax2(amax2(amax2(amax2(m2, r[u].x), r[u].y), r[u].z), r[u].w);
  const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  return m < 0x7f80u ? __uint_as_float(m << 16) : 0.f;
}
// The common exponent of queries up to `amax` and rotary ones up to `rmax`, which
// go along as 2^e q_pe: these stay below 2^60 (2^63 in the lo rows), so that no
// sum of theirs overflows where the others are far smaller.
__device__ __forceinline__ int query_exponent(float amax, float rmax) {
  const int e = limb_exponent(amax);
  if (!(rmax > 0.f)) return e;
  int k;
  frexpf(rmax, &k);  // rmax < 2^k
  return min(e, 60 - k);
}

// =============================================================================
// sparse_attend_fp8_kernel
//
// Per tile of 128 positions:
//   S[r, t]      = q_r . code_t   M = 128 rows: the hi and lo limbs of 64 heads'
//                                 queries (TMEM; 16 heads' hi rows, then their
//                                 lo rows, in every 32 lanes), N = 128 positions
//                                 (K-major, as gathered), plus the bf16 rotary
//                                 product, half of it in each.  S_hi + S_lo / 16
//                                 meets in one shuffle across half a warp;
//   y[h, t]      = scale s_t S + log2 s_t, the log2 weight of position t's codes;
//   P[h, t]      = 2^(y - m_h), row sum += P / s_t;
//   O^T[c, h]   += code_t[c] P[h, t]   M = 128 latent columns, N = the heads, the
//                                 same codes read M-major, P as two limbs one
//                                 after the other.
// Every score is formed whole in one SM and in f32.  O is kept transposed so
// that P is the N operand: as rows, P's two limbs would need two sets of
// accumulators.
//
// Pair (more than 64 heads): a 2-CTA cluster per (row, split).  CTA r owns 64
// heads of QK and softmax, and latent columns 256 r.. of O for all heads, so it
// sends its P to the peer (bulk copies: the softmax warps go on meanwhile).  N
// is 128 in both products: an MMA of N = 64 takes 60 cycles, one of N = 128
// takes 65.  Only P crosses SMs; the rows are read by both, once from L2.
// Single (at most 64 heads): one CTA per (row, split) owns all 512 columns.
//
// m_h is the largest y of some tile plus a margin, and moves only when P would
// leave E4M3's range or lose its small weights; the softmax warps then rescale
// the columns of O of the heads it moved for between two PVs, in both CTAs of a
// pair (which tell each other as soon as they know; P does not wait for that,
// only PV does).
//
// Shared memory: blocks of 16 KB (128 positions x 128 bytes, 128-byte swizzle).
//   Pair:   three for what only QK reads (rotary rows, the peer's columns),
//           three stages of the CTA's own columns (two blocks each, held until
//           PV has read them), three limbs of P of 128 heads.
//   Single: a ring of two for the rotary rows, two stages of four blocks, two
//           buffers of P.
//
// Warps (512 threads): 0-7 softmax (warp w: TMEM lanes 32 (w % 4).., positions
// 64 (w / 4)..), 8-11 gather (one on each sub-partition of the SM: two warps on
// two of them took 4900 cycles a tile), 12 query load and QK issue, 13 TMEM and PV
// issue, 14 positions, scales and L2 prefetch, 15 pushes.
//
// Measured (one B200, 64 rows of 2048 positions, 128 heads): 50 us, of which 10
// lie before the first and behind the last tile (set-up 1.5, the query 0.6 and
// its limbs 2.5, the last tile's way to O 1.5, O to memory 1.9) and 2.4 us, 4500
// cycles, are a tile's.  A tile's limits are 2340 cycles of MMA, about 2800 of
// shared-memory traffic (the MMAs' operands, the copies, P) and 2850 of gather
// from HBM (1290 from L2); what sets the pace is the chain of hand-overs between
// them, each of a few hundred cycles: without the softmax's arithmetic a tile
// takes 5% less, with half the MMAs 7%, with the peer's columns not copied 8%,
// with all three 22%.  Slower: MMAs over both CTAs (cta_group::2, M = 256, N =
// 128, no pushes: 135 cycles an MMA, 59.6 us), two full sets of P and two stages
// (59), one set of P and a ring of four (53.3), PV behind the next QK but one
// (58.5), the L2 prefetch in bulk (59.7) or none (50.0).
// =============================================================================
constexpr int kF8Heads = 64;           // heads of a CTA's QK and softmax
constexpr int kF8Nt = 128;             // positions of a tile
constexpr int kF8Block = kF8Nt * 128;  // 16 KB
__host__ __device__ constexpr int f8_ring(bool pair) { return pair ? 3 : 2; }         // blocks that only QK reads
__host__ __device__ constexpr int f8_ring_per(bool pair) { return pair ? 3 : 1; }     // of them a tile
__host__ __device__ constexpr int f8_stages(bool pair) { return pair ? 3 : 2; }       // stages of own columns
__host__ __device__ constexpr int f8_own(bool pair) { return pair ? 2 : 4; }          // blocks of a stage
__host__ __device__ constexpr int f8_own_at(bool pair, int st, int i) { return (f8_ring(pair) + f8_own(pair) * st + i) * kF8Block; }
// A limb of a CTA's P: 64 heads x 128 positions (K-major, 128-byte swizzle).
constexpr int kF8Limb = kF8Nt * kF8Heads;
// Where tile j's hi or lo limbs of P lie.  Pair: three buffers of 128 heads take
// turns (two for each limb would cost a stage).  Single: two of both limbs.
__host__ __device__ constexpr int f8_p_at(bool pair, int j, int lo) {
  return f8_own_at(pair, f8_stages(pair), 0) + (pair ? (2 * j + lo) % 3 * (2 * kF8Limb) : (j & 1) * (2 * kF8Limb) + lo * kF8Limb);
}
constexpr int kF8OffQpe = 12 * kF8Block;                     // 128 rows
constexpr int kF8OffKey = kF8OffQpe + kF8Block;              // f32 [4][3][128]: what a position's scale enters by
constexpr int kF8OffPos = kF8OffKey + 4 * 3 * kF8Nt * 4;     // int [4][128]: a tile's positions, -1 = masked
constexpr int kF8OffRed = kF8OffPos + 4 * kF8Nt * 4;         // f32 [4][2][64]
constexpr int kF8OffMove = kF8OffRed + 4 * 2 * kF8Heads * 4; // F8Move [2][2]
constexpr int kF8OffFin = kF8OffMove + 2 * 2 * 272;          // f32 [128]: one over the row sums
constexpr int kF8OffBar = kF8OffFin + kH * 4;
constexpr int kF8SmemBytes = kF8OffBar + 512 + kSmemAlignPad;
constexpr int kF8SoftmaxWarps = 8;
constexpr int kF8GatherWarp = 8, kF8GatherWarps = 4, kF8QkWarp = 12, kF8PvWarp = 13, kF8IndexWarp = 14, kF8PushWarp = 15;
constexpr int kF8Threads = 512;
constexpr uint32_t kF8ColS = 0;    // scores: 128 columns
constexpr uint32_t kF8ColQ = 128;  // the query's limbs: 128 columns of four codes
constexpr uint32_t kF8ColO = 256;  // pair: 2 blocks of 128 heads; single: 4 blocks of 64
// P is formed in fp16 at 2^-8 of what the products see; the powers below are
// theirs.  Its first limb is E4M3, its second what that leaves, as E5M2: 2^-4 of
// 2^-4, eight significant bits like bf16's, down to P = 2^-6.  A smaller P keeps
// fewer (E4M3 steps by 2^-9 there, E5M2 has three bits of the rest): it is off by
// 2^-14 at most.  Over a tile that may add up to 2^-7, so it has to be little
// beside what the head has:
//   a new m_h puts the largest P of its tile at 2^2, and a later one may reach
//   2^8.75 = 430 (E4M3's largest value is 448) before m_h has to rise;
//   m_h falls again where a tile's largest is below 2^1 and the sum of P over the
//   j tiles before it below 2^1 (j + 1): a tile that keeps its m_h is then off by
//   2^-8 of its largest weight or of the mean of the tiles' sums at most.
// m_h falls no further than 2^-32 of the largest weight so far.  A second limb in
// E4M3, with references that only rise, loses all weights below 2^-13 of the
// largest: beside one of 0.8 of the softmax the mix of 2048 positions is off by
// 3.2e-2, of 8192 by 1.0e-1, against 2e-4 and 8e-5 so (bf16 weights 8e-4; a
// restatement on the CPU).  Measured, 64 rows of 2048 positions whose scales
// differ by factors of four: 50.7 us, 49.6 without falling references; new ones
// at 2^3 51.4, at 2^4 52.8 (they fall and rise more often).
constexpr float kF8RefMargin = 8.0f - 2.0f;
constexpr float kF8RefLimit = 8.75f - 8.0f;
constexpr float kF8RefFloor = 1.0f - 8.0f;
constexpr float kF8MassFloor = 1.f / 128.f;  // 2^kF8RefFloor
constexpr float kF8RefFall = 32.f;
constexpr float kF8NoRef = -1e30f;  // m_h before any position counted
// How a tile moves the references of a CTA's 64 heads.
struct F8Move {
  float factor[kF8Heads];  // O's columns are multiplied by it
  uint32_t moved[4];       // the heads whose factor is not 1, 16 a word
};
static_assert(sizeof(F8Move) == 272, "kF8OffFin");
static_assert(kF8SmemBytes <= 232448, "shared memory");
static_assert(4 * kF8GatherWarps % 8 == 0, "a gather warp's rows share their swizzle");
static_assert(f8_own_at(true, 3, 0) + 3 * kF8Block <= kF8OffQpe && f8_own_at(false, 2, 0) + 2 * kF8Block <= kF8OffQpe, "blocks");

struct F8Bars {
  uint64_t q_tma;         // the query's boxes landed
  uint64_t q_full;        // 8 softmax warps: the query's limbs are in TMEM
  uint64_t ring_full[2];  // the gather lanes, once a block: the tile's ring blocks have landed
  uint64_t ring_empty[3]; // MMA commit: QK has read it
  uint64_t own_full[3];   // the same of its stage
  uint64_t own_empty[3];  // MMA commit: PV has read the stage
  uint64_t tile_full[4];  // a tile's positions and scales
  uint64_t tile_done[4];  // MMA commit: its PV is done
  uint64_t s_full;        // MMA commit: scores ready
  uint64_t s_empty;       // 8 softmax warps: scores read
  uint64_t p_own[2];      // 8 softmax warps: the CTA's part of P written
  uint64_t o_ready[2];    // the same: O rescaled
  uint64_t p_hi[2], p_lo[2];  // pair: one arming arrival and the peer's limb
  uint64_t moves[2];      // pair: one arming arrival and the peer's F8Move
  uint64_t hi_free;       // pair: MMA commit of both CTAs' PV of the hi limbs
  uint64_t p_free[2];     // MMA commit of the CTA's (pair: and the peer's) PV: P free, pushes gone, O stable
  uint64_t fin_full;      // pair: one arming arrival and the peer's half of fin
  uint64_t drained[2];    // the MMAs of an aborted kernel
  uint32_t tmem_addr;
  int abort_flag;
  int selected;           // 0: the split has no valid position
};
static_assert(sizeof(F8Bars) <= 512, "barrier block");

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <bool kPair>
__global__ void __launch_bounds__(kF8Threads, 1)
sparse_attend_fp8_kernel(const __grid_constant__ CUtensorMap tm_q, const uint8_t* q_exp, int n_rows,
                         const __nv_bfloat16* __restrict__ q_pe,
                         const uint8_t* __restrict__ kv8, const __nv_bfloat16* __restrict__ pe8,
                         const float* __restrict__ kv_scale, int block_shift, int n_blocks,
                         const int32_t* __restrict__ end_pos, const int32_t* __restrict__ topk_idx, float scale,
                         __nv_bfloat16* __restrict__ o_part, float* __restrict__ lse_part, int K, int S_max,
                         int n_split, int span, const __nv_bfloat16* __restrict__ w_next,
                         const int32_t* __restrict__ cache_slot, int n_slots, int n_heads, int* d_status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  constexpr int kRing = f8_ring(kPair), kRingPer = f8_ring_per(kPair), kOwn = f8_own(kPair);
  constexpr int kStages = f8_stages(kPair);
  constexpr int kCols = kPair ? kH : kF8Heads;  // heads of O and P
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u, peer = rank ^ 1u;
  const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int b = unit / n_split, split = unit % n_split;
  const int k_begin = split * span, k_end = min(K, k_begin + span);
  const int n_tiles = (k_end - k_begin + kF8Nt - 1) / kF8Nt;
  const int h0 = (int)rank * kF8Heads;
  const int live = min(kF8Heads, n_heads - h0);
  // the CTA's own latent columns are 128 (kOwn rank + i).., the peer's follow them
  auto lat = [&](int i) -> int { return ((int)(kOwn * rank) + i) & 3; };
  int ep = end_pos[b];
  ep = ep < 0 ? 0 : (ep > S_max ? S_max : ep);
  int slot = b;
  if (cache_slot != nullptr) {
    slot = cache_slot[b];
    if (slot < 0 || slot >= n_slots) slot = 0, ep = 0;  // such a row has no valid position
  }

  const uint32_t s0 = smem_u32(smem);
  float* key = reinterpret_cast<float*>(smem + kF8OffKey);      // [tile & 3][s | log2 s | 1/s][128]
  float* red = reinterpret_cast<float*>(smem + kF8OffRed);      // tops, then sums: [tile & 1][position half][head]
  int* pos_s = reinterpret_cast<int*>(smem + kF8OffPos);        // [tile & 3][128]
  F8Move* moves = reinterpret_cast<F8Move*>(smem + kF8OffMove);  // [tile & 1][rank]
  float* fin = reinterpret_cast<float*>(smem + kF8OffFin);
  F8Bars* bars = reinterpret_cast<F8Bars*>(smem + kF8OffBar);
  const AbortState ab{&bars->abort_flag, d_status};

  if (warp == kF8QkWarp) {
    // (the lanes share the barriers: one thread took a microsecond)
    if (lane == 0) {
      bars->abort_flag = 0;
      bars->selected = 1;
      mbar_init(smem_u32(&bars->q_tma), 1);
      mbar_init(smem_u32(&bars->q_full), kF8SoftmaxWarps);
      mbar_init(smem_u32(&bars->s_full), 1);
      mbar_init(smem_u32(&bars->s_empty), kF8SoftmaxWarps);
      mbar_init(smem_u32(&bars->hi_free), 2);
      mbar_init(smem_u32(&bars->fin_full), 1);
      if (kPair) mbar_arrive_expect_tx(smem_u32(&bars->fin_full), kF8Heads * 4);
    } else if (lane < 3) {
      const int s = lane - 1;
      mbar_init(smem_u32(&bars->ring_full[s]), 32 * kF8GatherWarps * kRingPer);
      mbar_init(smem_u32(&bars->drained[s]), 1);
      mbar_init(smem_u32(&bars->p_own[s]), kF8SoftmaxWarps);
      mbar_init(smem_u32(&bars->o_ready[s]), kF8SoftmaxWarps);
      mbar_init(smem_u32(&bars->p_free[s]), kPair ? 2 : 1);
    } else if (lane < 5) {
      const int s = lane - 3;
      mbar_init(smem_u32(&bars->p_hi[s]), 1);
      mbar_init(smem_u32(&bars->p_lo[s]), 1);
      mbar_init(smem_u32(&bars->moves[s]), 1);
      if (kPair) {  // armed for the first tiles
        mbar_arrive_expect_tx(smem_u32(&bars->p_hi[s]), kF8Limb);
        mbar_arrive_expect_tx(smem_u32(&bars->p_lo[s]), kF8Limb);
        mbar_arrive_expect_tx(smem_u32(&bars->moves[s]), sizeof(F8Move));
      }
    } else if (lane < 9) {
      const int s = lane - 5;
      mbar_init(smem_u32(&bars->tile_full[s]), 1);
      mbar_init(smem_u32(&bars->tile_done[s]), 1);
      if (s < kRing) mbar_init(smem_u32(&bars->ring_empty[s]), 1);
      if (s < kStages) {
        mbar_init(smem_u32(&bars->own_full[s]), 32 * kF8GatherWarps * kOwn);
        mbar_init(smem_u32(&bars->own_empty[s]), 1);
      }
    }
    fence_mbarrier_init_cluster();
    __syncwarp();
  }
  if (warp == kF8PvWarp) {
    tmem_alloc(smem_u32(&bars->tmem_addr), 512);
    tmem_relinquish();
  }
  if (tid < kH) fin[tid] = 0.f;
  tc_fence_before();
  if (kPair)
    cluster_sync();  // barriers of both CTAs initialised before any remote access
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_addr;
  grid_dep_launch();  // the value-up kernel may start loading its weights

  const int qd = warp & 3, ch = warp >> 2;  // softmax warps
  constexpr uint32_t kSoftmaxThreads = 32 * kF8SoftmaxWarps;

  const int32_t* idx_row = topk_idx + (size_t)b * K;
  const uint8_t* kv_row = kv8 + (size_t)slot * S_max * kDl;
  const uint8_t* pe_row = reinterpret_cast<const uint8_t*>(pe8 + (size_t)slot * S_max * kDr);

  if (warp == kF8IndexWarp) {
    // ------------------------------------------------------------ positions
    // Up to four tiles ahead of PV: the tile's positions, what their scales
    // enter by (a masked position weighs exactly 0), and the L2 prefetch of the
    // next tile's rows (a pair's CTAs take half of them each).  The loads for
    // the tiles after that are in flight meanwhile.
    const float* sc_row = kv_scale + (size_t)slot * n_blocks;
    struct Four {
      int pos[4];
    };
    auto load = [&](int j) -> Four {  // positions 32 i + lane of tile j
      Four f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k_begin + j * kF8Nt + 32 * i + lane;
        const int v = k < k_end ? __ldg(idx_row + k) : -1;
        f.pos[i] = (v >= 0 && v < ep) ? v : -1;
      }
      return f;
    };
    auto prefetch = [&](const Four& f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (f.pos[i] < 0 || (kPair && (i >> 1) != (int)rank)) continue;
        const uint8_t* r = kv_row + (size_t)f.pos[i] * kDl;
#pragma unroll
        for (int u = 0; u < 4; ++u) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + u * 128));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(pe_row + (size_t)f.pos[i] * (kDr * 2)));
      }
    };
    Four cur = load(0), next = load(1);
    float sv[4], sv_next[4];
    int selected = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = cur.pos[i] >= 0 ? __ldg(sc_row + (cur.pos[i] >> block_shift)) : 0.f;
    for (int j = 0; j < n_tiles; ++j) {
      const Four next2 = load(j + 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) sv_next[i] = next.pos[i] >= 0 ? __ldg(sc_row + (next.pos[i] >> block_shift)) : 0.f;
      if (j >= 4) wait(smem_u32(&bars->tile_done[j & 3]), ((j >> 2) - 1) & 1, ab);
      float* kt = key + (j & 3) * (3 * kF8Nt);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * i + lane;
        const bool on = !(sv[i] <= 0.f);
        pos_s[(j & 3) * kF8Nt + n] = cur.pos[i];
        selected |= cur.pos[i] >= 0;
        kt[n] = sv[i];
        kt[kF8Nt + n] = on ? __log2f(sv[i]) : -INFINITY;
        kt[2 * kF8Nt + n] = on ? __frcp_rn(sv[i]) : 0.f;
      }
      if (j == n_tiles - 1 && !__any_sync(0xffffffffu, selected)) bars->selected = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->tile_full[j & 3]));
      prefetch(next);
      cur = next;
      next = next2;
#pragma unroll
      for (int i = 0; i < 4; ++i) sv[i] = sv_next[i];
    }
    // One head's W_UV into L2 for the value-up kernel that follows.
    if (lane == 0 && w_next != nullptr && (int)blockIdx.x < n_heads) {
      const __nv_bfloat16* w = w_next + (size_t)(blockIdx.x * kHeadRows + kDn) * kDl;
#pragma unroll
      for (int part = 0; part < 4; ++part) prefetch_l2(w + part * 32 * kDl, 32 * kDl * 2);
    }
  } else if (warp >= kF8GatherWarp && warp < kF8GatherWarp + kF8GatherWarps) {
    // ------------------------------------------------------------ gather
    // A copy instruction brings 128 bytes of four positions; the warps
    // share a block's 32 of them, each with its positions in registers for all
    // five blocks (read for each copy, the copies issued at half the rate).
    // Nothing here waits for a copy: the barriers complete when the data lands
    // (with warps that wait for it and report it, 56.4 us instead of 53.3 at 64
    // rows of 2048: a report needs a proxy fence, and waits behind the issue).
    const int g = warp - kF8GatherWarp;
    constexpr int kCopies = 32 / kF8GatherWarps;
    int rs = 0, st = 0;          // ring slot, stage
    uint32_t rph = 1, sph = 1;   // parity of the release to wait for (passes at once the first time round)
    const uint32_t dst0 = s0 + sw128_offset(4 * g + (lane >> 3), lane & 7);
    for (int j = 0; j < n_tiles; ++j) {
      int pos[kCopies];
      const bool known = wait(smem_u32(&bars->tile_full[j & 3]), (j >> 2) & 1, ab);  // else timed out: nothing is read
#pragma unroll
      for (int i = 0; i < kCopies; ++i) pos[i] = known ? pos_s[(j & 3) * kF8Nt + 4 * (g + kF8GatherWarps * i) + (lane >> 3)] : -1;
      // the rotary rows, then 128 columns at a time: the peer's, the CTA's own
      // (one body for all: the warps of an SM fetch more code than its
      // instruction cache likes)
#pragma unroll 1
      for (int i = 0; i < 5; ++i) {
        const bool ring = i < kRingPer;
        uint32_t dst;
        uint64_t* full;
        if (ring) {
          wait(smem_u32(&bars->ring_empty[rs]), rph, ab);
          full = &bars->ring_full[j & 1];
          dst = dst0 + rs * kF8Block;
          if (++rs == kRing) rs = 0, rph ^= 1;
        } else {
          if (i == kRingPer) {
            // the query's boxes lie in the stages behind the first until they are in TMEM
            if (j == 1) wait(smem_u32(&bars->q_full), 0, ab);
            wait(smem_u32(&bars->own_empty[st]), sph, ab);
          }
          full = &bars->own_full[st];
          dst = dst0 + f8_own_at(kPair, 0, 0) + (st * kOwn + i - kRingPer) * kF8Block;
        }
        const uint8_t* src = (i == 0 ? pe_row : kv_row + lat(ring ? kOwn + i - 1 : i - kRingPer) * 128) + (lane & 7) * 16;
        const uint32_t row_bytes = i == 0 ? kDr * 2 : kDl;
#pragma unroll
        for (int u = 0; u < kCopies; ++u) {
          cp_async_16(dst + u * (4 * kF8GatherWarps * 128), src + (uint64_t)max(pos[u], 0) * row_bytes, pos[u] >= 0 ? 16u : 0u);
        }
        cp_async_arrive(smem_u32(full));
      }
      if (++st == kStages) st = 0, sph ^= 1;
    }
  } else if (warp == kF8QkWarp) {
    // ------------------------------------------------ query load, QK issue
    if (lane == 0) {
      // eight boxes of 64 columns x 64 heads (heads past the call's read as zero)
      tma_prefetch_desc(&tm_q);
      grid_dep_wait();  // q_lat comes from the absorption kernel
      mbar_arrive_expect_tx(smem_u32(&bars->q_tma), kF8Heads * kDl * 2);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        tma_load_3d(s0 + f8_own_at(kPair, 1, 0) + i * (kF8Heads * 128), &tm_q, smem_u32(&bars->q_tma), i * 64, h0, b);

      constexpr uint32_t id_pe = idesc_bf16_f32(128, kF8Nt, false, false);
      constexpr uint32_t id_qk = idesc_e4m3_f32(128, kF8Nt, false, false);
      const uint64_t d_0 = smem_desc_sw128(s0, 16, 1024);
      const uint64_t d_qpe = smem_desc_sw128(s0 + kF8OffQpe, 16, 1024);
      const uint32_t dst = tmem + kF8ColS, q = tmem + kF8ColQ;
      auto qk = [&](uint64_t k0, int block) {  // 128 columns of the latent
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8_ts(dst, q + block * 32 + k * 8, k0 + (uint64_t)(k * 2), id_qk, 1u);
      };
      wait(smem_u32(&bars->q_full), 0, ab);
      int rs = 0, st = 0;
      uint32_t sph = 0;
      for (int j = 0; j < n_tiles; ++j) {
        // One wait and one proxy fence for the ring blocks and one for the
        // stage: a pair of them costs as much as a block's four MMAs.
        wait(smem_u32(&bars->ring_full[j & 1]), (j >> 1) & 1, ab);
        fence_proxy_async_smem();
        if (j >= 1) wait(smem_u32(&bars->s_empty), (j - 1) & 1, ab);
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < kRingPer; ++i) {
          const uint64_t k0 = d_0 + (uint64_t)((rs * kF8Block) >> 4);
          if (i == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(dst, d_qpe + (uint64_t)(k * 2), k0 + (uint64_t)(k * 2), id_pe, k > 0 ? 1u : 0u);
          } else {
            qk(k0, lat(kOwn + i - 1));
          }
          mma_commit(smem_u32(&bars->ring_empty[rs]));
          if (++rs == kRing) rs = 0;
        }
        wait(smem_u32(&bars->own_full[st]), sph, ab);
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < kOwn; ++i)
          qk(d_0 + (uint64_t)((f8_own_at(kPair, 0, 0) + (st * kOwn + i) * kF8Block) >> 4), lat(i));
        if (++st == kStages) st = 0, sph ^= 1;
        mma_commit(smem_u32(&bars->s_full));
      }
      if (*ab.flag) drain_mmas(smem_u32(&bars->drained[0]));
    }
    __syncwarp();
  } else if (warp == kF8PushWarp) {
    // ------------------------------------------------ pushes
    if (kPair && lane == 0) {
      for (int j = 0; j < n_tiles; ++j) {
        const int pb = j & 1;
        if (!wait(smem_u32(&bars->p_own[pb]), (j >> 1) & 1, ab)) break;
        // The peer's buffers are free: p_free and hi_free, which the softmax
        // warps waited for, count its PVs too.
        const uint32_t hi = s0 + f8_p_at(true, j, 0) + rank * kF8Limb, lo = s0 + f8_p_at(true, j, 1) + rank * kF8Limb;
        bulk_push(cluster_map(hi, peer), hi, kF8Limb, cluster_map(smem_u32(&bars->p_hi[pb]), peer));
        bulk_push(cluster_map(lo, peer), lo, kF8Limb, cluster_map(smem_u32(&bars->p_lo[pb]), peer));
      }
    }
    __syncwarp();
  } else if (warp == kF8PvWarp) {
    // ------------------------------------------------ PV issue
    if (lane == 0) {
      constexpr uint32_t id_hi = idesc_e4m3_f32(128, kCols, true, false), id_lo = id_hi | kIdescBE5m2;
      const uint64_t d_0 = smem_desc_sw128(s0, 16, 1024);
      int st = 0;
      for (int j = 0; j < n_tiles; ++j) {
        const int pb = j & 1;
        const uint32_t ph = (j >> 1) & 1;
        wait(smem_u32(&bars->o_ready[pb]), ph, ab);  // P is written before that
        if (kPair) {
          if (wait_cluster(smem_u32(&bars->p_hi[pb]), ph, ab) && j + 2 < n_tiles)
            mbar_arrive_expect_tx(smem_u32(&bars->p_hi[pb]), kF8Limb);
        }
        tc_fence_after();
        // 128 latent columns x the heads, 32 positions a step, hi limbs and
        // lo limbs.  Pair: all hi limbs first, the peer's lo limbs are still
        // on their way.
        const uint64_t v0 = d_0 + (uint64_t)((f8_own_at(kPair, 0, 0) + st * (kOwn * kF8Block)) >> 4);
        const uint64_t p_hi = d_0 + (uint64_t)(f8_p_at(kPair, j, 0) >> 4), p_lo = d_0 + (uint64_t)(f8_p_at(kPair, j, 1) >> 4);
        auto pv = [&](int m, int k, uint64_t p, uint32_t id, bool first) {
          mma_f8_ss(tmem + kF8ColO + m * kCols, v0 + (uint64_t)((m * kF8Block + k * 32 * 128) >> 4), p + (uint64_t)((k * 32) >> 4),
                    id, first ? 0u : 1u);
        };
        if (kPair) {
#pragma unroll 1
          for (int m = 0; m < kOwn; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) pv(m, k, p_hi, id_hi, j == 0 && k == 0);
          mma_commit_to(smem_u32(&bars->hi_free), (uint16_t)3);
          if (wait_cluster(smem_u32(&bars->p_lo[pb]), ph, ab) && j + 2 < n_tiles)
            mbar_arrive_expect_tx(smem_u32(&bars->p_lo[pb]), kF8Limb);
        }
#pragma unroll 1
        for (int m = 0; m < kOwn; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (!kPair) pv(m, k, p_hi, id_hi, j == 0 && k == 0);
            pv(m, k, p_lo, id_lo, false);
          }
        mma_commit(smem_u32(&bars->own_empty[st]));
        mma_commit(smem_u32(&bars->tile_done[j & 3]));
        if (kPair)
          mma_commit_to(smem_u32(&bars->p_free[pb]), (uint16_t)3);
        else
          mma_commit(smem_u32(&bars->p_free[pb]));
        if (++st == kStages) st = 0;
      }
      if (*ab.flag) drain_mmas(smem_u32(&bars->drained[1]));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int hd = 16 * qd + (lane & 15);  // head; lanes 0..15 hold its hi row, 16..31 its lo row
    const bool hi_row = lane < 16;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;

    // The query's limbs.  One power of two for the CTA's 64 heads: a softmax
    // feels the absolute error of a score, and a head of small queries gets
    // the same absolute error as the largest one.  A thread takes 256 columns
    // of its row (both rows of a head read the same values).
    float c2;  // scores to log2 units
    bool bad;
    {
      const uint32_t box = s0 + f8_own_at(kPair, 1, 0) + (uint32_t)(4 * ch) * (kF8Heads * 128) + (uint32_t)hd * 128u;
      auto piece = [&](int c) {  // eight of the 256 columns
        return ld_shared_v4(box + (uint32_t)(c >> 3) * (kF8Heads * 128) + (uint32_t)(((c & 7) ^ (hd & 7)) << 4));
      };
      // the rotary part's row, from memory
      uint4 r4[4];
      const uint4* psrc = reinterpret_cast<const uint4*>(q_pe + ((size_t)b * n_heads + h0 + hd) * kDr) + 4 * ch;
#pragma unroll
      for (int u = 0; u < 4; ++u) r4[u] = hd < live ? __ldg(psrc + u) : make_uint4(0, 0, 0, 0);

      // scaled (fp16): the exponents of the thread's two times 128 columns
      const bool scaled = q_exp != nullptr;
      int ex[2] = {0, 0};
      if (scaled) {
        grid_dep_wait();
        if (hd < live) {
#pragma unroll
          for (int i = 0; i < 2; ++i) ex[i] = 127 - (int)__ldcg(q_exp + (size_t)((h0 + hd) * 4 + 2 * ch + i) * n_rows + b);
        }
      }

      const float rtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rotary_top(r4))));

      wait(smem_u32(&bars->q_tma), 0, ab);
      float top = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t m2 = 0;
#pragma unroll
        for (int c = 8 * i; c < 8 * i + 8; ++c) {  // the two rows of a head share its columns
          const uint4 v = piece(2 * c + (hi_row ? 0 : 1));
          m2 = amax2(amax2(amax2(amax2(m2, v.x), v.y), v.z), v.w);
        }
        const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
        finite &= m < (scaled ? 0x7c00u : 0x7f80u);
        top = fmaxf(top, scaled ? __half2float(__ushort_as_half((unsigned short)m)) * exp2_int(ex[i]) : __uint_as_float(m << 16));
      }
      if (!finite) {  // an infinity or NaN: the head's scores are NaN, the others' scale is not its
        fin[hd] = 1.f;
        top = 0.f;
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      if (lane == 0) red[warp] = top, red[kF8SoftmaxWarps + warp] = rtop;
      named_bar_sync(1, kSoftmaxThreads);
      bad = fin[hd] != 0.f;
      float am = red[0], rm = red[kF8SoftmaxWarps];
#pragma unroll
      for (int w = 1; w < kF8SoftmaxWarps; ++w) am = fmaxf(am, red[w]), rm = fmaxf(rm, red[kF8SoftmaxWarps + w]);
      const int e = query_exponent(am, rm);
      const float mul = exp2_int(e);
      c2 = scale * 1.4426950408889634f * exp2_int(-e);
      // The rotary factors in both rows of a head, half in each (S_lo counts a
      // 16th): a zero would turn a key's infinity into NaN.
      const float mul_r = hi_row ? 0.5f * mul : (0.5f / kLimbLo) * mul;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t w[4] = {r4[u].x, r4[u].y, r4[u].z, r4[u].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // times a power of two: exact
          o[i] = pack_bf16x2(__uint_as_float(w[i] << 16) * mul_r, __uint_as_float(w[i] & 0xffff0000u) * mul_r);
        st_shared_v4(s0 + kF8OffQpe + sw128_offset(32 * qd + lane, 4 * ch + u), o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      // 64 columns at a time: of two pieces of eight, each row of the head
      // converts one.  The loads go first, so that their latency is met once.
#pragma unroll 1
      for (int c4 = 0; c4 < 4; ++c4) {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = piece(8 * c4 + 2 * q + (hi_row ? 0 : 1));
        // as fp16 numbers 2^(e - 8) x
        if (scaled) {
          auto times = [&](int x) {
            const __half2 to = half2_power(x);
            auto one = [&](uint32_t h) { return half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&h), to)); };
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = make_uint4(one(v[q].x), one(v[q].y), one(v[q].z), one(v[q].w));
          };
          const int x = (c4 < 2 ? ex[0] : ex[1]) + e - 8, x1 = min(max(x, -14), 15);
          times(x1);
          if (__any_sync(0xffffffffu, x != x1)) times(x - x1);  // a chunk far from its bound, or from the largest
        } else {
          const float to = mul * (1.f / 256.f);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = make_uint4(half2_of_bf16(v[q].x, to), half2_of_bf16(v[q].y, to), half2_of_bf16(v[q].z, to),
                              half2_of_bf16(v[q].w, to));
        }
        uint32_t keep[8], send[8], r[16];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t hi, lo;
            limbs4_half(u ? v[q].z : v[q].x, u ? v[q].w : v[q].y, 1.f / kLimbLo, &hi, &lo);
            keep[2 * q + u] = hi_row ? hi : lo;
            send[2 * q + u] = hi_row ? lo : hi;
          }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, send[2 * q + u], 16);
            r[4 * q + u] = hi_row ? keep[2 * q + u] : other;
            r[4 * q + 2 + u] = hi_row ? other : keep[2 * q + u];
          }
        tmem_st16(tmem + lane_base + kF8ColQ + 64 * ch + 16 * c4, r);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
    }

    // Of the 64 positions of the warp, lanes 0..15 finish the first 32 and
    // lanes 16..31 the others: each sends its partner the other half.
    const int first = 64 * ch + (hi_row ? 0 : 32);
    if (bad) c2 = __int_as_float(0x7fffffff);
    const float w_k = hi_row ? c2 : c2 * kLimbLo, w_r = hi_row ? c2 * kLimbLo : c2;
    const uint64_t w_keep = pack_f32x2(w_k, w_k), w_recv = pack_f32x2(w_r, w_r);
    // l: the row sum; mass: the sum of P (fp16's range, which is enough to choose
    // m_h by); both of the thread's positions
    float m_ref = kF8NoRef, peak = -INFINITY, l = 0.f, mass = 0.f;
    if (hi_row) red[(4 + ch) * kF8Heads + hd] = 0.f;
    for (int j = 0; j < n_tiles; ++j) {
      const ulonglong2* kt = reinterpret_cast<const ulonglong2*>(key + (j & 3) * (3 * kF8Nt) + first);
      F8Move* mv = moves + 2 * (j & 1) + rank;  // tile j - 2's is done: its PVs are
      uint64_t y[16];  // pairs of positions
      wait(smem_u32(&bars->s_full), j & 1, ab);
      tc_fence_after();
      {
        uint32_t v[64];
        tmem_ld32(tmem + lane_base + kF8ColS + 64 * ch, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
        tmem_ld32(tmem + lane_base + kF8ColS + 64 * ch + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float keep[2], recv[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a = v[2 * i + u], c = v[32 + 2 * i + u];
            keep[u] = __uint_as_float(hi_row ? a : c);
            recv[u] = __shfl_xor_sync(0xffffffffu, __uint_as_float(hi_row ? c : a), 16);
          }
          y[i] = fma_f32x2(pack_f32x2(keep[0], keep[1]), w_keep, mul_f32x2(pack_f32x2(recv[0], recv[1]), w_recv));
        }
      }
      wait(smem_u32(&bars->tile_full[j & 3]), (j >> 2) & 1, ab);
      float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const ulonglong2 f = kt[q], g = kt[kF8Nt / 4 + q];
        y[2 * q] = fma_f32x2(y[2 * q], f.x, g.x);
        y[2 * q + 1] = fma_f32x2(y[2 * q + 1], f.y, g.y);
        const float2 a = unpack_f32x2(y[2 * q]), c = unpack_f32x2(y[2 * q + 1]);
        top4[q & 3] = fmaxf(fmaxf(top4[q & 3], fmaxf(a.x, a.y)), fmaxf(c.x, c.y));
      }
      float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      // the head's other 64 positions (two buffers: a warp may run a tile ahead)
      float* rt = red + (j & 1) * (2 * kF8Heads);
      if (hi_row) rt[ch * kF8Heads + hd] = top;
      named_bar_sync(2 + qd, 64);
      top = fmaxf(top, rt[(ch ^ 1) * kF8Heads + hd]);
      const float sums = rt[4 * kF8Heads + hd] + rt[5 * kF8Heads + hd];

      peak = fmaxf(peak, top);
      const float at = fmaxf(top, peak - kF8RefFall);
      const bool fall = at - m_ref < kF8RefFloor && sums < kF8MassFloor * (float)(j + 1) && top > -INFINITY;
      const bool move = at - m_ref > kF8RefLimit || fall;
      const float now = move ? at + kF8RefMargin : m_ref;
      const float factor = move ? ex2_approx(m_ref - now) : 1.f;
      // nothing to rescale before the first PV
      const uint32_t moved = j > 0 ? __ballot_sync(0xffffffffu, move) & 0xffffu : 0u;
      if (ch == 0) {
        const uint32_t far = cluster_map(smem_u32(&bars->moves[j & 1]), peer);
        if (hi_row) {
          mv->factor[hd] = factor;
          if (kPair) st_async_b32(cluster_map(smem_u32(&mv->factor[hd]), peer), __float_as_uint(factor), far);
        }
        if (lane == 0) {
          mv->moved[qd] = moved;
          if (kPair) st_async_b32(cluster_map(smem_u32(&mv->moved[qd]), peer), moved, far);
        }
      }
      m_ref = now;
      l *= factor;
      mass *= factor;

      // P and its limbs, four positions a word.
      uint32_t p_hi[8], p_lo[8];
      uint64_t l2[2] = {0, 0};
      __half2 sum2 = __float2half2_rn(0.f);
      const uint64_t minus_m = pack_f32x2(-m_ref, -m_ref);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const ulonglong2 r = kt[2 * (kF8Nt / 4) + q];
        const float2 ya = unpack_f32x2(add_f32x2(y[2 * q], minus_m)), yc = unpack_f32x2(add_f32x2(y[2 * q + 1], minus_m));
        const float p0 = ex2_approx(ya.x), p1 = ex2_approx(ya.y), p2 = ex2_approx(yc.x), p3 = ex2_approx(yc.y);
        l2[0] = fma_f32x2(pack_f32x2(p0, p1), r.x, l2[0]);
        l2[1] = fma_f32x2(pack_f32x2(p2, p3), r.y, l2[1]);
        const uint32_t f01 = pack_f16x2_sat(p0, p1), f23 = pack_f16x2_sat(p2, p3);
        sum2 = __hadd2(sum2, __hadd2(*reinterpret_cast<const __half2*>(&f01), *reinterpret_cast<const __half2*>(&f23)));
        const uint32_t a01 = limb_first(f01), a23 = limb_first(f23);
        p_hi[q] = limb_bytes_positive(a01, a23);
        p_lo[q] = limb_bytes_e5m2(limb_rest(f01, a01), limb_rest(f23, a23));
      }
      const float2 l01 = unpack_f32x2(add_f32x2(l2[0], l2[1]));
      l += l01.x + l01.y;
      mass += __low2float(sum2) + __high2float(sum2);

      if (j >= 2) wait_cluster(smem_u32(&bars->p_free[j & 1]), ((j >> 1) - 1) & 1, ab);  // tile j - 2's lo limbs lay where the hi limbs go
      const uint32_t hi_at = s0 + f8_p_at(kPair, j, 0) + rank * kF8Limb, lo_at = s0 + f8_p_at(kPair, j, 1) + rank * kF8Limb;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        st_shared_v4(hi_at + sw128_offset(hd, (first >> 4) + u), p_hi[4 * u], p_hi[4 * u + 1], p_hi[4 * u + 2], p_hi[4 * u + 3]);
      // the lo limbs go where tile j - 1's hi limbs lay
      if (kPair && j >= 1) wait_cluster(smem_u32(&bars->hi_free), (j - 1) & 1, ab);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        st_shared_v4(lo_at + sw128_offset(hd, (first >> 4) + u), p_lo[4 * u], p_lo[4 * u + 1], p_lo[4 * u + 2], p_lo[4 * u + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_own[j & 1]));
      // (for the next tile; the other warp has read the last one's)
      const float half = mass + __shfl_xor_sync(0xffffffffu, mass, 16);
      if (hi_row) red[((j & 1) ^ 1) * (2 * kF8Heads) + (4 + ch) * kF8Heads + hd] = half;

      // The heads of either CTA that moved: their columns of this CTA's O,
      // between PV(j - 1) and PV(j); 16 columns that hold none of them are left
      // alone.  The CTA's own words come from its other warps.
      if (kPair) {
        if (wait_cluster(smem_u32(&bars->moves[j & 1]), (j >> 1) & 1, ab) && tid == 0 && j + 2 < n_tiles)
          mbar_arrive_expect_tx(smem_u32(&bars->moves[j & 1]), sizeof(F8Move));
      }
      named_bar_sync(1, kSoftmaxThreads);
      if (j > 0) {
        const F8Move* both = moves + 2 * (j & 1);
        const uint4 w0 = *reinterpret_cast<const uint4*>(both[0].moved);
        const uint4 w1 = kPair ? *reinterpret_cast<const uint4*>(both[1].moved) : make_uint4(0, 0, 0, 0);
        if ((w0.x | w0.y | w0.z | w0.w | w1.x | w1.y | w1.z | w1.w) != 0) {
          wait_cluster(smem_u32(&bars->p_free[(j - 1) & 1]), ((j - 1) >> 1) & 1, ab);  // PV(j - 1) is done
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            const int col = (cc * 16) % kCols, h16 = col % kF8Heads;
            const F8Move* who = both + col / kF8Heads;
            if (who->moved[h16 >> 4] == 0) continue;
            const uint32_t at = tmem + lane_base + kF8ColO + 128 * ch + cc * 16;
            uint32_t ov[16];
            tmem_ld16(at, ov);
            tmem_wait_ld();
            const float4* f4 = reinterpret_cast<const float4*>(who->factor + h16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = f4[i];
              ov[4 * i] = __float_as_uint(__uint_as_float(ov[4 * i]) * f.x);
              ov[4 * i + 1] = __float_as_uint(__uint_as_float(ov[4 * i + 1]) * f.y);
              ov[4 * i + 2] = __float_as_uint(__uint_as_float(ov[4 * i + 2]) * f.z);
              ov[4 * i + 3] = __float_as_uint(__uint_as_float(ov[4 * i + 3]) * f.w);
            }
            tmem_st16(at, ov);
          }
          tmem_wait_st();
          tc_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->o_ready[j & 1]));
    }

    // The row sums over the positions; what normalises O goes to the peer too.
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    named_bar_sync(2 + qd, 64);  // both warps are past the last tile's exchange
    if (hi_row) red[ch * kF8Heads + hd] = l;
    named_bar_sync(2 + qd, 64);
    if (ch == 0 && hi_row) {
      const float sum = l + red[kF8Heads + hd];
      const float inv = sum == 0.f ? 0.f : (1.f / 256.f) / sum;  // P's E4M3 value is 2^8 times its fp16 one
      fin[h0 + hd] = inv;
      if (kPair)
        st_async_b32(cluster_map(smem_u32(&fin[h0 + hd]), peer), __float_as_uint(inv), cluster_map(smem_u32(&bars->fin_full), peer));
      float lse = (m_ref + log2f(sum)) * 0.6931471805599453f;
      if (sum == 0.f || !bars->selected) lse = -INFINITY;
      if (hd < live) lse_part[((size_t)b * n_split + split) * n_heads + h0 + hd] = lse;
    }
    // the last PV ends after all others
    wait_cluster(smem_u32(&bars->p_free[(n_tiles - 1) & 1]), ((n_tiles - 1) >> 1) & 1, ab);
    tc_fence_after();
  }

  // A CTA that gave up waiting leaves nothing on its way into its own or its
  // peer's memory.
  cp_async_wait_all();
  if (*ab.flag) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  if (kPair) cluster_arrive();  // from here on nothing of the peer's is touched

  if (warp < kF8SoftmaxWarps) {
    // O normalised: of two heads, an even lane takes the first and its
    // neighbour the second, two latent columns in one word.  A warp writes 64
    // bytes of each of two heads at a time.
    named_bar_sync(1, kSoftmaxThreads);
    if (kPair) wait_cluster(smem_u32(&bars->fin_full), 0, ab);
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    uint32_t* o_row = reinterpret_cast<uint32_t*>(o_part + ((size_t)b * n_split + split) * n_heads * kDl) + rank * 128 + 16 * qd + (lane >> 1);
    auto write = [&](int cc, const uint32_t (&ov)[32]) {
      const int c0 = 128 * ch + 32 * cc, m = c0 / kCols, hb = c0 % kCols + (lane & 1);
      const float4* f4 = reinterpret_cast<const float4*>(fin + c0 % kCols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = f4[i];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float x = __uint_as_float(ov[4 * i + 2 * u]) * (u ? f.z : f.x);
          const float y = __uint_as_float(ov[4 * i + 2 * u + 1]) * (u ? f.w : f.y);
          const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
          const uint32_t w = (lane & 1) ? pack_bf16x2(other, y) : pack_bf16x2(x, other);
          const int head = hb + 4 * i + 2 * u;
          if (head < n_heads) o_row[(uint32_t)head * (kDl / 2) + m * 64] = w;
        }
      }
    };
    const uint32_t o_at = tmem + lane_base + kF8ColO + 128 * ch;
    uint32_t oa[32], ob[32];
    tmem_ld32(o_at, oa);
#pragma unroll 1
    for (int cc = 0; cc < 4; cc += 2) {
      tmem_wait_ld();
      tmem_ld32(o_at + 32 * (cc + 1), ob);
      write(cc, oa);
      tmem_wait_ld();
      if (cc == 0) tmem_ld32(o_at + 64, oa);
      write(cc + 1, ob);
    }
    // A query that is not finite makes P NaN at masked positions too.  Beside
    // valid ones, whose P is NaN then, that changes nothing; without any, the
    // thread's words become zeros.  (Selected as they are written, 0.6 us a call.)
    if (!bars->selected) {
#pragma unroll 1
      for (int c = 128 * ch; c < 128 * ch + 128; c += 2) {
        const int head = c % kCols + (lane & 1);
        if (head < n_heads) o_row[(uint32_t)head * (kDl / 2) + c / kCols * 64] = 0u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kF8PvWarp) tmem_dealloc(tmem, 512);
  if (kPair) cluster_wait();  // the peer may still write to this CTA until then
}

}  // namespace mla
