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
// A factor kept as two E4M3 numbers has 8 significant bits, bf16's own count,
// and 8-bit products run at twice the rate of bf16 products: two of them cost
// what one bf16 product costs, and the codes go to the tensor cores as they
// lie in the cache, with no conversion and at half of bf16's shared memory.

// Two floats of magnitude <= 448 to their E4M3 pair (round to nearest even)
// and back.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

// Exponent e with |amax| 2^e in (224, 448] (0 for amax = 0).
__device__ __forceinline__ int limb_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int k;
  const float m = frexpf(amax, &k);          // amax = m 2^k, m in [1/2, 1)
  const int e = (m <= 0.875f ? 9 : 8) - k;   // 448 = 0.875 2^9
  return e < -100 ? -100 : (e > 100 ? 100 : e);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 126

// Eight bf16 numbers (one 16-byte load) times 2^e as limbs: x 2^e = hi + lo / 16.
// The second limb is scaled by 16 so that it keeps its bits however small x
// is.  An infinite or NaN x gives a NaN second limb.
constexpr float kLimbLo = 1.f / 16.f;
__device__ __forceinline__ void limbs8(const uint4& raw, float mul, uint2* hi, uint2* lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16) * mul, b = __uint_as_float(w[i] & 0xffff0000u) * mul;
    h[i] = pack_e4m3x2(a, b);
    const float2 r = unpack_e4m3x2(h[i]);
    l[i] = pack_e4m3x2(fmaf(a, 0.f, (a - r.x) * 16.f), fmaf(b, 0.f, (b - r.y) * 16.f));
  }
  *hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  *lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// The largest finite magnitude among eight bf16 numbers.
__device__ __forceinline__ float amax8(const uint4& raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
    if (a < 0x7f80u) m = max(m, a);
    if (b < 0x7f80u) m = max(m, b);
  }
  return __uint_as_float(m << 16);
}

// Thirty-two values of each lane, reduced over the lanes: lane i returns the
// result of value i (31 exchanges instead of 160).
template <typename Op>
__device__ __forceinline__ float reduce_transposed(float (&v)[32], int lane, Op op) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = up ? v[i + s] : v[i], send = up ? v[i] : v[i + s];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  return v[0];
}

// =============================================================================
// sparse_attend_fp8_kernel
//
// One CTA per (row, key split, group of 64 heads), no cluster: everything is
// transposed, positions on the MMA's 128 rows, so that 64 heads and all 512
// latent columns fit one SM's tensor memory and no score crosses SMs:
//   S^T[t, h] = code_t . q_h      M = 128 positions, N = 64 hi + 64 lo limbs
//                                 of the query (E4M3, K-major both), plus the
//                                 bf16 rotary product into the hi columns;
//   O^T[c, h] += code_t[c] P[t, h]  M = 128 latent columns (four blocks),
//                                 N = 64, the tile's codes read M-major from
//                                 the same shared memory, P as two limbs.
// A softmax thread holds one position (TMEM lane) and 32 heads.  Its scale
// enters as two scalars: y = s_t scale (S_hi + S_lo / 16) + log2 s_t is the
// log2 weight of the position's *codes*, P = 2^(y - m_h), and the row sum adds
// P / s_t.  m_h is the largest y of some tile plus a margin; it moves only
// when P would leave E4M3's range (a vote among the CTA's softmax warps, one
// barrier a tile), and then O is rescaled in place.
//
// Shared memory: two 64 KB stages of 128 positions x 512 codes (four 128-byte
// swizzled blocks), the query's limbs (64 KB) and rotary part (8 KB), P
// (16 KB).  A tile's rotary rows borrow the stage's block 0: they are the
// first to be multiplied, and the codes of columns 0..127 follow them.
//
// Warps (448 threads): 0-7 softmax (warp w: positions 32 (w % 4).., heads
// 32 (w / 4)..), 8 QK issue, 9 TMEM and PV issue, 10-13 gather (32 positions
// of every tile each).
// =============================================================================
constexpr int kF8Heads = 64;                        // heads of a CTA
constexpr int kF8Nt = 128;                          // positions of a tile
constexpr int kF8Block = kF8Nt * 128;               // 128 codes of every position: 16 KB
constexpr int kF8StageBytes = 4 * kF8Block;
constexpr int kF8QBytes = 4 * 2 * kF8Heads * 128;   // per 128 columns: 64 hi rows, 64 lo rows
constexpr int kF8PBytes = kF8Nt * kF8Heads;         // one limb of P
constexpr int kF8QpeBytes = kF8Heads * 128;
constexpr int kF8OffQ = 2 * kF8StageBytes;
constexpr int kF8OffP = kF8OffQ + kF8QBytes;
constexpr int kF8OffQpe = kF8OffP + 2 * kF8PBytes;
constexpr int kF8OffScale = kF8OffQpe + kF8QpeBytes;         // f32 [2][128]: the positions' scales, 0 = masked
constexpr int kF8OffRed = kF8OffScale + 2 * kF8Nt * 4;       // f32 [4][64]
constexpr int kF8OffRef = kF8OffRed + 4 * kF8Heads * 4;      // f32 [64]: m_h
constexpr int kF8OffAlpha = kF8OffRef + kF8Heads * 4;        // f32 [64]
constexpr int kF8OffBar = kF8OffAlpha + kF8Heads * 4;
constexpr int kF8SmemBytes = kF8OffBar + 512 + kSmemAlignPad;
constexpr int kF8SoftmaxWarps = 8;
constexpr int kF8QkWarp = 8, kF8PvWarp = 9, kF8GatherWarp = 10, kF8GatherWarps = 4;
constexpr int kF8Threads = 32 * (kF8GatherWarp + kF8GatherWarps);
constexpr uint32_t kF8ColS = 0;    // two score buffers of 64 hi + 64 lo columns
constexpr uint32_t kF8ColO = 256;  // four blocks of 64 columns
// P is formed in fp16 at 2^-8 of its E4M3 value (fp16's exponent field is then
// E4M3's, so a limb is a byte of the fp16 number).  A new m_h puts the largest
// P of its tile at 2^-3 (2^5 in E4M3); a later one may reach 2^0.75 (430 in
// E4M3, of at most 448) before m_h has to move.
constexpr float kF8RefMargin = 3.0f;
constexpr float kF8RefLimit = 0.75f;
constexpr float kF8NoRef = -1e30f;  // m_h before any position counted
static_assert(kF8SmemBytes <= 232448, "shared memory");
static_assert(kF8OffQ % 1024 == 0 && kF8OffP % 1024 == 0 && kF8OffQpe % 1024 == 0, "swizzle atoms");
static_assert(kF8GatherWarps * 32 == kF8Nt, "a gather lane per position");

struct F8Bars {
  uint64_t q_full;       // 8 softmax warps: the query's limbs are in shared memory
  uint64_t full[2][5];   // 128 gather lanes: block i of the stage (4: the rotary rows) has landed
  uint64_t empty[2][4];  // MMA commit: PV has read block i
  uint64_t pe_done[2];   // MMA commit: the rotary product has read block 0
  uint64_t sc_full[2];   // 4 gather warps: the positions' scales
  uint64_t s_full[2];    // MMA commit: scores of the buffer
  uint64_t s_empty[2];   // 8 softmax warps: scores read
  uint64_t p_full;       // 8 softmax warps: P written
  uint64_t p_free;       // MMA commit: PV done (P free, O stable)
  uint32_t tmem_addr;
  int abort_flag;
};
static_assert(sizeof(F8Bars) <= 512, "barrier block");

__global__ void __launch_bounds__(kF8Threads, 1)
sparse_attend_fp8_kernel(const __nv_bfloat16* __restrict__ q_lat, const __nv_bfloat16* __restrict__ q_pe,
                         const uint8_t* __restrict__ kv8, const __nv_bfloat16* __restrict__ pe8,
                         const float* __restrict__ kv_scale, int block_shift, int n_blocks,
                         const int32_t* __restrict__ end_pos, const int32_t* __restrict__ topk_idx, float scale,
                         __nv_bfloat16* __restrict__ o_part, float* __restrict__ lse_part, int K, int S_max,
                         int n_split, int span, const __nv_bfloat16* __restrict__ w_next,
                         const int32_t* __restrict__ cache_slot, int n_slots, int n_heads, int n_groups,
                         int* d_status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x / n_groups;
  const int h0 = (blockIdx.x % n_groups) * kF8Heads;  // the groups of a row run side by side and share its rows in L2
  const int b = unit / n_split, split = unit % n_split;
  const int k_begin = split * span, k_end = min(K, k_begin + span);
  const int n_tiles = (k_end - k_begin + kF8Nt - 1) / kF8Nt;
  const int live = min(kF8Heads, n_heads - h0);
  int ep = end_pos[b];
  ep = ep < 0 ? 0 : (ep > S_max ? S_max : ep);
  int slot = b;
  if (cache_slot != nullptr) {
    slot = cache_slot[b];
    if (slot < 0 || slot >= n_slots) slot = 0, ep = 0;  // such a row has no valid position
  }

  const uint32_t s0 = smem_u32(smem);
  float* sc = reinterpret_cast<float*>(smem + kF8OffScale);
  float* red = reinterpret_cast<float*>(smem + kF8OffRed);
  float* mref = reinterpret_cast<float*>(smem + kF8OffRef);
  float* alpha = reinterpret_cast<float*>(smem + kF8OffAlpha);
  F8Bars* bars = reinterpret_cast<F8Bars*>(smem + kF8OffBar);
  const AbortState ab{&bars->abort_flag, d_status};

  if (tid == 0) {
    bars->abort_flag = 0;
    mbar_init(smem_u32(&bars->q_full), kF8SoftmaxWarps);
    for (int s = 0; s < 2; ++s) {
      for (int i = 0; i < 5; ++i) mbar_init(smem_u32(&bars->full[s][i]), kF8Nt);
      for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->empty[s][i]), 1);
      mbar_init(smem_u32(&bars->pe_done[s]), 1);
      mbar_init(smem_u32(&bars->sc_full[s]), kF8GatherWarps);
      mbar_init(smem_u32(&bars->s_full[s]), 1);
      mbar_init(smem_u32(&bars->s_empty[s]), kF8SoftmaxWarps);
    }
    mbar_init(smem_u32(&bars->p_full), kF8SoftmaxWarps);
    mbar_init(smem_u32(&bars->p_free), 1);
    fence_mbarrier_init_cluster();
  }
  if (warp == kF8PvWarp) {
    tmem_alloc(smem_u32(&bars->tmem_addr), 512);
    tmem_relinquish();
  }
  if (tid < kF8Heads) mref[tid] = kF8NoRef;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_addr;
  grid_dep_launch();  // the value-up kernel may start loading its weights

  if (warp >= kF8GatherWarp) {
    // ------------------------------------------------------------ gather
    // Lane l of warp g owns position 32 g + l of every tile: its index, its
    // scale, its L2 prefetch.  A copy instruction brings 128 bytes of four
    // positions.  Nothing here waits for a copy: the barriers complete when
    // the data lands.
    const int g = warp - kF8GatherWarp;
    const int32_t* idx_row = topk_idx + (size_t)b * K;
    const uint8_t* kv_row = kv8 + (size_t)slot * S_max * kDl;
    const uint8_t* pe_row = reinterpret_cast<const uint8_t*>(pe8 + (size_t)slot * S_max * kDr);
    const float* sc_row = kv_scale + (size_t)slot * n_blocks;
    auto load_idx = [&](int j) -> int {
      const int k = k_begin + j * kF8Nt + 32 * g + lane;
      const int v = k < k_end ? __ldg(idx_row + k) : -1;
      return (v >= 0 && v < ep) ? v : -1;
    };
    auto load_scale = [&](int pos) -> float { return pos >= 0 ? __ldg(sc_row + (pos >> block_shift)) : 0.f; };
    auto prefetch = [&](int pos) {
      if (pos >= 0) {
        const uint8_t* r = kv_row + (size_t)pos * kDl;
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + i * 128));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(pe_row + (size_t)pos * (kDr * 2)));
      }
    };
    auto copy = [&](uint32_t dst, const uint8_t* base, int row_bytes, int idx) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        const int pos = __shfl_sync(0xffffffffu, idx, r);
        const size_t p = pos >= 0 ? (size_t)pos : 0;
        cp_async_16(dst + sw128_offset(32 * g + r, lane & 7), base + p * row_bytes + (lane & 7) * 16,
                    pos >= 0 ? 16u : 0u);
      }
    };
    int idx0 = load_idx(0), idx1 = load_idx(1);
    float sc0 = load_scale(idx0);
    prefetch(idx1);
    for (int j = 0; j < n_tiles; ++j) {
      const int st = j & 1;
      const uint32_t ph = (j >> 1) & 1, was = ph ^ 1;
      const uint32_t stage = s0 + st * kF8StageBytes;
      const int idx2 = load_idx(j + 2);
      const float sc1 = load_scale(idx1);
      if (j >= 2) wait(smem_u32(&bars->empty[st][0]), was, ab);
      copy(stage, pe_row, kDr * 2, idx0);
      cp_async_arrive(smem_u32(&bars->full[st][4]));
      sc[st * kF8Nt + 32 * g + lane] = sc0;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->sc_full[st]));
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        if (j >= 2) wait(smem_u32(&bars->empty[st][i]), was, ab);
        copy(stage + i * kF8Block, kv_row + i * 128, kDl, idx0);
        cp_async_arrive(smem_u32(&bars->full[st][i]));
      }
      prefetch(idx2);
      wait(smem_u32(&bars->pe_done[st]), ph, ab);
      copy(stage, kv_row, kDl, idx0);
      cp_async_arrive(smem_u32(&bars->full[st][0]));
      idx0 = idx1;
      idx1 = idx2;
      sc0 = sc1;
    }
    // One head's W_UV into L2 for the value-up kernel that follows.
    if (g == 0 && lane == 0 && w_next != nullptr && (int)blockIdx.x < n_heads) {
      const __nv_bfloat16* w = w_next + (size_t)(blockIdx.x * kHeadRows + kDn) * kDl;
#pragma unroll
      for (int part = 0; part < 4; ++part) prefetch_l2(w + part * 32 * kDl, 32 * kDl * 2);
    }
  } else if (warp == kF8QkWarp) {
    // ------------------------------------------------------------ QK issue
    if (lane == 0) {
      constexpr uint32_t id_pe = idesc_bf16_f32(128, 64, false, false);
      constexpr uint32_t id_half = idesc_e4m3_f32(128, 64, false, false);
      constexpr uint32_t id_both = idesc_e4m3_f32(128, 128, false, false);
      const uint64_t d_stage = smem_desc_sw128(s0, 16, 1024);
      const uint64_t d_q = smem_desc_sw128(s0 + kF8OffQ, 16, 1024);
      const uint64_t d_qpe = smem_desc_sw128(s0 + kF8OffQpe, 16, 1024);
      wait(smem_u32(&bars->q_full), 0, ab);
      for (int j = 0; j < n_tiles; ++j) {
        const int st = j & 1;
        const uint32_t ph = (j >> 1) & 1;
        const uint64_t a0 = d_stage + (uint64_t)((st * kF8StageBytes) >> 4);
        const uint32_t dst = tmem + kF8ColS + st * 128;
        if (j >= 2) wait(smem_u32(&bars->s_empty[st]), ph ^ 1, ab);
        wait(smem_u32(&bars->full[st][4]), ph, ab);
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(dst, a0 + (uint64_t)(k * 2), d_qpe + (uint64_t)(k * 2), id_pe, k > 0 ? 1u : 0u);
        mma_commit(smem_u32(&bars->pe_done[st]));
#pragma unroll
        for (int o = 1; o <= 4; ++o) {
          const int i = o & 3;  // blocks 1, 2, 3, 0
          wait(smem_u32(&bars->full[st][i]), ph, ab);
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t a = a0 + (uint64_t)((i * kF8Block) >> 4);
          const uint64_t q = d_q + (uint64_t)((i * kF8Block) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (o == 1 && k == 0) {  // the hi columns hold the rotary product, the lo columns start at zero
              mma_f8_ss(dst, a, q, id_half, 1u);
              mma_f8_ss(dst + 64, a, q + (uint64_t)((kF8Heads * 128) >> 4), id_half, 0u);
            } else {
              mma_f8_ss(dst, a + (uint64_t)(k * 2), q + (uint64_t)(k * 2), id_both, 1u);
            }
          }
        }
        mma_commit(smem_u32(&bars->s_full[st]));
      }
    }
    __syncwarp();
  } else if (warp == kF8PvWarp) {
    // ------------------------------------------------------------ PV issue
    if (lane == 0) {
      constexpr uint32_t id_pv = idesc_e4m3_f32(128, 64, true, true);
      const uint64_t d_stage = smem_desc_sw128(s0, 16, 1024);
      const uint64_t d_p = smem_desc_sw64(s0 + kF8OffP, 512);
      for (int j = 0; j < n_tiles; ++j) {
        const int st = j & 1;
        wait(smem_u32(&bars->p_full), j & 1, ab);
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint64_t a = d_stage + (uint64_t)((st * kF8StageBytes + m * kF8Block) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 32 positions a step
            const uint64_t ak = a + (uint64_t)((k * 32 * 128) >> 4);
            const uint64_t pk = d_p + (uint64_t)((k * 32 * 64) >> 4);
            mma_f8_ss(tmem + kF8ColO + m * 64, ak, pk, id_pv, (j > 0 || k > 0) ? 1u : 0u);
            mma_f8_ss(tmem + kF8ColO + m * 64, ak, pk + (uint64_t)(kF8PBytes >> 4), id_pv, 1u);
          }
          mma_commit(smem_u32(&bars->empty[st][m]));
        }
        mma_commit(smem_u32(&bars->p_free));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int qd = warp & 3, hh = warp >> 2;
    const int row = 32 * qd + lane;  // position of the tile
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    constexpr uint32_t kAll = 32 * kF8SoftmaxWarps;
    auto fmax2 = [](float x, float y) { return fmaxf(x, y); };
    auto fadd2 = [](float x, float y) { return x + y; };

    // The query's limbs.  One power of two for the CTA's 64 heads: a softmax
    // feels the absolute error of a score, and a head of small queries gets
    // the same absolute error as the largest one.
    float c2;  // scores to log2 units
    {
      grid_dep_wait();  // q_lat comes from the absorption kernel
      const uint4* src = reinterpret_cast<const uint4*>(q_lat + ((size_t)b * n_heads + h0) * kDl);
      uint4 v[16];
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = i * (int)kAll + tid;  // 16-byte piece c of the 64 x 64
        v[i] = (c >> 6) < live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        am = fmaxf(am, amax8(v[i]));
      }
#pragma unroll
      for (int s = 16; s >= 1; s >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, s));
      if (lane == 0) red[warp] = am;
      named_bar_sync(1, kAll);
#pragma unroll
      for (int w = 0; w < kF8SoftmaxWarps; ++w) am = fmaxf(am, red[w]);
      const int e = limb_exponent(am);
      const float mul = exp2_int(e);
      c2 = scale * 1.4426950408889634f * exp2_int(-e);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = i * (int)kAll + tid, hd = c >> 6, piece = c & 63;
        uint2 hi, lo;
        limbs8(v[i], mul, &hi, &lo);
        const uint32_t dst = s0 + kF8OffQ + (piece >> 4) * kF8Block + sw128_offset(hd, (piece & 15) >> 1) + (piece & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(hi.x), "r"(hi.y) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst + kF8Heads * 128), "r"(lo.x), "r"(lo.y) : "memory");
      }
      const uint4* psrc = reinterpret_cast<const uint4*>(q_pe + ((size_t)b * n_heads + h0) * kDr);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = i * (int)kAll + tid, hd = c >> 3;
        const uint4 r = hd < live ? __ldg(psrc + c) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        uint32_t o[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)  // times a power of two: exact
          o[u] = pack_bf16x2(__uint_as_float(w[u] << 16) * mul, __uint_as_float(w[u] & 0xffff0000u) * mul);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(s0 + kF8OffQpe + sw128_offset(hd, c & 7)),
                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
    }

    const float4* mref4 = reinterpret_cast<const float4*>(mref + 32 * hh);
    const float4* alpha4 = reinterpret_cast<const float4*>(alpha + 32 * hh);
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;

    for (int j = 0; j < n_tiles; ++j) {
      const int st = j & 1;
      const uint32_t ph = (j >> 1) & 1;
      wait(smem_u32(&bars->sc_full[st]), ph, ab);
      const float s_t = sc[st * kF8Nt + row];
      const bool on = s_t > 0.f;
      const float f = s_t * c2;
      const float lg = on ? __log2f(s_t) : -INFINITY;
      const float rs = on ? __frcp_rn(s_t) : 0.f;
      wait(smem_u32(&bars->s_full[st]), ph, ab);
      tc_fence_after();
      float y[32];
      {
        uint32_t hi[32], lo[32];
        tmem_ld32(tmem + lane_base + kF8ColS + st * 128 + 32 * hh, hi);
        tmem_ld32(tmem + lane_base + kF8ColS + st * 128 + 64 + 32 * hh, lo);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          y[i] = fmaf(fmaf(__uint_as_float(lo[i]), kLimbLo, __uint_as_float(hi[i])), f, lg);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty[st]));

      float top = -INFINITY;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 m = mref4[q];
        top = fmaxf(top, fmaxf(fmaxf(y[4 * q] - m.x, y[4 * q + 1] - m.y), fmaxf(y[4 * q + 2] - m.z, y[4 * q + 3] - m.w)));
      }
      if (named_bar_or(1, kAll, top > kF8RefLimit)) {
        // Some P leaves E4M3's range: the tile's largest y of every head, the
        // new m_h of the heads it asks for, and O and the sums brought to it.
        float t[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) t[i] = y[i];
        red[qd * kF8Heads + 32 * hh + lane] = reduce_transposed(t, lane, fmax2);
        named_bar_sync(1, kAll);
        if (tid < kF8Heads) {
          const float mx = fmaxf(fmaxf(red[tid], red[kF8Heads + tid]), fmaxf(red[2 * kF8Heads + tid], red[3 * kF8Heads + tid]));
          const float old = mref[tid];
          const float now = mx - old > kF8RefLimit ? mx + kF8RefMargin : old;
          alpha[tid] = ex2_approx(old - now);
          mref[tid] = now;
        }
        named_bar_sync(1, kAll);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 a = alpha4[q];
          l[4 * q] *= a.x, l[4 * q + 1] *= a.y, l[4 * q + 2] *= a.z, l[4 * q + 3] *= a.w;
        }
        if (j > 0) {
          wait(smem_u32(&bars->p_free), (j - 1) & 1, ab);  // every PV issued so far is done
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            const uint32_t at = tmem + lane_base + kF8ColO + 128 * hh + cc * 16;
            uint32_t ov[16];
            tmem_ld16(at, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha[(cc & 3) * 16 + i]);
            tmem_st16(at, ov);
          }
          tmem_wait_st();
        }
      }

      // P and its limbs, four heads a word: the hi limb is the fp16 number
      // truncated to E4M3's bits, the lo limb what that left, rounded.
      uint32_t ph4[8], pl4[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 m = mref4[q];
        const float p0 = ex2_approx(y[4 * q] - m.x), p1 = ex2_approx(y[4 * q + 1] - m.y);
        const float p2 = ex2_approx(y[4 * q + 2] - m.z), p3 = ex2_approx(y[4 * q + 3] - m.w);
        l[4 * q] = fmaf(p0, rs, l[4 * q]);
        l[4 * q + 1] = fmaf(p1, rs, l[4 * q + 1]);
        l[4 * q + 2] = fmaf(p2, rs, l[4 * q + 2]);
        l[4 * q + 3] = fmaf(p3, rs, l[4 * q + 3]);
        uint32_t h[2], r[2];
        h[0] = pack_f16x2_sat(p0, p1);
        h[1] = pack_f16x2_sat(p2, p3);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t cut = h[u] & 0x3f803f80u;
          __half2 a, c;
          memcpy(&a, &h[u], 4);
          memcpy(&c, &cut, 4);
          const __half2 d = __hsub2(a, c);
          memcpy(&r[u], &d, 4);
          r[u] += 0x00400040u;
        }
        ph4[q] = __byte_perm(h[0] << 1, h[1] << 1, 0x7531);
        pl4[q] = __byte_perm(r[0] << 1, r[1] << 1, 0x7531);
      }
      if (j > 0) wait(smem_u32(&bars->p_free), (j - 1) & 1, ab);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t dst = s0 + kF8OffP + sw64_offset(row, 2 * hh + u);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(ph4[4 * u]), "r"(ph4[4 * u + 1]),
                     "r"(ph4[4 * u + 2]), "r"(ph4[4 * u + 3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + kF8PBytes), "r"(pl4[4 * u]),
                     "r"(pl4[4 * u + 1]), "r"(pl4[4 * u + 2]), "r"(pl4[4 * u + 3])
                     : "memory");
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_full));
    }

    // Epilogue: the row sums over the positions, O normalised and turned
    // round through the idle stages (a head's 512 columns contiguous), one
    // bulk copy a head.
    red[qd * kF8Heads + 32 * hh + lane] = reduce_transposed(l, lane, fadd2);
    named_bar_sync(1, kAll);
    if (tid < kF8Heads) {
      const float sum = (red[tid] + red[kF8Heads + tid]) + (red[2 * kF8Heads + tid] + red[3 * kF8Heads + tid]);
      alpha[tid] = sum == 0.f ? 0.f : (1.f / 256.f) / sum;  // P's E4M3 value is 2^8 times its fp16 one
      if (tid < live)
        lse_part[((size_t)b * n_split + split) * n_heads + h0 + tid] =
            sum == 0.f ? -INFINITY : (mref[tid] + log2f(sum)) * 0.6931471805599453f;
    }
    wait(smem_u32(&bars->p_free), (n_tiles - 1) & 1, ab);
    tc_fence_after();
    named_bar_sync(1, kAll);
    constexpr uint32_t kRow = kDl * 2 + 16;
#pragma unroll 1
    for (int cc = 0; cc < 4; ++cc) {
      const int m = 2 * hh + (cc >> 1), hb = (cc & 1) * 32;
      uint32_t ov[32];
      tmem_ld32(tmem + lane_base + kF8ColO + m * 64 + hb, ov);
      tmem_wait_ld();
      const uint32_t dst = s0 + (uint32_t)(m * 128 + row) * 2u;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const __nv_bfloat16 v = __float2bfloat16_rn(__uint_as_float(ov[i]) * alpha[hb + i]);
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + (uint32_t)(hb + i) * kRow), "h"(__bfloat16_as_ushort(v))
                     : "memory");
      }
    }
    fence_proxy_async_smem();
    named_bar_sync(1, kAll);
    if (tid < live) {
      bulk_store(o_part + (((size_t)b * n_split + split) * n_heads + h0 + tid) * kDl, s0 + tid * kRow, kDl * 2);
      bulk_commit();
      bulk_wait_read();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kF8PvWarp) tmem_dealloc(tmem, 512);
}

}  // namespace mla
