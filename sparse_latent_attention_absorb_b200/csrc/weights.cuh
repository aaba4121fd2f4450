// The attention weight every selected position got, summed over the heads and
// added to its running total (no counterpart on the pages; what eviction goes
// by):
//   acc[b, t] += sum_h exp(score_{h,t} - lse_h)        t selected in row b
// with the scores of the decode step (model.py 596-597 of the atlas page
// "Query-key similarity") and the log-sum-exps it left, over the bf16 cache or
// the 8-bit one.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "attend_fp8.cuh"

namespace mla {

// Thirty-two values of each lane, summed over the lanes: lane i returns the
// sum of value i (31 exchanges instead of 160).
__device__ __forceinline__ float sum_transposed(float (&v)[32], int lane) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = up ? v[i + s] : v[i], send = up ? v[i] : v[i + s];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  return v[0];
}

// =============================================================================
// accumulate_weights_kernel
//
// One CTA per (row, key split), all 128 heads: M = 128 heads, N = 128
// positions.  The query is the A operand in TMEM for the CTA's life (bf16
// cache: 256 columns of bf16 pairs; 8-bit cache: its E4M3 limbs, 128 columns
// each, both accumulating into the same scores: the second limb is then not
// scaled up, which leaves 2^-19 of the largest factor); the scores have two
// buffers.  A softmax thread holds one head and 64 positions of a tile; a
// position's sum over the heads goes across the lanes and, in shared memory,
// across the four lane quarters.
//
// Bound: the gather, 1152 (640) bytes a position, each read once.  The rows
// come in groups of blocks (16 KB: 128 positions x 128 bytes): a group is
// awaited, multiplied and released as one, since a wait and its proxy fence
// cost as much as a block's MMAs.  Measured: 64 rows of 2048 positions in bf16
// (162 MB) 32.9 us, 4.9 TB/s; 8 rows in 8 bits 11.3 us, most of it the query's
// way into TMEM.  An L2 prefetch of the next tile's rows held up the copies in
// the load pipeline (43 us); eight gather warps change nothing.
//
// Warps (448 threads): 0-7 weights (warp w: heads 32 (w % 4).., positions
// 64 (w / 4)..), 8-11 gather, 12 TMEM, query load and QK issue, 13 positions and
// scales.
// =============================================================================
constexpr int kWtNt = 128;
constexpr int kWtBlock = kWtNt * 128;
__host__ __device__ constexpr int wt_blocks(bool fp8) { return fp8 ? 5 : 9; }  // a tile's: rotary, then latent
__host__ __device__ constexpr int wt_group(bool fp8) { return fp8 ? 5 : 3; }   // blocks of a group
__host__ __device__ constexpr int wt_groups(bool fp8) { return fp8 ? 2 : 4; }  // groups of the ring
constexpr int kWtBox = 4;  // the query's eight boxes lie in the ring's blocks 4 .. 11 at first
constexpr int kWtOffQpe = 12 * kWtBlock;
constexpr int kWtOffScale = kWtOffQpe + kWtBlock;          // f32 [4][128]
constexpr int kWtOffPos = kWtOffScale + 4 * kWtNt * 4;     // int [4][128], -1 = masked
constexpr int kWtOffRed = kWtOffPos + 4 * kWtNt * 4;       // f32 [2][4][128]
constexpr int kWtOffBad = kWtOffRed + 2 * 4 * kWtNt * 4;   // f32 [128]
constexpr int kWtOffBar = kWtOffBad + kH * 4;
constexpr int kWtSmemBytes = kWtOffBar + 256 + kSmemAlignPad;
constexpr int kWtThreads = 448;
constexpr int kWtGatherWarp = 8, kWtGatherWarps = 4, kWtQkWarp = 12, kWtIndexWarp = 13;
constexpr uint32_t kWtColS = 0, kWtColQ = 256;
static_assert(kWtSmemBytes <= 232448, "shared memory");

struct WtBars {
  uint64_t q_tma, q_full;
  uint64_t full[4], empty[4];            // groups
  uint64_t tile_full[4], tile_done[4];   // positions and scales written, used up
  uint64_t s_full[2], s_empty[2];
  uint64_t drained;                      // the MMAs of an aborted kernel
  uint32_t tmem_addr;
  int abort_flag;
};
static_assert(sizeof(WtBars) <= 256, "barrier block");

template <bool kFp8>
__global__ void __launch_bounds__(kWtThreads, 1)
accumulate_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __nv_bfloat16* __restrict__ q_pe,
                          const uint8_t* __restrict__ kv, const uint8_t* __restrict__ pe,
                          const float* __restrict__ kv_scale, int block_shift, int n_blocks,
                          const int32_t* __restrict__ end_pos, const int32_t* __restrict__ topk_idx, float scale,
                          const float* __restrict__ lse, float* __restrict__ acc, int K, int S_max, int n_split,
                          int span, int n_heads, int* d_status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  constexpr int kBlocks = wt_blocks(kFp8), kGroup = wt_group(kFp8), kGroups = wt_groups(kFp8);
  constexpr int kPer = kBlocks / kGroup;        // groups of a tile
  constexpr int kRowBytes = kFp8 ? kDl : 2 * kDl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / n_split, split = blockIdx.x % n_split;
  const int k_begin = split * span, k_end = min(K, k_begin + span);
  const int n_tiles = (k_end - k_begin + kWtNt - 1) / kWtNt;
  int ep = end_pos[b];
  ep = ep < 0 ? 0 : (ep > S_max ? S_max : ep);

  const uint32_t s0 = smem_u32(smem);
  float* sc = reinterpret_cast<float*>(smem + kWtOffScale);
  int* pos_s = reinterpret_cast<int*>(smem + kWtOffPos);
  float* red = reinterpret_cast<float*>(smem + kWtOffRed);
  float* bad_s = reinterpret_cast<float*>(smem + kWtOffBad);
  WtBars* bars = reinterpret_cast<WtBars*>(smem + kWtOffBar);
  const AbortState ab{&bars->abort_flag, d_status};

  if (tid == 0) {
    bars->abort_flag = 0;
    mbar_init(smem_u32(&bars->q_tma), 1);
    mbar_init(smem_u32(&bars->q_full), 8);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 32 * kWtGatherWarps * kGroup);
      mbar_init(smem_u32(&bars->empty[i]), 1);
      mbar_init(smem_u32(&bars->tile_full[i]), 1);
      mbar_init(smem_u32(&bars->tile_done[i]), 4);
    }
    mbar_init(smem_u32(&bars->drained), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      mbar_init(smem_u32(&bars->s_empty[i]), 8);
    }
    fence_mbarrier_init_cluster();
  }
  if (warp == kWtQkWarp) {
    tmem_alloc(smem_u32(&bars->tmem_addr), 512);
    tmem_relinquish();
  }
  if (tid < kH) bad_s[tid] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_addr;
  const uint8_t* kv_row = kv + (size_t)b * S_max * kRowBytes;
  const uint8_t* pe_row = pe + (size_t)b * S_max * (kDr * 2);

  if (warp == kWtIndexWarp) {
    // ---------------------------------------------------------- positions
    // Up to four tiles ahead; the loads for the tiles after are in flight.
    const int32_t* idx_row = topk_idx + (size_t)b * K;
    const float* sc_row = kFp8 ? kv_scale + (size_t)b * n_blocks : nullptr;
    struct Four {
      int pos[4];
    };
    auto load = [&](int j) -> Four {
      Four f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k_begin + j * kWtNt + 32 * i + lane;
        const int v = k < k_end ? __ldg(idx_row + k) : -1;
        f.pos[i] = (v >= 0 && v < ep) ? v : -1;
      }
      return f;
    };
    auto scale_of = [&](int p) -> float { return kFp8 && p >= 0 ? __ldg(sc_row + (p >> block_shift)) : 0.f; };
    Four cur = load(0), next = load(1);
    float sv[4], sv_next[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sv[i] = scale_of(cur.pos[i]);
    for (int j = 0; j < n_tiles; ++j) {
      const Four next2 = load(j + 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) sv_next[i] = scale_of(next.pos[i]);
      if (j >= 4) wait(smem_u32(&bars->tile_done[j & 3]), ((j >> 2) - 1) & 1, ab);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pos_s[(j & 3) * kWtNt + 32 * i + lane] = cur.pos[i];
        if (kFp8) sc[(j & 3) * kWtNt + 32 * i + lane] = sv[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->tile_full[j & 3]));
      cur = next;
      next = next2;
#pragma unroll
      for (int i = 0; i < 4; ++i) sv[i] = sv_next[i];
    }
  } else if (warp >= kWtGatherWarp && warp < kWtGatherWarp + kWtGatherWarps) {
    // ------------------------------------------------------------ gather
    // A copy instruction brings 128 bytes of four positions; a warp holds its
    // positions in registers for all blocks of the tile.
    const int g = warp - kWtGatherWarp;
    constexpr int kCopies = 32 / kWtGatherWarps;
    const uint32_t dst0 = s0 + sw128_offset(4 * g + (lane >> 3), lane & 7);
    int gr = 0;
    uint32_t ph = 1;
    for (int j = 0; j < n_tiles; ++j) {
      int pos[kCopies];
      const bool known = wait(smem_u32(&bars->tile_full[j & 3]), (j >> 2) & 1, ab);  // else timed out: nothing is read
#pragma unroll
      for (int u = 0; u < kCopies; ++u) pos[u] = !known ? -1 : pos_s[(j & 3) * kWtNt + 4 * (g + kWtGatherWarps * u) + (lane >> 3)];
#pragma unroll 1
      for (int i = 0; i < kBlocks; ++i) {
        if (i % kGroup == 0) wait(smem_u32(&bars->empty[gr]), ph, ab);
        // the query's boxes lie in the ring until they are in TMEM
        if (j == 0 && gr * kGroup + i % kGroup == kWtBox) wait(smem_u32(&bars->q_full), 0, ab);
        const uint8_t* src = (i == 0 ? pe_row : kv_row + (i - 1) * 128) + (lane & 7) * 16;
        const uint32_t row_bytes = i == 0 ? kDr * 2 : kRowBytes;
        const uint32_t dst = dst0 + (gr * kGroup + i % kGroup) * kWtBlock;
#pragma unroll
        for (int u = 0; u < kCopies; ++u)
          cp_async_16(dst + u * (4 * kWtGatherWarps * 128), src + (uint64_t)max(pos[u], 0) * row_bytes, pos[u] >= 0 ? 16u : 0u);
        cp_async_arrive(smem_u32(&bars->full[gr]));
        if (i % kGroup == kGroup - 1 && ++gr == kGroups) gr = 0, ph ^= 1;
      }
    }
  } else if (warp == kWtQkWarp) {
    // ------------------------------------------------ query load, QK issue
    if (lane == 0) {
      // eight boxes of 64 columns x 128 heads (heads past the call's read as zero)
      tma_prefetch_desc(&tm_q);
      mbar_arrive_expect_tx(smem_u32(&bars->q_tma), kH * kDl * 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) tma_load_3d(s0 + (kWtBox + i) * kWtBlock, &tm_q, smem_u32(&bars->q_tma), i * 64, 0, b);

      constexpr uint32_t id_16 = idesc_bf16_f32(128, kWtNt, false, false);
      constexpr uint32_t id_8 = idesc_e4m3_f32(128, kWtNt, false, false);
      const uint64_t d_0 = smem_desc_sw128(s0, 16, 1024);
      const uint64_t d_qpe = smem_desc_sw128(s0 + kWtOffQpe, 16, 1024);
      const uint32_t q = tmem + kWtColQ;
      wait(smem_u32(&bars->q_full), 0, ab);
      int gr = 0;
      uint32_t ph = 0;
      for (int j = 0; j < n_tiles; ++j) {
        const uint32_t dst = tmem + kWtColS + (j & 1) * kWtNt;
        if (j >= 2) wait(smem_u32(&bars->s_empty[j & 1]), ((j >> 1) - 1) & 1, ab);
#pragma unroll 1
        for (int t = 0; t < kPer; ++t) {
          wait(smem_u32(&bars->full[gr]), ph, ab);
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < kGroup; ++u) {
            const int i = t * kGroup + u;
            const uint64_t k0 = d_0 + (uint64_t)(((gr * kGroup + u) * kWtBlock) >> 4);
            if (i == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ss(dst, d_qpe + (uint64_t)(k * 2), k0 + (uint64_t)(k * 2), id_16, k > 0 ? 1u : 0u);
            } else if (kFp8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                mma_f8_ts(dst, q + (i - 1) * 32 + k * 8, k0 + (uint64_t)(k * 2), id_8, 1u);
                mma_f8_ts(dst, q + 128 + (i - 1) * 32 + k * 8, k0 + (uint64_t)(k * 2), id_8, 1u);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ts(dst, q + (i - 1) * 32 + k * 8, k0 + (uint64_t)(k * 2), id_16, 1u);
            }
          }
          mma_commit(smem_u32(&bars->empty[gr]));
          if (++gr == kGroups) gr = 0, ph ^= 1;
        }
        mma_commit(smem_u32(&bars->s_full[j & 1]));
      }
      if (*ab.flag) drain_mmas(smem_u32(&bars->drained));
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ weights
    const int qd = warp & 3, ch = warp >> 2;
    const int hd = 32 * qd + lane;
    const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
    float c2 = scale * 1.4426950408889634f;  // scores to log2 units
    const bool live = hd < n_heads;
    {
      // the query's row: 256 of its columns, and half of its rotary part
      const uint32_t box = s0 + (uint32_t)(kWtBox + 4 * ch) * kWtBlock + (uint32_t)hd * 128u;
      auto piece = [&](int c) {  // eight columns
        return ld_shared_v4(box + (uint32_t)(c >> 3) * kWtBlock + (uint32_t)(((c & 7) ^ (hd & 7)) << 4));
      };
      uint4 r4[4];
      const uint4* psrc = reinterpret_cast<const uint4*>(q_pe + ((size_t)b * n_heads + (live ? hd : 0)) * kDr) + 4 * ch;
#pragma unroll
      for (int u = 0; u < 4; ++u) r4[u] = live ? __ldg(psrc + u) : make_uint4(0, 0, 0, 0);
      const float rtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rotary_top(r4))));
      wait(smem_u32(&bars->q_tma), 0, ab);
      float mul = 1.f;
      if (kFp8) {
        uint32_t m2 = 0;
#pragma unroll 8
        for (int c = 0; c < 32; ++c) {
          const uint4 v = piece(c);
          m2 = amax2(amax2(amax2(amax2(m2, v.x), v.y), v.z), v.w);
        }
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
        if (m >= 0x7f80u) {  // an infinity or NaN: the head's weights are NaN, the others' scale is not its
          bad_s[hd] = 1.f;
          m = 0;
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) red[warp] = __uint_as_float(m << 16), red[8 + warp] = rtop;
        named_bar_sync(1, 256);
        float am = red[0], rm = red[8];
#pragma unroll
        for (int w = 1; w < 8; ++w) am = fmaxf(am, red[w]), rm = fmaxf(rm, red[8 + w]);
        const int e = query_exponent(am, rm);
        mul = exp2_int(e);
        c2 *= exp2_int(-e);
        if (bad_s[hd] != 0.f) c2 = __int_as_float(0x7fffffff);
      }
      // the loads first, so that their latency is met once a round
      constexpr int kRound = kFp8 ? 8 : 4;  // pieces
#pragma unroll 1
      for (int c = 0; c < 32; c += kRound) {
        uint4 v[kRound];
#pragma unroll
        for (int q = 0; q < kRound; ++q) v[q] = piece(c + q);
        uint32_t r[16];
        if constexpr (kFp8) {
          uint32_t lo[16];
#pragma unroll
          for (int q = 0; q < kRound; ++q) {
            limbs4(v[q].x, v[q].y, mul * (1.f / 256.f), 1.f, &r[2 * q], &lo[2 * q]);
            limbs4(v[q].z, v[q].w, mul * (1.f / 256.f), 1.f, &r[2 * q + 1], &lo[2 * q + 1]);
          }
          tmem_st16(tmem + lane_base + kWtColQ + 64 * ch + 2 * c, r);
          tmem_st16(tmem + lane_base + kWtColQ + 128 + 64 * ch + 2 * c, lo);
        } else {
#pragma unroll
          for (int q = 0; q < kRound; ++q) r[4 * q] = v[q].x, r[4 * q + 1] = v[q].y, r[4 * q + 2] = v[q].z, r[4 * q + 3] = v[q].w;
          tmem_st16(tmem + lane_base + kWtColQ + 128 * ch + 4 * c, r);
        }
      }
      tmem_wait_st();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t w[4] = {r4[u].x, r4[u].y, r4[u].z, r4[u].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // times a power of two: exact
          o[i] = kFp8 ? pack_bf16x2(__uint_as_float(w[i] << 16) * mul, __uint_as_float(w[i] & 0xffff0000u) * mul) : w[i];
        st_shared_v4(s0 + kWtOffQpe + sw128_offset(hd, 4 * ch + u), o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
    }
    // 2^(x - lse) of a lane without a head is 0
    const float lse2 = live ? lse[(size_t)b * n_heads + hd] * 1.4426950408889634f : INFINITY;
    const uint64_t c2p = pack_f32x2(live ? c2 : 0.f, live ? c2 : 0.f), off = pack_f32x2(-lse2, -lse2);

    for (int j = 0; j < n_tiles; ++j) {
      float* rt = red + (j & 1) * (4 * kWtNt) + qd * kWtNt + 64 * ch;
      const ulonglong2* kt = reinterpret_cast<const ulonglong2*>(sc + (j & 3) * kWtNt + 64 * ch);
      wait(smem_u32(&bars->tile_full[j & 3]), (j >> 2) & 1, ab);
      wait(smem_u32(&bars->s_full[j & 1]), (j >> 1) & 1, ab);
      tc_fence_after();
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + kWtColS + (j & 1) * kWtNt + 64 * ch + 32 * r, v);
        tmem_wait_ld();
        float p[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint64_t x0 = pack_f32x2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]));
          uint64_t x1 = pack_f32x2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
          if (kFp8) {
            const ulonglong2 f = kt[8 * r + q];
            x0 = mul_f32x2(x0, f.x);
            x1 = mul_f32x2(x1, f.y);
          }
          const float2 a = unpack_f32x2(fma_f32x2(x0, c2p, off)), d = unpack_f32x2(fma_f32x2(x1, c2p, off));
          p[4 * q] = ex2_approx(a.x);
          p[4 * q + 1] = ex2_approx(a.y);
          p[4 * q + 2] = ex2_approx(d.x);
          p[4 * q + 3] = ex2_approx(d.y);
        }
        if (n_heads < kH) {  // absent heads: zeros, which an infinite row turns into NaN
#pragma unroll
          for (int i = 0; i < 32; ++i) p[i] = live ? p[i] : 0.f;
        }
        rt[32 * r + lane] = sum_transposed(p, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty[j & 1]));
      named_bar_sync(1, 256);  // two buffers of sums: the next tile's go elsewhere
      if (warp < 4) {
        const float* s4 = red + (j & 1) * (4 * kWtNt) + tid;
        const int pos = pos_s[(j & 3) * kWtNt + tid];
        // Distinct positions: an addition a position, in whatever order.  Once a
        // wait of any warp has timed out (seen through the barriers since), the
        // scores may be anything, and nothing is added any more.
        if (!*ab.flag && pos >= 0) atomicAdd(acc + (size_t)b * S_max + pos, (s4[0] + s4[kWtNt]) + (s4[2 * kWtNt] + s4[3 * kWtNt]));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->tile_done[j & 3]));
      }
    }
  }

  cp_async_wait_all();  // after a timed-out wait, copies may still be in flight
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWtQkWarp) tmem_dealloc(tmem, 512);
}

}  // namespace mla
