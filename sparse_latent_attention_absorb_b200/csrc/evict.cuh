// Eviction from a latent cache by accumulated attention weight (no counterpart
// on the pages: their cache only grows).  Of a row's n positions the last
// `recent` stay, and of the others those of the largest total weight, `keep` in
// all; they move up in their order.
//
//   evict_select_kernel  the kept positions: the weight of rank `keep - recent`
//                        by three passes of radix selection (11, 11 and 10
//                        bits), ties by position, then one scan that numbers
//                        the kept positions; the totals move along
//   evict_move_kernel    the rows
//
// Bound: the select reads a row's totals five times from L1 and L2 with one
// CTA a row, the move is HBM traffic.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "append_fp8.cuh"

namespace mla {

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;

// Bits whose unsigned order is the weights' order, NaN above all, the two zeros
// equal.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Sums over the block of threads before this one (exclusive), and of all.
__device__ __forceinline__ int2 block_scan2(int2 v, int2* warp_sums, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, s), b = __shfl_up_sync(0xffffffffu, x.y, s);
    if (lane >= s) x.x += a, x.y += b;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int2 w = warp_sums[lane];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, w.x, s), b = __shfl_up_sync(0xffffffffu, w.y, s);
      if (lane >= s) w.x += a, w.y += b;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int2 before = warp > 0 ? warp_sums[warp - 1] : make_int2(0, 0);
  *total = warp_sums[31];
  return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

__global__ void __launch_bounds__(kSelectThreads, 1)
evict_select_kernel(const float* acc, const int32_t* __restrict__ end_pos, float* acc_out,
                    int32_t* __restrict__ kept, int32_t* __restrict__ new_end, int S_max, int keep, int recent) {
  __shared__ uint32_t bins[kSelectBins];
  __shared__ int2 warp_sums[32];
  __shared__ uint32_t found[2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const float* w = acc + (size_t)b * S_max;
  int32_t* kp = kept + (size_t)b * keep;
  int n = end_pos[b];
  n = n < 0 ? 0 : (n > S_max ? S_max : n);
  const int n_new = min(n, keep);
  const int late = n - min(recent, keep);  // positions from here on stay (n > keep)

  if (n <= keep) {
    for (int i = tid; i < keep; i += kSelectThreads) kp[i] = i < n ? i : -1;
  } else {
    // the key of rank `rank` (from 0, largest first) among [0, late)
    uint32_t prefix = 0, mask = 0;
    int rank = keep - min(recent, keep);  // how many of [0, late) stay
    if (rank > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), width = pass == 2 ? 10 : 11;
        for (int i = tid; i < kSelectBins; i += kSelectThreads) bins[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < late; i0 += kSelectThreads) {
          const int i = i0 + tid;
          const uint32_t k = i < late ? weight_key(w[i]) : 0u;
          const bool in = i < late && (k & mask) == prefix;
          const uint32_t bin = (k >> shift) & ((1u << width) - 1u);
          // equal weights (never selected: 0) would queue up at one bin: the
          // lanes that share the first lane's bin count as one
          const uint32_t act = __ballot_sync(0xffffffffu, in);
          if (act) {
            const uint32_t lead = __shfl_sync(0xffffffffu, bin, __ffs(act) - 1);
            const uint32_t same = __ballot_sync(0xffffffffu, in && bin == lead);
            if (lane == __ffs(act) - 1)
              atomicAdd(&bins[lead], (uint32_t)__popc(same));
            else if (in && bin != lead)
              atomicAdd(&bins[bin], 1u);
          }
        }
        __syncthreads();
        // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
        const int b0 = kSelectBins - 1 - 2 * tid;
        const int c0 = (int)bins[b0], c1 = (int)bins[b0 - 1];
        int2 total;
        const int before = block_scan2(make_int2(c0 + c1, 0), warp_sums, &total).x;
        if (before < rank && rank <= before + c0) found[0] = (uint32_t)b0, found[1] = (uint32_t)before;
        if (before + c0 < rank && rank <= before + c0 + c1) found[0] = (uint32_t)(b0 - 1), found[1] = (uint32_t)(before + c0);
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= ((1u << width) - 1u) << shift;
        rank -= (int)found[1];
        __syncthreads();
      }
    } else {
      prefix = 0xffffffffu;  // no key is larger, and none of the ties stays
    }
    // Above the key, or one of its first `rank` ties, or late: a thread takes
    // a run of positions, so that one scan numbers them all.
    const int run = (n + kSelectThreads - 1) / kSelectThreads;
    const int i0 = min(n, tid * run), i1 = min(n, i0 + run);
    int2 c = make_int2(0, 0);
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = i < late ? weight_key(w[i]) : 0u;
      c.x += i >= late || k > prefix;
      c.y += i < late && k == prefix;
    }
    int2 total;
    int2 at = block_scan2(c, warp_sums, &total);
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = i < late ? weight_key(w[i]) : 0u;
      const bool tie = i < late && k == prefix;
      const bool stays = i >= late || k > prefix || (tie && at.y < rank);
      // positions above the key before i, and the ties among them that stay
      if (stays) kp[at.x + min(at.y, rank)] = i;
      at.x += i >= late || k > prefix;
      at.y += tie;
    }
  }
  if (tid == 0) new_end[b] = n_new;
  __syncthreads();
  // The totals of the kept positions, then zeros.  acc_out may be acc: what a
  // step writes, [i0, i0 + 1024), no later step reads, and its own reads are
  // done.
  float* out = acc_out + (size_t)b * S_max;
  for (int i0 = 0; i0 < n_new; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const float v = i < n_new ? w[kp[i]] : 0.f;
    __syncthreads();
    if (i < n_new) out[i] = v;
  }
  __syncthreads();
  for (int i = n_new + tid; i < S_max; i += kSelectThreads) out[i] = 0.f;
}

// Rows kept[i] of a slot to rows i, 128 a step: 16 warps of eight rows, held in
// registers.  The 8-bit cache's new blocks get the largest scale of their rows,
// and rows of a smaller one are rounded again.
//   out of place: a CTA per 128 rows;
//   in place: a cluster of eight CTAs per slot walks up its rows, and writes a
//   step once all of it has been read (kept[i] >= i: what a step writes, no
//   later step reads).
constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 128;
constexpr int kMoveCluster = 8;

struct MoveArgs {
  const uint8_t* kv;   // bf16 rows of 1024 bytes or codes of 512
  const uint8_t* pe;   // rows of 128 bytes
  const float* scale;  // 8-bit cache only
  uint8_t* kv_out;
  uint8_t* pe_out;
  float* scale_out;
  const int32_t* kept;     // [B, keep]
  const int32_t* new_end;  // [B]
  const int32_t* end_pos;  // [B]
  int S_max, keep, shift, n_blocks;
};

template <bool kFp8, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, 1) evict_move_kernel(const MoveArgs a) {
  constexpr int kVecs = kFp8 ? 1 : 2;  // 16-byte pieces of a lane
  constexpr size_t kRow = kVecs * 512;
  __shared__ float src_scale[kMoveRows], dst_scale[kMoveRows];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.new_end[b];
  const int32_t* kept = a.kept + (size_t)b * a.keep;
  const size_t row0 = (size_t)b * a.S_max;
  const int block = 1 << a.shift;
  const int step = kInPlace ? kMoveCluster * kMoveRows : kMoveRows;
  for (int base = kInPlace ? 0 : blockIdx.x * kMoveRows; base < n; base += step) {
    const int i0 = kInPlace ? base + (int)blockIdx.x * kMoveRows : base;
    if (kInPlace) {
      const int last = min(base + step, n) - 1;
      if (kept[last] == last) continue;  // nothing has moved up to here
    }
    int src[8];
    uint4 v[8][kVecs];
    uint32_t pe[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int i = i0 + 8 * warp + r;
      src[r] = i < n ? kept[i] : -1;
    }
    if (kFp8 && tid < kMoveRows) {
      const int s = i0 + tid < n ? kept[i0 + tid] : -1;
      src_scale[tid] = s >= 0 ? a.scale[(size_t)b * a.n_blocks + (s >> a.shift)] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (src[r] < 0) continue;
      const size_t at = row0 + src[r];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) v[r][u] = reinterpret_cast<const uint4*>(a.kv + at * kRow)[32 * u + lane];
      pe[r] = reinterpret_cast<const uint32_t*>(a.pe + at * (kDr * 2))[lane];
    }
    __syncthreads();
    if (kFp8 && tid < kMoveRows) {
      // the block's largest scale (a tile holds whole blocks)
      const int t0 = tid & ~(block - 1);
      float s = src_scale[t0];
      for (int t = t0 + 1; t < t0 + block; ++t) s = fmaxf(s, src_scale[t]);
      dst_scale[tid] = s;
    }
    if (kInPlace) {
      cluster_sync();
    } else {
      __syncthreads();
    }
    if (kFp8 && tid < kMoveRows && i0 + tid < n && (tid & (block - 1)) == 0)
      a.scale_out[(size_t)b * a.n_blocks + ((i0 + tid) >> a.shift)] = dst_scale[tid];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (src[r] < 0) continue;
      const size_t at = row0 + i0 + 8 * warp + r;
      if (kFp8) {
        const float from = src_scale[8 * warp + r], to = dst_scale[8 * warp + r];
        if (from != to) {
          v[r][0] = recode16(v[r][0], from / to);
          pe[r] = rescale_pe(pe[r], from / to);
        }
      }
#pragma unroll
      for (int u = 0; u < kVecs; ++u) reinterpret_cast<uint4*>(a.kv_out + at * kRow)[32 * u + lane] = v[r][u];
      reinterpret_cast<uint32_t*>(a.pe_out + at * (kDr * 2))[lane] = pe[r];
    }
    __syncthreads();  // the scales of this step are used up
  }
}

}  // namespace mla
