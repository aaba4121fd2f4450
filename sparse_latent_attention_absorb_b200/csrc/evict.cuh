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
// Bound: the selection by its chain of passes (a row is one CTA, of a few long
// rows a cluster of eight: 64 rows of 8192 take about 13 us, 27000 cycles of
// which 6300 are the first read of the totals and their histogram, 4600 the
// numbering), the move by HBM (64 rows of up to 8192 keeping 2500 in 8 bits, 209 MB:
// 35 us, 6.0 TB/s).  The move's CTAs come up while the selection runs.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "append_fp8.cuh"

namespace mla {

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;
constexpr int kSelectHold = 8;  // totals that a thread holds
constexpr int kSelectCluster = 8;

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

// A row's CTAs (one, or a cluster of kSelectCluster for long rows) take a run
// of its positions each; histograms and counts meet through distributed shared
// memory.
__global__ void __launch_bounds__(kSelectThreads, 1)
evict_select_kernel(const float* acc, const int32_t* __restrict__ end_pos, float* acc_out,
                    int32_t* kept, int32_t* __restrict__ new_end, int S_max, int keep, int recent) {
  __shared__ uint32_t bins[kSelectBins], meet[kSelectBins];
  __shared__ int2 warp_sums[32];
  __shared__ uint32_t found[2];
  __shared__ int2 counts;
  grid_dep_launch();  // the rows' kernel may come up
  const int n_cta = (int)cluster_size(), rank = (int)cluster_ctarank();
  const int b = blockIdx.x / n_cta, tid = threadIdx.x, lane = tid & 31;
  const float* w = acc + (size_t)b * S_max;
  float* out = acc_out + (size_t)b * S_max;
  const bool apart = acc_out != acc;
  int32_t* kp = kept + (size_t)b * keep;
  int n = end_pos[b];
  n = n < 0 ? 0 : (n > S_max ? S_max : n);
  const int n_new = min(n, keep);
  const int late = n - min(recent, keep);  // positions from here on stay (n > keep)
  const int all = n_cta * kSelectThreads, me = rank * kSelectThreads + tid;

  if (n <= keep) {
    for (int i = me; i < keep; i += all) {
      kp[i] = i < n ? i : -1;
      if (apart && i < n) out[i] = w[i];
    }
  } else {
    const int seg = (n + n_cta * 1024 - 1) / (n_cta * 1024) * 1024;  // a CTA's positions
    const int s0 = min(n, rank * seg), s1 = min(n, s0 + seg);
    // A warp takes 1/32 of the CTA's positions, 32 at a time.  Up to 8192
    // positions of a CTA stay in registers through all passes; of more, each
    // pass reads them again (from L1 and L2).
    const int run = seg / 32;
    const int i0 = min(s1, s0 + (tid >> 5) * run), i1 = min(s1, i0 + run);
    float x[kSelectHold];
    bool held = false;
    auto fetch = [&](int i) {
      if (held) return;
#pragma unroll
      for (int u = 0; u < kSelectHold; ++u) x[u] = i + 32 * u + lane < i1 ? w[i + 32 * u + lane] : 0.f;
      held = run <= 32 * kSelectHold;
    };
    auto sync_row = [&]() {
      if (n_cta > 1)
        cluster_sync();
      else
        __syncthreads();
    };
    // the key of rank `left` (from 1, largest first) among [0, late)
    uint32_t prefix = 0, mask = 0;
    int left = keep - min(recent, keep);  // how many of [0, late) stay
    if (left > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), width = pass == 2 ? 10 : 11;
        for (int i = tid; i < kSelectBins; i += kSelectThreads) bins[i] = 0;
        __syncthreads();
        for (int i = i0; i < i1; i += 32 * kSelectHold) {
          fetch(i);
#pragma unroll
          for (int u = 0; u < kSelectHold; ++u) {
            if (i + 32 * u >= i1) break;
            const uint32_t k = weight_key(x[u]);
            const bool in = i + 32 * u + lane < min(i1, late) && (k & mask) == prefix;
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
        }
        sync_row();
        // bins from the top, of all CTAs: thread t holds bins 2047 - 2t and 2046 - 2t
        const int b0 = kSelectBins - 1 - 2 * tid;
        const uint32_t* sums = bins;
        if (n_cta > 1) {
          // a CTA adds up its share of the bins and tells everyone
          const int share = kSelectBins / kSelectCluster;
          if (tid < share) {
            const uint32_t at = smem_u32(&bins[rank * share + tid]), to = smem_u32(&meet[rank * share + tid]);
            uint32_t sum = 0;
#pragma unroll
            for (int r = 0; r < kSelectCluster; ++r) sum += ld_cluster_u32(cluster_map(at, (uint32_t)r));
#pragma unroll
            for (int r = 0; r < kSelectCluster; ++r) st_cluster_u32(cluster_map(to, (uint32_t)r), sum);
          }
          cluster_sync();
          sums = meet;
        }
        const int c0 = (int)sums[b0], c1 = (int)sums[b0 - 1];
        int2 total;
        const int before = block_scan2(make_int2(c0 + c1, 0), warp_sums, &total).x;
        if (before < left && left <= before + c0) found[0] = (uint32_t)b0, found[1] = (uint32_t)before;
        if (before + c0 < left && left <= before + c0 + c1) found[0] = (uint32_t)(b0 - 1), found[1] = (uint32_t)(before + c0);
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= ((1u << width) - 1u) << shift;
        left -= (int)found[1];
      }
    } else {
      prefix = 0xffffffffu;  // no key is larger, and none of the ties stays
    }
    // Above the key, or one of its first `left` ties, or late: every warp counts
    // its own, and the sums over the warps and CTAs before it tell it where they
    // go.
    // the lanes of a step whose position is above the key, and its ties
    auto look = [&](float v, int i, uint32_t* above, uint32_t* ties) {
      const uint32_t k = weight_key(v);
      *above = __ballot_sync(0xffffffffu, i < i1 && (i >= late || k > prefix));
      *ties = __ballot_sync(0xffffffffu, i < i1 && i < late && k == prefix);
    };
    int2 c = make_int2(0, 0);
    for (int i = i0; i < i1; i += 32 * kSelectHold) {
      fetch(i);
#pragma unroll
      for (int u = 0; u < kSelectHold; ++u) {
        if (i + 32 * u >= i1) break;
        uint32_t above, ties;
        look(x[u], i + 32 * u + lane, &above, &ties);
        c.x += __popc(above), c.y += __popc(ties);
      }
    }
    int2 total;
    int2 at = block_scan2(lane == 31 ? c : make_int2(0, 0), warp_sums, &total);
    at.x = __shfl_sync(0xffffffffu, at.x, 0), at.y = __shfl_sync(0xffffffffu, at.y, 0);
    if (tid == 0) counts = total;
    sync_row();
    for (int r = 0; r < rank; ++r) {
      const uint32_t far = cluster_map(smem_u32(&counts), (uint32_t)r);
      at.x += (int)ld_cluster_u32(far), at.y += (int)ld_cluster_u32(far + 4);
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i = i0; i < i1; i += 32 * kSelectHold) {
      fetch(i);
#pragma unroll
      for (int u = 0; u < kSelectHold; ++u) {
        if (i + 32 * u >= i1) break;
        uint32_t above, ties;
        look(x[u], i + 32 * u + lane, &above, &ties);
        const int tie = at.y + __popc(ties & below);
        // positions above the key before this one, and the ties among them that stay
        const int to = at.x + __popc(above & below) + min(tie, left);
        if ((above >> lane & 1u) || ((ties >> lane & 1u) && tie < left)) {
          kp[to] = i + 32 * u + lane;
          if (apart) out[to] = x[u];
        }
        at.x += __popc(above), at.y += __popc(ties);
      }
    }
  }
  if (me == 0) new_end[b] = n_new;
  if (apart) {
    for (int i = n_new + me; i < S_max; i += all) out[i] = 0.f;
  }
  if (n_cta > 1)
    cluster_sync();  // kept is whole, and no CTA reads another's memory any more
  else
    __syncthreads();
  if (apart || rank != 0) return;
  // In place, one CTA: what a step writes, [i0, i0 + 1024), no later step
  // reads, and its own reads are done.
  for (int i0 = 0; n > keep && i0 < n_new; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const float v = i < n_new ? w[kp[i]] : 0.f;
    __syncthreads();
    if (i < n_new) out[i] = v;
  }
  __syncthreads();
  for (int i = n_new + tid; i < S_max; i += kSelectThreads) out[i] = 0.f;
}

// Rows kept[i] of a slot to rows i: 16 warps of eight rows (four), held in
// registers.  The 8-bit cache's new blocks get the largest scale of their rows,
// and rows of a smaller one are rounded again.
//   out of place: a CTA per 128 (64) rows;
//   in place: a cluster of eight CTAs per slot walks up its rows, and writes a
//   step once all of it has been read (kept[i] >= i: what a step writes, no
//   later step reads).  Reads and writes take turns, and few slots leave SMs
//   idle: whole calls 18.2, 75.8 and 121.0 us (1 row of 4096, 64 of up to 8192 in
//   8 bits, 8 of 32768 in bf16) against 14.4, 50.6 and 64.0 out of place.
constexpr int kMoveThreads = 512;
// Rows of a warp, and of a CTA: out of place two CTAs share an SM, so that one
// reads while the other writes, and bf16 rows then leave registers for four a
// warp.  (A CTA's 128 rows of the 8-bit cache are whole blocks of positions.)
__host__ __device__ constexpr int move_warp_rows(bool fp8, bool in_place) { return fp8 || in_place ? 8 : 4; }
__host__ __device__ constexpr int move_rows(bool fp8, bool in_place) { return kMoveThreads / 32 * move_warp_rows(fp8, in_place); }
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
  int S_max, keep, shift, n_blocks;
};

template <bool kFp8, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, kInPlace ? 1 : 2) evict_move_kernel(const MoveArgs a) {
  constexpr int kVecs = kFp8 ? 1 : 2;  // 16-byte pieces of a lane
  constexpr size_t kRow = kVecs * 512;
  constexpr int kWarpRows = move_warp_rows(kFp8, kInPlace), kMoveRows = move_rows(kFp8, kInPlace);
  __shared__ float src_scale[kMoveRows], dst_scale[kMoveRows];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_wait();  // kept and new_end come from the selection
  const int n = a.new_end[b];
  const int32_t* kept = a.kept + (size_t)b * a.keep;
  const size_t row0 = (size_t)b * a.S_max;
  const int block = 1 << a.shift;
  const int step = (int)gridDim.x * kMoveRows;  // out of place: the grid covers `keep`, one step
  for (int base = 0; base < n; base += step) {
    const int i0 = base + (int)blockIdx.x * kMoveRows;
    if (!kInPlace && i0 >= n) break;
    if (kInPlace) {
      const int last = min(base + step, n) - 1;
      if (kept[last] == last) continue;  // nothing has moved up to here
    }
    int src[kWarpRows];
    uint4 v[kWarpRows][kVecs];
    uint32_t pe[kWarpRows];
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      const int i = i0 + kWarpRows * warp + r;
      src[r] = i < n ? kept[i] : -1;
    }
    if (kFp8 && tid < kMoveRows) {
      const int s = i0 + tid < n ? kept[i0 + tid] : -1;
      src_scale[tid] = s >= 0 ? a.scale[(size_t)b * a.n_blocks + (s >> a.shift)] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      if (src[r] < 0) continue;
      const size_t at = row0 + src[r];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) v[r][u] = reinterpret_cast<const uint4*>(a.kv + at * kRow)[32 * u + lane];
      pe[r] = reinterpret_cast<const uint32_t*>(a.pe + at * (kDr * 2))[lane];
    }
    __syncthreads();
    if (kFp8 && tid < kMoveRows) {
      // the block's largest scale, of 32 rows at most
      float s = src_scale[tid];
      for (int o = 1; o < min(block, 32); o <<= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
      dst_scale[tid] = s;
    }
    if (kInPlace) {
      cluster_sync();
    } else {
      __syncthreads();
    }
    auto block_scale = [&](int t) {  // (a tile holds whole blocks)
      float s = dst_scale[t];
      for (int o = 32; o < block; o += 32) s = fmaxf(s, dst_scale[(t & ~(block - 1)) | ((t + o) & (block - 1))]);
      return s;
    };
    if (kFp8 && tid < kMoveRows && i0 + tid < n && (tid & (block - 1)) == 0)
      a.scale_out[(size_t)b * a.n_blocks + ((i0 + tid) >> a.shift)] = block_scale(tid);
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      if (src[r] < 0) continue;
      const size_t at = row0 + i0 + kWarpRows * warp + r;
      if (kFp8) {
        const float from = src_scale[kWarpRows * warp + r], to = block_scale(kWarpRows * warp + r);
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
