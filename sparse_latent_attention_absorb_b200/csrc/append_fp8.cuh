// New tokens into the 8-bit latent cache (the pages' cache writer stores bf16
// rows; its body is not on them).  A block of positions shares one power-of-two
// scale s, the smallest with max|kv| <= 448 s over the block's rows:
//   code = e4m3(kv / s),  pe' = bf16(pe / s)      (both divisions exact)
// Where a run of tokens starts inside a block, its earlier rows keep their
// codes unless the scale has to grow; then they are rounded once more:
//   code' = e4m3(e4m3(code) old / s),  pe'' = bf16(pe' old / s).
// A power of two costs E4M3 no precision (its values are floating) and makes
// every step but the one rounding exact.
//
// Bound: HBM and, for a decode step's few rows, launch and load latency.  1152
// bytes are read and 640 written a token.  Measured: 64 tokens 2.1 us, 2.9 where
// 64 positions share a scale; 16K prompt tokens in blocks of 16 (29 MB) 9.8 us,
// 3.0 TB/s, most of it the first loads' latency and the launch of 1100 CTAs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "append_plan.h"
#include "attend_fp8.cuh"

namespace mla {

constexpr int kAppendThreads = 256;
constexpr int kMinScaleExp = -40;

// log2 of the smallest scale that holds `amax` (>= 0, finite).
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.f)) return kMinScaleExp;
  int k;
  const float m = frexpf(amax, &k);         // amax = m 2^k, m in [1/2, 1); 448 = 0.875 2^9
  return max(k - (m <= 0.875f ? 9 : 8), kMinScaleExp);
}

// How many of f(1) .. f(n_seq), which do not fall, are at most i.  Every lane
// probes one point of the range that is left (log32 n_seq rounds of loads).
template <typename F>
__device__ __forceinline__ int count_at_most(F f, int n_seq, int i, int lane) {
  int lo = 0, hi = n_seq;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int k = lo + (lane + 1) * step;  // f(k) <= i: the answer is at least k
    const uint32_t yes = __ballot_sync(0xffffffffu, k <= hi && f(min(k, n_seq)) <= i);
    const int n = __popc(yes);             // a prefix of the lanes
    lo += n * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

struct AppendArgs {
  const __nv_bfloat16* kv_new;  // [N, 512]
  const __nv_bfloat16* pe_new;  // [N, 64]
  const int32_t* cu_rows;       // [n_seq + 1]
  const int32_t* start_pos;     // [n_seq]
  const int32_t* cache_slot;    // [n_seq] or null
  uint8_t* kv8;
  __nv_bfloat16* pe8;
  float* kv_scale;
  int N, n_seq, S_max, n_slots, shift, n_blocks;
};

// A warp's lane holds columns 8 lane.. and 256 + 8 lane.. of a latent row.
struct LatentRow {
  uint4 v[2];
};
__device__ __forceinline__ LatentRow load_row(const __nv_bfloat16* row, int lane) {
  const uint4* p = reinterpret_cast<const uint4*>(row) + lane;
  return {{__ldg(p), __ldg(p + 32)}};
}

// Largest finite magnitude of the row (all lanes).
__device__ __forceinline__ float row_amax(const LatentRow& r) {
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t w[4] = {r.v[u].x, r.v[u].y, r.v[u].z, r.v[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) m = max(m, lo);
      if (hi < 0x7f80u) m = max(m, hi);
    }
  }
  return __uint_as_float(__reduce_max_sync(0xffffffffu, m) << 16);
}

// Two floats to E4M3 codes; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  return c | (isinf(a) ? 0x7fu : 0u) | (isinf(b) ? 0x7f00u : 0u);
}

__device__ __forceinline__ void store_row(const AppendArgs& a, int slot, int pos, const LatentRow& r, uint32_t pe2,
                                          float inv, int lane) {
  const size_t at = (size_t)slot * a.S_max + pos;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t w[4] = {r.v[u].x, r.v[u].y, r.v[u].z, r.v[u].w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = codes2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
    reinterpret_cast<uint2*>(a.kv8 + at * kDl)[32 * u + lane] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
  reinterpret_cast<uint32_t*>(a.pe8 + at * kDr)[lane] =
      pack_bf16x2(__uint_as_float(pe2 << 16) * inv, __uint_as_float(pe2 & 0xffff0000u) * inv);
}

__device__ __forceinline__ uint32_t load_pe(const __nv_bfloat16* row, int lane) {
  return __ldg(reinterpret_cast<const uint32_t*>(row) + lane);
}

__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

// Sixteen E4M3 codes times a factor, rounded to E4M3 again.
__device__ __forceinline__ uint4 recode16(const uint4& v, float ratio) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_e4m3x2(w[i] & 0xffffu), b = unpack_e4m3x2(w[i] >> 16);
    o[i] = (uint32_t)codes2(a.x * ratio, a.y * ratio) | ((uint32_t)codes2(b.x * ratio, b.y * ratio) << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t rescale_pe(uint32_t pe2, float ratio) {
  return pack_bf16x2(__uint_as_float(pe2 << 16) * ratio, __uint_as_float(pe2 & 0xffff0000u) * ratio);
}

// A scale a token: a warp per token, its row held in registers between the
// maximum and the rounding.
__global__ void __launch_bounds__(kAppendThreads)
append_fp8_rows_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, i = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.N) return;
  const LatentRow r = load_row(a.kv_new + (size_t)i * kDl, lane);  // in flight during the search
  const uint32_t pe2 = load_pe(a.pe_new + (size_t)i * kDr, lane);
  const int seq = count_at_most([&](int q) { return __ldg(a.cu_rows + q); }, a.n_seq, i, lane);
  if (seq >= a.n_seq) return;  // behind the last sequence
  const int first = __ldg(a.cu_rows + seq);
  const long long at = (long long)__ldg(a.start_pos + seq) + (i - first);
  const int slot = a.cache_slot ? __ldg(a.cache_slot + seq) : seq;
  if (i < first || at < 0 || at >= a.S_max || slot < 0 || slot >= a.n_slots) return;
  const int e = scale_exponent(row_amax(r));
  store_row(a, slot, (int)at, r, pe2, exp2_int(-e), lane);
  if (lane == 0) a.kv_scale[(size_t)slot * a.n_blocks + at] = exp2_int(e);
}

// Shared scales: a CTA per block of positions, all warps at its rows, up to
// kHold rows of a warp held in registers between the maximum and the rounding
// (the others are read twice, the second time from L1 or L2): two where a block
// has no more (16 positions), and six CTAs an SM then, else four.
// (Which block a CTA takes: append_plan.h.)

template <int kHold>
__global__ void __launch_bounds__(kAppendThreads, kHold == 2 ? 6 : 4)
append_fp8_blocks_kernel(const AppendArgs a) {
  constexpr int kWarps = kAppendThreads / 32;
  __shared__ float tops[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = (int)blockIdx.x;
  auto first_cta = [&](int q) { return append_first_cta(__ldg(a.cu_rows + q), a.N, q, a.shift); };
  const int seq = count_at_most(first_cta, a.n_seq, at, lane);
  if (seq >= a.n_seq) return;
  const int row0 = __ldg(a.cu_rows + seq), row1 = min(__ldg(a.cu_rows + seq + 1), a.N), start = __ldg(a.start_pos + seq);
  const int slot = a.cache_slot ? __ldg(a.cache_slot + seq) : seq;
  if (row0 < 0 || row0 >= row1 || slot < 0 || slot >= a.n_slots) return;
  AppendSpan span;
  if (!append_span(at - first_cta(seq), start, row1 - row0, a.S_max, a.shift, &span)) return;
  const int block0 = span.block0, p0 = span.p0, count = span.p1 - p0, earlier = p0 - block0;
  const __nv_bfloat16* kv = a.kv_new + ((long long)row0 + (p0 - (long long)start)) * kDl;
  const __nv_bfloat16* pe = a.pe_new + ((long long)row0 + (p0 - (long long)start)) * kDr;
  float* sp = a.kv_scale + (size_t)slot * a.n_blocks + (p0 >> a.shift);
  LatentRow held[kHold];
  uint32_t held_pe[kHold];
#pragma unroll
  for (int u = 0; u < kHold; ++u) {
    const int r = warp + u * kWarps;
    held[u] = r < count ? load_row(kv + (size_t)r * kDl, lane) : LatentRow{};
    held_pe[u] = r < count ? load_pe(pe + (size_t)r * kDr, lane) : 0u;
  }
  const float old = earlier > 0 ? *sp : 0.f;
  float top = 0.f;
#pragma unroll
  for (int u = 0; u < kHold; ++u) top = fmaxf(top, row_amax(held[u]));
  for (int r = warp + kHold * kWarps; r < count; r += kWarps) top = fmaxf(top, row_amax(load_row(kv + (size_t)r * kDl, lane)));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w]);
  const float s = fmaxf(exp2_int(scale_exponent(top)), old);
  const float inv = 1.f / s;
  if (earlier > 0 && s != old) {
    const float ratio = old / s;
    for (int r = warp; r < earlier; r += kWarps) {
      const size_t row = (size_t)slot * a.S_max + block0 + r;
      uint4* c = reinterpret_cast<uint4*>(a.kv8 + row * kDl) + lane;
      uint32_t* q = reinterpret_cast<uint32_t*>(a.pe8 + row * kDr) + lane;
      const uint4 codes = *c;
      const uint32_t pe2 = *q;
      *c = recode16(codes, ratio);
      *q = rescale_pe(pe2, ratio);
    }
  }
#pragma unroll
  for (int u = 0; u < kHold; ++u) {
    const int r = warp + u * kWarps;
    if (r < count) store_row(a, slot, p0 + r, held[u], held_pe[u], inv, lane);
  }
  for (int r = warp + kHold * kWarps; r < count; r += kWarps)
    store_row(a, slot, p0 + r, load_row(kv + (size_t)r * kDl, lane), load_pe(pe + (size_t)r * kDr, lane), inv, lane);
  if (threadIdx.x == 0) *sp = s;  // (everyone has read it: the barrier)
}

}  // namespace mla
