// Work partition of the 8-bit append with shared scales (append_fp8.cuh), shared
// by the kernel and a host-side test.
//
// A CTA takes one block of positions of one sequence.  Sequence q's blocks are
// the CTAs from cu[q] / block + 2 q on: L tokens touch at most L / block + 2
// blocks, so they end before the next sequence's, and the CTAs behind them
// have nothing to do.
#pragma once

#if defined(__CUDACC__)
#define MLA_APPEND_FN __host__ __device__ __forceinline__
#else
#define MLA_APPEND_FN inline
#endif

namespace mla {

MLA_APPEND_FN int append_blocks_grid(int N, int n_seq, int shift) { return (N >> shift) + 2 * n_seq; }

// The first CTA of sequence q, whose rows begin at `row`.
MLA_APPEND_FN int append_first_cta(int row, int N, int q, int shift) {
  return ((row < 0 ? 0 : (row > N ? N : row)) >> shift) + 2 * q;
}

// Positions [p0, p1) of the block that begins at block0.
struct AppendSpan {
  int block0, p0, p1;
};

// What the CTA `index` places behind its sequence's first writes of `rows` rows
// that go to positions `start` ..; false: nothing.  (index < 0: rows before the
// first sequence's; no position inside the cache: nothing, although `start` may
// lie in its last block, behind S_max.)
MLA_APPEND_FN bool append_span(int index, int start, int rows, int S_max, int shift, AppendSpan* s) {
  const int pos0 = start > 0 ? start : 0;
  const long long end = (long long)start + rows;
  const int pos1 = (int)(end < S_max ? end : S_max);
  if (index < 0 || pos0 >= pos1) return false;
  const long long block0 = (long long)((pos0 >> shift) + index) << shift;
  if (block0 >= pos1) return false;
  const long long next = block0 + (1 << shift);
  s->block0 = (int)block0;
  s->p0 = block0 > pos0 ? (int)block0 : pos0;
  s->p1 = next < pos1 ? (int)next : pos1;
  return true;
}

}  // namespace mla
