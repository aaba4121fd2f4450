"""The work partition of the 8-bit append with shared scales
(csrc/append_plan.h), checked on the host against a plain walk over the rows:
every row inside the cache is written by one CTA, in the block that holds it, and
no CTA reaches outside its block or the cache, wherever a sequence's rows begin
(the first may not begin at row 0), wherever they go (before the cache, behind
it), and for row offsets that are no such list.  g++ compiles the header into a
small checker (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER_DIR = os.path.join(ROOT, "sparse_latent_attention_absorb_b200", "csrc")

CHECKER = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "append_plan.h"
using namespace mla;

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  long bad = 0, cases = 0, rows_seen = 0;
  for (int it = 0; it < 200000; ++it) {
    const int n = pick(1, 4), S = pick(1, 90), shift = pick(0, 7), block = 1 << shift;
    std::vector<int> cu(n + 1), start(n);
    const bool list = pick(0, 9) > 0;  // else: any numbers
    cu[0] = pick(0, 2) ? 0 : pick(0, 300);
    for (int q = 0; q < n; ++q) cu[q + 1] = cu[q] + (pick(0, 3) ? pick(0, 40) : 0);
    const int N = cu[n] + pick(0, 20) + 1;
    if (!list) for (int& c : cu) c = pick(-300, 600);
    for (int& s : start) s = pick(0, 5) ? pick(-60, S + 150) : (pick(0, 1) ? 2147483647 - pick(0, 50) : -2147483647 - 1 + pick(0, 50));
    std::vector<std::vector<int>> hits(n);
    if (list) for (int q = 0; q < n; ++q) hits[q].assign(cu[q + 1] - cu[q], 0);
    for (int at = 0; at < append_blocks_grid(N, n, shift); ++at) {
      int seq = 0;  // how many of the first CTAs of sequences 1 .. n are at most this one
      for (int k = 1; k <= n; ++k) seq += append_first_cta(cu[k], N, k, shift) <= at;
      for (int s = list ? seq : 0; s < (list ? seq + 1 : n); ++s) {  // of no list, any sequence may be found
        if (s >= n) continue;
        const int row0 = cu[s], row1 = cu[s + 1] < N ? cu[s + 1] : N;
        if (row0 < 0 || row0 >= row1) continue;
        AppendSpan p;
        if (!append_span(at - append_first_cta(row0, N, s, shift), start[s], row1 - row0, S, shift, &p)) continue;
        // whole: the block lies in the cache, the positions in it, their rows in the sequence's
        if (p.block0 < 0 || p.block0 % block || p.p0 < p.block0 || p.p1 <= p.p0 || p.p1 > p.block0 + block || p.p1 > S) ++bad;
        const long long r0 = (long long)p.p0 - start[s], r1 = (long long)p.p1 - start[s];
        if (r0 < 0 || r1 > row1 - row0) { ++bad; continue; }
        if (list) for (long long r = r0; r < r1; ++r) ++hits[s][(size_t)r];
      }
    }
    if (list)
      for (int q = 0; q < n; ++q)
        for (size_t r = 0; r < hits[q].size(); ++r) {
          const long long t = (long long)start[q] + (long long)r;
          const int want = t >= 0 && t < S;
          rows_seen += want;
          if (hits[q][r] != want) ++bad;
        }
    ++cases;
  }
  std::printf("%ld cases, %ld rows, %ld violations\n", cases, rows_seen, bad);
  return bad == 0 ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_append_partition_is_exact(tmp_path):
    src = tmp_path / "plan_check.cpp"
    src.write_text(CHECKER)
    exe = tmp_path / "plan_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", HEADER_DIR, "-o", str(exe), str(src)], check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr
    assert " 0 violations" in p.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 2, 16, 128])
def test_append_leaves_out_rows_before_the_first_sequence_and_positions_behind_the_cache(block):
    """Row lists that begin behind row 0, and runs that begin behind the cache's end inside its last block, next to scales that
    are not set (0): exact, and nothing else is touched."""
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    import torch
    from tests import cache8_refs as ref
    import sparse_latent_attention_absorb_b200 as mla
    from tests.test_cache8 import DEV, bf, gen, make_cache
    g = gen(block)
    S = 70
    c = make_cache(g, 5, S, block)
    c.scale[0], c.scale[1] = 0, 0
    c.scale[3] = 0
    cu, start = [90, 100, 140, 140, 160, 163], [0, 75, 3, 71, 69]
    N = 170
    x, r = torch.randn(N, 512, generator=g, device=DEV).to(bf), torch.randn(N, 64, generator=g, device=DEV).to(bf)
    want = [t.clone() for t in (c.kv, c.pe, c.scale)]
    ref.append(*want, block, x, r, cu, start)
    for _ in range(5):  # the order of the CTAs may not matter
        got = mla.Fp8Cache(c.kv.clone(), c.pe.clone(), c.scale.clone(), block)
        mla.mla_append_fp8(got, x, r, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(start, dtype=torch.int32, device=DEV))
        assert torch.equal(got.kv, want[0]) and torch.equal(got.scale, want[2])
        assert torch.equal(got.pe.view(torch.int16), want[1].view(torch.int16))
