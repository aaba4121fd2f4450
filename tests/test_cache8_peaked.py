"""The 8-bit cache's attention where a few positions take most of a softmax (an
attention sink, a top-k in falling order): the many small weights beside them
still count.

Tolerance of a mix (`mix_bound`).  A weight w_t (times its position's scale)
enters as two numbers of four and three significant bits, in units that put the
largest of its tile (128 slots) above 2, or the sum over the j tiles before it
above 2 (j + 1):
  from 2^-6 on, what the first number leaves is at most 2^-4 of w, and the
    second's half step 2^-4 of that again: 2^-8 of w, and fp16's 2^-11 before it;
  below, the first number's half step is 2^-10, and the second's half step of
    anything up to that 2^-14 (fp16's 2^-17 before it): 2^-15 of the tile's
    largest, or of the sum before it over j + 1;
  a tile whose weights lie below 2^-32 of the split's largest is held as one at
    2^-32 of it.
The small weights' term adds up to 2^-8 of a tile's largest over a tile, whatever
the number of tiles.  Then the output's bf16 rounding, 2^-8 of it, and what the
scores are off by (`score_bound` of the other tests, in every weight and in the
row sum).
"""
import math

import pytest
import torch

from tests import cache8_refs as ref
import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, bf, gen, parts, score_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


def mix_bound(x, mix, cache, slot, t, tile, n_tiles, sb):
    """[h, 512]: see above; x [h, T] scores of the split's valid positions t, tile [T] the tile of each."""
    c, _ = ref.rows_of(cache, slot, t)
    code = ref.e4m3_values(cache[0][slot, t]).abs()
    p = torch.softmax(x, 1)
    v = p * cache[2][slot, t // cache[3]].double()
    top = torch.zeros(x.shape[0], n_tiles, dtype=torch.float64, device=x.device)
    top = top.scatter_reduce(1, tile.expand_as(v), v, "amax")
    sums = torch.zeros_like(top).scatter_add(1, tile.expand_as(v), v)
    before = (sums.cumsum(1) - sums) / torch.arange(1, n_tiles + 1, device=x.device)
    small = 2.0 ** -15 * (top + before)[:, tile] + 2.0 ** -46 * v.amax(1, keepdim=True)
    return 2.0 ** -8 * mix.abs() + (1.125 * 2.0 ** -8 + 2.0 ** -18 + 2 * sb.amax(1, keepdim=True)) * (p @ c.abs()) + 1.125 * (small @ code)


def check(q_lat, q_pe, c, end, idx, slots, rows):
    """Rows of the attention against 64 bits."""
    R, h = q_lat.shape[:2]
    K = idx.shape[1]
    n = mla.num_splits_fp8(R, K, h)
    span = -(-(-(-K // 128)) // n) * 128
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE, cache_slot=slots, d_status=status)
    assert int(status) == 0
    for b in rows:
        slot = int(slots[b])
        for s in range(n):
            part = idx[b, s * span:(s + 1) * span]
            ok = (part >= 0) & (part < int(end[b]))
            t, tile = part[ok].long(), torch.arange(part.numel(), device=DEV)[ok] // 128
            x, mix, want = ref.attend(q_lat[b], q_pe[b], parts(c), slot, t, SCALE)
            sb = score_bound(q_lat[b], q_pe[b], parts(c), slot, t, 2.0 ** -17)
            assert bool(((lse[b, s].double() - want).abs() <= sb.amax(1) + 2.0 ** -20 * want.abs()).all())
            bound = mix_bound(x, mix, parts(c), slot, t, tile, -(-part.numel() // 128), sb)
            off = (o[b, s].double() - mix).abs()
            assert bool((off <= bound).all()), (b, s, float((off / bound).max()))
    return n


def cache_of(g, S, block, b):
    """One slot: latents around a common vector (lost weight then shows), rotary keys b_t in the first column."""
    c = mla.Fp8Cache.empty(1, S, block)
    x = torch.randn(1, 512, generator=g, device=DEV) + torch.randn(S, 512, generator=g, device=DEV)
    r = torch.zeros(S, 64, device=DEV)
    r[:, 0] = b
    mla.mla_append_fp8(c, x.to(bf), r.to(bf), torch.tensor([0, S], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    return c


def queries(g, R, h, a):
    """Latent queries that hardly matter, and a_h in the first rotary column."""
    q_pe = torch.zeros(R, h, 64, device=DEV)
    q_pe[:, :, 0] = a
    return (torch.randn(R, h, 512, generator=g, device=DEV) * 0.02).to(bf), q_pe.to(bf)


def sink(g, h, K, spread):
    """Rotary keys and queries: position 0 takes 0.3 to 0.98 of a head's softmax over K positions, the others are near equal."""
    b = spread * torch.randn(K, generator=g, device=DEV)
    b[0] = 32
    share = torch.linspace(0.3, 0.98, h, device=DEV)
    return b, torch.log((K - 1) * share / (1 - share)) / (32 * SCALE)


def orders(g, b):
    """Index rows: the largest first, last, in a random place, falling, rising."""
    K = b.numel()
    mixed = [torch.randperm(K, generator=g, device=DEV) for _ in range(3)]
    first, last = (m[m != 0] for m in mixed[:2])
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    fall = b.argsort(descending=True)
    return torch.stack([torch.cat([zero, first]), torch.cat([last, zero]), mixed[2], fall, fall.flip(0)]).to(torch.int32)


@pytest.mark.parametrize("h", [128, 64])
@pytest.mark.parametrize("K,block,R,spread", [
    (2048, 1, 76, 0.25),   # one split
    (2048, 64, 76, 0.0),   # the others exactly equal
    (8192, 16, 76, 0.25),  # many tiles in one split
    (8192, 1, 76, 0.0),
    (2048, 16, 5, 0.25),   # several splits
])
def test_a_sink_leaves_the_others_their_weight(h, K, block, R, spread):
    g = gen(K + h + block)
    b, a = sink(g, h, K, spread)
    c = cache_of(g, K, block, b)
    idx = orders(g, b).repeat(-(-R // 5), 1)[:R].contiguous()
    end, slots = torch.full((R,), K, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    n = check(*queries(g, R, h, a), c, end, idx, slots, range(5))
    assert (n == 1) == (R == 76)


@pytest.mark.parametrize("h", [128, 33])
@pytest.mark.parametrize("K", [2048, 8192])
@pytest.mark.parametrize("sd", [1.0, 3.0, 8.0, 30.0])
def test_scores_of_any_spread_in_any_order(h, K, sd):
    """Normal scores of up to 30 nats' deviation, falling, rising and mixed (a tile's largest far below the last's, or far above)."""
    g = gen(int(10 * sd) + h)
    b = torch.randn(K, generator=g, device=DEV)
    c = cache_of(g, K, 1, b)
    R = 76
    idx = orders(g, b).repeat(-(-R // 5), 1)[:R].contiguous()
    idx[2, ::3] = -1  # holes
    idx[2, 640:900] = -1  # and two tiles of nothing else
    end, slots = torch.full((R,), K, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    check(*queries(g, R, h, sd / SCALE * torch.linspace(0.5, 1, h, device=DEV)), c, end, idx, slots, range(5))


@pytest.mark.parametrize("h", [128, 40])
@pytest.mark.parametrize("loud", [2.0 ** 6, 2.0 ** 12])
def test_blocks_of_far_larger_scales(h, loud):
    """Quiet positions that share a scale with a loud one which is not selected: their codes are small, their weights (times the
    scale) the row's largest."""
    g = gen(88)
    K, S, R = 2000, 2048, 76
    c = cache_of(g, S, 16, 0.25 * torch.randn(S, generator=g, device=DEV))
    big = torch.randn(1, 512, generator=g, device=DEV) * loud
    for at in (48, 1024):  # the blocks' scales grow: rows before the loud one are rounded again
        mla.mla_append_fp8(c, big.to(bf), torch.zeros(1, 64, dtype=bf, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                           torch.tensor([at + 9], dtype=torch.int32, device=DEV))
    idx = torch.randperm(S, generator=g, device=DEV)
    idx = idx[(idx != 57) & (idx != 1033)][:K].to(torch.int32).expand(R, K).contiguous()
    end, slots = torch.full((R,), S, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    check(*queries(g, R, h, torch.full((h,), 10.0, device=DEV)), c, end, idx, slots, range(2))


@pytest.mark.parametrize("R", [76, 4])
@pytest.mark.parametrize("K", [2048, 8192])
def test_the_step_with_a_sink(R, K):
    """The whole decode under the framework's bound for it, sinks first and last."""
    g = gen(5 + K)
    h = 128
    b, a = sink(g, h, K, 0.0)
    c = cache_of(g, K, 1, b)
    idx = orders(g, b).repeat(-(-R // 5), 1)[:R].contiguous()
    end, slots = torch.full((R,), K, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    _, q_pe = queries(g, R, h, a)
    qn = (0.05 * torch.randn(R, h, 128, generator=g, device=DEV)).to(bf)
    w = (torch.randn(h * 256, 512, generator=g, device=DEV) * 512 ** -0.5).to(bf)
    out = mla.mla_sparse_decode_fp8(qn, q_pe, c, end, idx, w, SCALE, cache_slot=slots)
    some = list(range(min(R, 5)))
    want, _ = ref.decode(qn[some], q_pe[some], parts(c), slots, end, idx[some], w, SCALE)
    assert float((out[some].double() - want).abs().max()) <= 1e-2 * float(want.abs().max()) + 1e-3
