"""Eviction by accumulated attention weight on the GPU, and the cache's
operators one after another as a serving loop uses them.  Everything that an
eviction writes is copied, counted, or an 8-bit value rounded once more by a
power of two, so every comparison is exact."""
import math

import pytest
import torch

from tests import cache8_refs as ref
import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, bf, decode_inputs, gen, make_cache, parts, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


def totals(g, B, S):
    acc = torch.exp(2 * torch.randn(B, S, generator=g, device=DEV)) * (torch.rand(B, S, generator=g, device=DEV) < 0.6)
    return acc.contiguous()


def expected(src, acc, end, keep, recent, to):
    """The buffers after the eviction: (kv, pe, scale or None, acc, kept, new_end); `to` are the outputs before it."""
    kv, pe, scale, block = src
    okv, ope, oscale = (None if t is None else t.clone() for t in to[:3])
    oacc = torch.zeros_like(acc)
    B, S = acc.shape
    kept = torch.full((B, keep), -1, dtype=torch.int32, device=DEV)
    new_end = torch.zeros(B, dtype=torch.int32, device=DEV)
    for b in range(B):
        n = max(0, min(int(end[b]), S))
        at = ref.keep_positions(acc[b, :n].tolist(), n, keep, recent)
        t = torch.tensor(at, dtype=torch.long, device=DEV)
        m = len(at)
        new_end[b] = m
        kept[b, :m] = t.to(torch.int32)
        oacc[b, :m] = acc[b, t]
        if scale is None:
            okv[b, :m], ope[b, :m] = kv[b, t], pe[b, t]
            continue
        s = scale[b, t // block]
        for k in range(-(-m // block)):
            rows = slice(k * block, min(m, (k + 1) * block))
            top = float(s[rows].max())
            oscale[b, k] = top
            f = (s[rows].double() / top)[:, None]
            okv[b, rows] = ref.e4m3_codes(ref.e4m3_values(kv[b, t[rows]]) * f)
            ope[b, rows] = (pe[b, t[rows]].double() * f).to(bf)
    return okv, ope, oscale, oacc, kept, new_end


def run(c, acc, end, keep, recent, in_place):
    """Evicts and compares; c is an Fp8Cache, or (kv, pe) in bf16."""
    fp8 = isinstance(c, mla.Fp8Cache)
    src = parts(c) if fp8 else (*c, None, 1)
    B, S = acc.shape
    if in_place:
        to, acc_to = src, acc
    else:
        to = tuple(None if t is None else torch.full_like(t, 3) for t in src[:3])
        acc_to = torch.full_like(acc, -1)
    want = expected(tuple(t.clone() if isinstance(t, torch.Tensor) else t for t in src), acc.clone(), end, keep, recent, to)
    if fp8 and in_place:
        kept, n = mla.mla_evict_fp8(c, acc, end, keep, recent)
    elif fp8:
        kept, n = mla.mla_evict_fp8(c, acc, end, keep, recent, cache_out=mla.Fp8Cache(*to, c.block), acc_out=acc_to)
    elif in_place:
        kept, n = mla.mla_evict(*c, acc, end, keep, recent)
    else:
        kept, n = mla.mla_evict(*c, acc, end, keep, recent, kv_out=to[0], pe_out=to[1], acc_out=acc_to)
    assert torch.equal(kept, want[4]) and torch.equal(n, want[5])
    assert torch.equal(acc_to.view(torch.int32), want[3].view(torch.int32))
    for b in range(B):  # rows behind the last kept one: left as they were
        for got, exp in zip(to[:2], want[:2]):
            a, e = got[b], exp[b]
            assert torch.equal(a.view(torch.uint8), e.view(torch.uint8))
    if fp8:
        assert torch.equal(to[2], want[2])
    return kept, n


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("block", [0, 1, 4, 128])
@pytest.mark.parametrize("B,S,keep,recent", [
    (1, 1, 1, 0), (2, 40, 7, 7), (3, 300, 129, 0), (5, 700, 256, 100), (2, 700, 700, 5), (2, 5000, 1, 1), (3, 5000, 2500, 300)])
def test_eviction_is_exact(B, S, keep, recent, block, in_place):
    g = gen(B * 1000 + keep + block)
    c = make_cache(g, B, S, block) if block else (torch.randn(B, S, 512, generator=g, device=DEV).to(bf),
                                                  torch.randn(B, S, 64, generator=g, device=DEV).to(bf))
    end = torch.randint(0, S + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    end[0] = S
    if B > 2:
        end[1], end[2] = -3, S + 50
    run(c, totals(g, B, S), end, keep, recent, in_place)


@pytest.mark.parametrize("B,S", [(1, 20000), (2, 9000), (12, 17000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_rows(B, S, in_place):
    """Rows that several CTAs share."""
    g = gen(S)
    c = (torch.randn(B, S, 512, generator=g, device=DEV).to(bf), torch.randn(B, S, 64, generator=g, device=DEV).to(bf))
    end = torch.randint(S // 2, S + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    run(c, totals(g, B, S), end, S // 3, 100, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_ties_zeros_and_what_is_not_finite(in_place):
    B, S = 6, 600
    g = gen(9)
    c = make_cache(g, B, S, 8)
    acc = torch.zeros(B, S, device=DEV)
    acc[1] = -0.0
    acc[1, ::2] = 0.0                       # the two zeros are one weight
    acc[2] = 1.5
    acc[3] = torch.randint(0, 4, (S,), generator=g, device=DEV).float()
    acc[4, ::5], acc[4, 3::7], acc[4, 1::11] = math.nan, math.inf, -math.inf
    acc[5] = -torch.rand(S, generator=g, device=DEV) * 1e-30
    end = torch.full((B,), S, dtype=torch.int32, device=DEV)
    run(c, acc, end, 250, 40, in_place)


def test_eviction_in_a_graph_on_another_stream():
    g = gen(12)
    c = make_cache(g, 4, 800, 16)
    to = mla.Fp8Cache.empty(4, 800, 16)
    acc, acc_to = totals(g, 4, 800), torch.empty(4, 800, device=DEV)
    end = torch.full((4,), 800, dtype=torch.int32, device=DEV)
    kept, n = torch.empty(4, 300, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.mla_evict_fp8(c, acc, end, 300, 50, cache_out=to, acc_out=acc_to, kept=kept, new_end=n)
    for _ in range(2):
        kept.zero_()
        acc = acc.copy_(totals(g, 4, 800))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.default_stream().wait_stream(side)
        want = expected(parts(c), acc, end, 300, 50, parts(to)[:3])
        assert torch.equal(kept, want[4]) and torch.equal(acc_to, want[3]) and torch.equal(to.kv, want[0])


@pytest.mark.parametrize("block", [1, 16])
def test_a_serving_loop(block):
    """Prompts, decode steps with their totals, an eviction, and decode steps on what it left: every decode against the 64-bit
    decode of what the cache holds."""
    g = gen(77)
    B, S, K = 3, 600, 200
    c = mla.Fp8Cache.empty(B, S, block)
    end = torch.tensor([411, 96, 250], dtype=torch.int32, device=DEV)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(end, 0)
    n = int(cu[-1])
    mla.mla_append_fp8(c, torch.randn(n, 512, generator=g, device=DEV).to(bf), torch.randn(n, 64, generator=g, device=DEV).to(bf), cu,
                       torch.zeros(B, dtype=torch.int32, device=DEV))
    acc = torch.zeros(B, S, device=DEV)
    one = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    w = decode_inputs(g, B, 128)[2]
    for step in range(6):
        mla.mla_append_fp8(c, torch.randn(B, 512, generator=g, device=DEV).to(bf), torch.randn(B, 64, generator=g, device=DEV).to(bf), one, end)
        end = end + 1
        qn, qp, _ = decode_inputs(g, B, 128)
        idx = selection(g, end.tolist(), K, S)
        lse = torch.empty(B, 128, device=DEV)
        out = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE, lse_out=lse)
        want, want_lse = ref.decode(qn, qp, parts(c), torch.arange(B), end, idx, w, SCALE)
        assert float((out.double() - want).abs().max()) <= 1e-2 * float(want.abs().max()) + 1e-3
        assert float((lse.double() - want_lse).abs().max()) <= 1e-2
        before = acc.sum(1)
        mla.mla_accumulate_weights_fp8(mla.mla_absorb_q(qn, w), qp, c, end, idx, SCALE, lse, acc)
        # every head's weights sum to one, to a weight's 2^-20 and what the totals' bf16 q_lat moves a score by: 0.072 * 0.5 * 2^-9 *
        # sqrt(512) = 1.6e-3 for one, of either sign, over 128 heads and 200 positions
        torch.testing.assert_close(acc.sum(1) - before, torch.full((B,), 128.0, device=DEV), rtol=1e-3, atol=0)
        if step == 2:
            kept, end = run(c, acc, end, 150, 30, in_place=True)
            assert end.tolist() == [150, 99, 150] and bool((kept[0] >= 0).all())
            assert float(acc[0, 150:].abs().sum()) == 0
