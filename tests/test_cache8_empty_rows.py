"""Rows of the 8-bit cache's calls that no index selects anything for, whose
queries nobody has filled (a padded batch): out = 0 and lse = -inf, and the other
rows as they are without them, for NaN and infinities in every query tensor.
Every comparison is exact."""
import math

import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, bf, decode_inputs, gen, make_cache, query, selection

pytestmark = pytest.mark.gpu

EMPTY = [1, 2, 3, 5]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


def rows(g, K):
    """Six rows of two slots; EMPTY: no end, no index, no slot, only indices past the end."""
    c = make_cache(g, 2, 500, 8)
    end = torch.tensor([500, 0, 500, 500, 130, 7], dtype=torch.int32, device=DEV)
    idx = selection(g, [500, 500, 500, 500, 130, 500], K, 500)
    idx[2] = -1
    idx[5] = torch.where(idx[5] < 7, torch.full_like(idx[5], 400), idx[5])
    slots = torch.tensor([0, 1, 0, 2, 1, 1], dtype=torch.int32, device=DEV)
    return c, end, idx, slots


@pytest.mark.parametrize("h", [128, 70, 33])
@pytest.mark.parametrize("K", [90, 400])  # one tile a split, and several
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_of_empty_rows(h, K, bad):
    g = gen(h + K)
    c, end, idx, slots = rows(g, K)
    q_lat, q_pe = query(g, 6, h)
    clean = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE, cache_slot=slots)
    for which in (0, 1):
        q = [q_lat.clone(), q_pe.clone()]
        q[which][EMPTY] = bad
        q[1 - which][EMPTY[0], h // 2, 3] = bad
        o, lse = mla.mla_sparse_attend_fp8(*q, c, end, idx, SCALE, cache_slot=slots)
        assert bool((o[EMPTY] == 0).all()) and bool((lse[EMPTY] == -math.inf).all())
        assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("h", [128, 33])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_the_step_on_empty_rows(h, bad):
    g = gen(h)
    c, end, idx, slots = rows(g, 200)
    qn, qp, w = decode_inputs(g, 6, h)
    lse, lse2 = torch.empty(6, h, device=DEV), torch.empty(6, h, device=DEV)
    clean = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE, cache_slot=slots, lse_out=lse)
    for which in (0, 1):
        q = [qn.clone(), qp.clone()]
        q[which][EMPTY] = bad
        out = mla.mla_sparse_decode_fp8(*q, c, end, idx, w, SCALE, cache_slot=slots, lse_out=lse2)
        assert bool((out[EMPTY] == 0).all()) and bool((lse2[EMPTY] == -math.inf).all())
        assert torch.equal(out, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [True, False])
def test_totals_of_empty_rows(fp8):
    """Nothing is added, whatever the queries and log-sum-exps hold."""
    g = gen(4)
    c = make_cache(g, 3, 300, 4)
    cache = (c,) if fp8 else (torch.randn(3, 300, 512, generator=g, device=DEV).to(bf), torch.randn(3, 300, 64, generator=g, device=DEV).to(bf))
    end = torch.tensor([0, 300, 250], dtype=torch.int32, device=DEV)
    idx = selection(g, [300, 300, 250], 150, 300)
    idx[1] = -1
    q_lat, q_pe = query(g, 3, 128)
    q_lat[:2], q_pe[:2] = math.nan, math.inf
    lse = torch.full((3, 128), 6.0, device=DEV)
    lse[0], lse[1] = -math.inf, math.nan
    acc = torch.rand(3, 300, generator=g, device=DEV)
    was = acc.clone()
    (mla.mla_accumulate_weights_fp8 if fp8 else mla.mla_accumulate_weights)(q_lat, q_pe, *cache, end, idx, SCALE, lse, acc)
    assert torch.equal(acc[:2], was[:2]) and bool(torch.isfinite(acc[2]).all()) and not torch.equal(acc[2], was[2])
