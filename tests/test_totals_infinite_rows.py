"""Totals of a call with fewer than 128 heads over cached rows that hold
infinities: a position whose scores are -inf in all of its heads weighs 0, as it
does with 128 heads (the rows of the absent heads, zeros times infinity, do not
count)."""
import math

import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, bf, gen, make_cache, query, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


@pytest.mark.parametrize("h", [128, 100, 16, 1])
@pytest.mark.parametrize("fp8", [True, False])
def test_a_position_of_minus_infinite_scores_weighs_nothing(fp8, h):
    g = gen(h)
    c = make_cache(g, 1, 300, 1)
    kv, pe = torch.randn(1, 300, 512, generator=g, device=DEV).to(bf), torch.randn(1, 300, 64, generator=g, device=DEV).to(bf)
    call = mla.mla_accumulate_weights_fp8 if fp8 else mla.mla_accumulate_weights
    cache = (c,) if fp8 else (kv, pe)
    end = torch.tensor([300], dtype=torch.int32, device=DEV)
    idx = selection(g, [300], 200, 300)
    q_lat, q_pe = query(g, 1, h)
    q_pe[:, :, 3] = -1  # every head meets the infinite key with the same sign
    lse = torch.full((1, h), 6.0, device=DEV)
    want = call(q_lat, q_pe, *cache, end, idx, SCALE, lse, torch.ones(1, 300, device=DEV))
    t = int(idx[0, 50])
    (c.pe if fp8 else pe)[0, t, 3] = math.inf
    got = call(q_lat, q_pe, *cache, end, idx, SCALE, lse, torch.ones(1, 300, device=DEV))
    assert float(got[0, t]) == 1.0
    want[0, t] = 1
    assert torch.equal(got, want)
