"""The 8-bit cache's attention over a rotary key that holds an infinity: a head
whose score there is -inf leaves the position out, exactly as if it were masked;
one whose score is +inf or NaN answers NaN, alone."""
import math

import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, gen, make_cache, query, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


@pytest.mark.parametrize("h", [128, 20])
@pytest.mark.parametrize("key", [math.inf, -math.inf])
def test_an_infinite_key_counts_by_its_sign(h, key):
    g = gen(h)
    c = make_cache(g, 1, 500, 4)
    end = torch.tensor([500], dtype=torch.int32, device=DEV)
    idx = selection(g, [500], 300, 500)
    q_lat, q_pe = query(g, 1, h)
    sign = torch.where(torch.rand(h, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    q_pe[0, :, 3] = sign.to(q_pe.dtype)
    masked = idx.clone()
    masked[0, 50] = -1
    c.pe[0, int(idx[0, 50]), 3] = key
    without, lse0 = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, masked, SCALE)
    o, lse = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE)
    n = o.shape[1]
    part = 50 // (-(-(-(-300 // 128)) // n) * 128)  # the split that holds slot 50
    out = sign * (1 if key > 0 else -1) < 0
    assert torch.equal(o[0, :, out], without[0, :, out]) and torch.equal(lse[0, :, out], lse0[0, :, out])
    assert bool(torch.isnan(o[0, part, ~out]).all()) and bool(torch.isnan(lse[0, part, ~out]).all())
    rest = [s for s in range(n) if s != part]
    assert torch.equal(o[0, rest], without[0, rest]) and torch.equal(lse[0, rest], lse0[0, rest])
