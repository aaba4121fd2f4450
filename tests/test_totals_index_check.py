"""The opt-in index checks reach the weight totals, where a repeated index adds
its weight twice: over both caches, reported in the status word, and off by
default."""
import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from tests.test_cache8 import DEV, SCALE, bf, gen, make_cache, query, selection

pytestmark = pytest.mark.gpu

BAD_INDEX = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


@pytest.mark.parametrize("fp8", [True, False])
def test_checks_run_before_the_totals(fp8):
    g = gen(8)
    c = make_cache(g, 2, 300, 4)
    cache = (c,) if fp8 else (torch.randn(2, 300, 512, generator=g, device=DEV).to(bf), torch.randn(2, 300, 64, generator=g, device=DEV).to(bf))
    call = mla.mla_accumulate_weights_fp8 if fp8 else mla.mla_accumulate_weights
    end = torch.tensor([300, 150], dtype=torch.int32, device=DEV)
    idx = selection(g, [300, 150], 100, 300)
    twice = idx.clone()
    twice[1, 17] = twice[1, 60]
    q, lse = query(g, 2, 128), torch.full((2, 128), 6.0, device=DEV)
    alone = call(*q, *cache, end, idx, SCALE, lse, torch.zeros(2, 300, device=DEV))
    prev = mla.set_index_checks(True)
    try:
        for rows, want in ((idx, 0), (twice, BAD_INDEX)):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            acc = call(*q, *cache, end, rows, SCALE, lse, torch.zeros(2, 300, device=DEV), d_status=status)
            assert int(status) == want
            assert torch.equal(acc[0], alone[0]) and (want or torch.equal(acc, alone))
        mla.set_index_checks(False)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        call(*q, *cache, end, twice, SCALE, lse, torch.zeros(2, 300, device=DEV), d_status=status)
        assert int(status) == 0
    finally:
        mla.set_index_checks(prev)
