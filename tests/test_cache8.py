"""The 8-bit latent cache on the GPU: appending to it, the sparse decode over
it and the running totals of attention weight, against plain 64-bit forms
(cache8_refs.py).  The pages keep the latents in bf16, so these operators have
no counterpart there; the decode's steps are those of model.py 595-606 on the
page "Query-key similarity".

Tolerances (eps / 2 of a type is its rounding: bf16 2^-8, E4M3 2^-4):
  codes, scales and rotary parts are exact: every step of an append is a
    division by a power of two and one rounding;
  the mix of mla_sparse_attend_fp8 (`mix_bound`): its own bf16 rounding, 2^-8 of
    each weight (two E4M3 limbs: 2^-4 of what 2^-4 left), and for small weights
    the limbs' grid: E4M3 steps by 2^-9, so a weight is off by 2^-10 where the
    head's largest is at least 2^3: 2^-13 of the largest;
  log-sum-exps and totals follow the scores (`score_bound`): f32 sums of 576
    products, and the query's limbs: exact to 2^-17 of its largest element,
    2^-19 where the second limb is not scaled up;
  the whole decode adds the bf16 rounding of the absorbed query and of the mix:
    the framework's bound for a decode, 1e-2 of the largest output + 1e-3.
"""
import math

import pytest
import torch

from tests import cache8_refs as ref
import sparse_latent_attention_absorb_b200 as mla

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
SCALE = 192.0 ** -0.5
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    mla.load_library()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_cache(g, slots, S, block, loud=True):
    """A filled cache whose tokens differ in size (and whose blocks in scale)."""
    c = mla.Fp8Cache.empty(slots, S, block)
    x = torch.randn(slots, S, 512, generator=g, device=DEV)
    if loud:
        x *= torch.exp2(torch.randint(-3, 4, (slots, S, 1), generator=g, device=DEV).float())
    r = torch.randn(slots, S, 64, generator=g, device=DEV)
    cu = torch.arange(slots + 1, device=DEV, dtype=torch.int32) * S
    mla.mla_append_fp8(c, x.to(bf).view(-1, 512), r.to(bf).view(-1, 64), cu, torch.zeros(slots, dtype=torch.int32, device=DEV))
    return c


def parts(c):
    return c.kv, c.pe, c.scale, c.block


def selection(g, end, K, S, holes=False):
    rows = []
    for e in end:
        e = max(0, min(e, S))
        take = torch.randperm(e, generator=g, device=DEV)[:K].to(torch.int32) if e else torch.empty(0, dtype=torch.int32, device=DEV)
        row = torch.full((K,), -1, dtype=torch.int32, device=DEV)
        row[:take.numel()] = take
        if holes and K > 4:  # padding anywhere, in every form that it may take
            row[torch.randperm(K, generator=g, device=DEV)[:K // 4]] = torch.tensor([-1, S, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                                                                                    device=DEV)[torch.arange(K // 4, device=DEV) % 4]
        rows.append(row)
    return torch.stack(rows)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("block", [1, 2, 8, 64, 128])
@pytest.mark.parametrize("S,new,start", [
    (300, [1, 1, 1], [0, 7, 299]),          # a decode step's tokens
    (300, [5, 0, 131, 1], [3, 9, 64, 128]),  # ragged, one empty
    (517, [517, 200], [0, 317]),            # a whole slot; up to the last position
    (64, [10, 10, 70, 3], [60, -4, -3, 64]),  # rows past either end are left out
])
def test_append_is_exact(block, S, new, start):
    g = gen(11 + block)
    B = len(new)
    c = make_cache(g, B, S, block)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    N = cu[-1] + 3  # three rows behind the last sequence
    x = (torch.randn(N, 512, generator=g, device=DEV) * torch.exp2(torch.randint(-12, 13, (N, 1), generator=g, device=DEV).float())).to(bf)
    r = torch.randn(N, 64, generator=g, device=DEV).to(bf)
    want = [t.clone() for t in (c.kv, c.pe, c.scale)]
    ref.append(*want, block, x, r, cu, start)
    mla.mla_append_fp8(c, x, r, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(start, dtype=torch.int32, device=DEV))
    assert torch.equal(c.kv, want[0]) and torch.equal(c.scale, want[2])
    assert torch.equal(c.pe.view(torch.int16), want[1].view(torch.int16))


@pytest.mark.parametrize("block", [1, 16])
def test_append_extremes(block):
    """Zero rows, infinities and NaN, the largest and the smallest bf16 magnitudes, and a scale that grows late."""
    c = make_cache(gen(5), 1, 64, block)
    x = torch.zeros(6, 512, dtype=bf, device=DEV)
    x[1, 3], x[1, 5], x[1, 7], x[1, 9] = math.inf, -math.inf, math.nan, 2.0
    x[2, 0] = torch.finfo(bf).max
    x[3] = torch.finfo(bf).tiny
    x[4, ::2] = 448.0
    x[5, 1::2] = 450.0
    r = torch.ones(6, 64, dtype=bf, device=DEV)
    want = [t.clone() for t in (c.kv, c.pe, c.scale)]
    for i in range(6):  # a token at a time, as a decode writes them
        ref.append(*want, block, x[i:i + 1], r[i:i + 1], [0, 1], [20 + i])
        mla.mla_append_fp8(c, x[i:i + 1].contiguous(), r[i:i + 1].contiguous(), torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                           torch.tensor([20 + i], dtype=torch.int32, device=DEV))
        a, b = ref.e4m3_values(c.kv), ref.e4m3_values(want[0])
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())
        assert torch.equal(c.scale, want[2]) and torch.equal(c.pe.float(), want[1].float())


def test_append_slots_many_sequences_and_streams():
    g = gen(3)
    c = make_cache(g, 70, 40, 4)
    n = 2000  # single tokens of more sequences than a warp's first probe tells apart
    slots = torch.randint(-2, 72, (n,), generator=g, device=DEV, dtype=torch.int32)
    start = torch.full((n,), 40, dtype=torch.int32, device=DEV)  # nowhere, but for one sequence a slot
    for s in range(70):
        hit = (slots == s).nonzero()
        if len(hit):
            start[hit[0, 0]] = s % 40
    x, r = torch.randn(n, 512, generator=g, device=DEV).to(bf), torch.randn(n, 64, generator=g, device=DEV).to(bf)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    want = [t.clone() for t in (c.kv, c.pe, c.scale)]
    ref.append(*want, 4, x, r, cu.tolist(), start.tolist(), slots.tolist())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.mla_append_fp8(c, x, r, cu, start, cache_slot=slots)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c.kv, want[0]) and torch.equal(c.scale, want[2]) and torch.equal(c.pe, want[1])


@pytest.mark.parametrize("block", [2, 16, 128])
def test_append_many_ragged_sequences(block):
    """Runs of 0 to 40 tokens that start anywhere, over both ends too: a block is written by one run, whole or in part."""
    g = gen(17 + block)
    n = 150
    c = make_cache(g, n, 60, block)
    new = torch.randint(0, 41, (n,), generator=g, device=DEV).tolist()
    start = torch.randint(-10, 65, (n,), generator=g, device=DEV).tolist()
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    N = cu[-1] + 40
    x = (torch.randn(N, 512, generator=g, device=DEV) * torch.exp2(torch.randint(-6, 7, (N, 1), generator=g, device=DEV).float())).to(bf)
    r = torch.randn(N, 64, generator=g, device=DEV).to(bf)
    want = [t.clone() for t in (c.kv, c.pe, c.scale)]
    ref.append(*want, block, x, r, cu, start)
    mla.mla_append_fp8(c, x, r, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(start, dtype=torch.int32, device=DEV))
    assert torch.equal(c.kv, want[0]) and torch.equal(c.scale, want[2])
    assert torch.equal(c.pe.view(torch.int16), want[1].view(torch.int16))


# ------------------------------------------------------------------- attention
def score_bound(q_lat, q_pe, cache, slot, t, limb):
    """How far a score may be from the 64-bit one, [h, t]."""
    c, r = ref.rows_of(cache, slot, t)
    size = q_lat.double().abs() @ c.abs().T + q_pe.double().abs() @ r.abs().T
    return SCALE * (576 * 2.0 ** -24 * size + limb * float(q_lat.abs().max()) * c.abs().sum(1)) + 2.0 ** -20


def check_attend(q_lat, q_pe, c, end, idx, slots):
    """Every row of the step, split by split, against the 64-bit form."""
    R, h = q_lat.shape[:2]
    K, S = idx.shape[1], c.S_max
    n = mla.num_splits_fp8(R, K, h)
    span = -(-(-(-K // 128)) // n) * 128
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE, cache_slot=slots, d_status=status)
    assert o.shape == (R, n, h, 512) and int(status) == 0
    for b in range(R):
        slot = b if slots is None else int(slots[b])
        for s in range(n):
            part = idx[b, s * span:(s + 1) * span]
            t = ref.selected(part, end[b], S) if 0 <= slot < c.n_slots else part[:0].long()
            x, mix, want = ref.attend(q_lat[b], q_pe[b], parts(c), max(0, min(slot, c.n_slots - 1)), t, SCALE)
            got, got_lse = o[b, s].double(), lse[b, s].double()
            if not len(t):
                assert bool((got == 0).all()) and bool((got_lse == -math.inf).all())
                continue
            sb = score_bound(q_lat[b], q_pe[b], parts(c), slot, t, 2.0 ** -17)
            assert bool(((got_lse - want).abs() <= sb.amax(1) + 2.0 ** -20 * want.abs()).all())
            cc, _ = ref.rows_of(parts(c), slot, t)
            p = torch.softmax(x, 1)
            top = (p * c.scale[slot, t // c.block].double()).amax(1, keepdim=True)  # the largest weight of codes
            grid = 2.0 ** -13 * top * ref.e4m3_values(c.kv[slot, t]).abs().sum(0)
            bound = 2.0 ** -8 * mix.abs() + (2.0 ** -8 + 2 * sb.amax(1, keepdim=True)) * (p @ cc.abs()) + grid
            assert bool(((got - mix).abs() <= bound).all()), float(((got - mix).abs() / bound).max())


def query(g, R, h, size=1.0):
    q = (torch.randn(R, h, 512, generator=g, device=DEV) * 0.5 * size).to(bf)
    return q, (torch.randn(R, h, 64, generator=g, device=DEV) * size).to(bf)


@pytest.mark.parametrize("R,h,K,S,block", [
    (1, 128, 1, 1, 1),         # one position
    (1, 1, 2, 50, 2),
    (2, 16, 31, 200, 8),
    (3, 64, 128, 300, 128),    # one tile, one CTA a row
    (3, 65, 129, 300, 64),     # a pair, two tiles
    (2, 127, 1000, 1001, 16),
    (80, 128, 700, 1500, 1),   # several tiles a split
    (150, 40, 520, 900, 4),
])
def test_attend_matches_64_bits(R, h, K, S, block):
    g = gen(100 + K)
    c = make_cache(g, R, S, block)
    end = torch.randint(1, S + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
    idx = selection(g, end.tolist(), K, S, holes=True)
    check_attend(*query(g, R, h), c, end, idx, None)


def test_attend_empty_rows_and_slots():
    g = gen(7)
    c = make_cache(g, 3, 200, 8)
    R = 9
    end = torch.tensor([200, 0, -5, 200, 1, 999, 200, 200, 130], dtype=torch.int32, device=DEV)
    idx = selection(g, [200, 200, 200, 200, 200, 200, 200, 200, 200], 150, 200)
    idx[3] = -1
    slots = torch.tensor([0, 1, 2, 0, 1, 2, -1, 3, 2], dtype=torch.int32, device=DEV)
    for h in (128, 16):
        check_attend(*query(g, R, h), c, end, idx, slots)


@pytest.mark.parametrize("h", [128, 33])
@pytest.mark.parametrize("size", [0.0, 0.05, 3.0, 12.0])
def test_attend_flat_and_sharp_scores(h, size):
    """From equal weights to one position that takes all of it."""
    g = gen(int(10 * size) + h)
    c = make_cache(g, 80, 900, 1)
    end = torch.full((80,), 900, dtype=torch.int32, device=DEV)
    check_attend(*query(g, 80, h, size), c, end, selection(g, end.tolist(), 900, 900), None)


@pytest.mark.parametrize("h", [128, 64])
@pytest.mark.parametrize("up", [True, False])
def test_attend_scores_that_move_along_the_tiles(h, up):
    """Every tile's largest score is far above (below) the last's: references move at every tile, or never again."""
    g = gen(1)
    R, S = 75, 1152
    c = make_cache(g, R, S, 1, loud=False)
    q_lat, q_pe = query(g, R, h, 1.0)
    for b in range(R):  # order each row's positions by the mean score of its heads
        t = torch.arange(S, device=DEV)
        x, _, _ = ref.attend(q_lat[b] * 0 + q_lat[b, :1], q_pe[b] * 0 + q_pe[b, :1], parts(c), b, t, 20 * SCALE)
        order = x[0].argsort(descending=not up)
        for buf in (c.kv, c.pe, c.scale):
            buf[b] = buf[b][order]
    q_lat[:] = q_lat[:, :1] * 20
    q_pe[:] = q_pe[:, :1] * 20
    end = torch.full((R,), S, dtype=torch.int32, device=DEV)
    idx = torch.arange(S, device=DEV, dtype=torch.int32).expand(R, S).contiguous()
    check_attend(q_lat, q_pe, c, end, idx, None)


@pytest.mark.parametrize("h", [128, 20])
@pytest.mark.parametrize("size", [2.0 ** -115, 2.0 ** -60])
def test_attend_latent_queries_far_below_the_rotary_ones(h, size):
    """The common power that would lift such queries would lift the rotary ones out of f32's range; totals too."""
    g = gen(57)
    c = make_cache(g, 2, 300, 4)
    q_lat = (torch.randn(2, h, 512, generator=g, device=DEV) * size).to(bf)
    q_pe = (torch.randn(2, h, 64, generator=g, device=DEV) * 100).to(bf)
    end = torch.tensor([300, 140], dtype=torch.int32, device=DEV)
    idx = selection(g, [300, 140], 200, 300)
    check_attend(q_lat, q_pe, c, end, idx, None)
    lse = torch.stack([ref.attend(q_lat[b], q_pe[b], parts(c), b, ref.selected(idx[b], end[b], 300), SCALE)[2] for b in range(2)]).float()
    acc = mla.mla_accumulate_weights_fp8(q_lat, q_pe, c, end, idx, SCALE, lse, torch.zeros(2, 300, device=DEV))
    # a row's weights add up to the heads; scores are f32 sums of 576 products, each off by 2^-24 of what it has reached, exp by as much
    size = float(lse.abs().max()) + 1
    assert float((acc.sum(1) - h).abs().max()) <= h * 640 * 2.0 ** -23 * size


def test_attend_reads_only_the_selected_rows():
    g = gen(21)
    c = make_cache(g, 2, 600, 1)
    end = torch.tensor([600, 450], dtype=torch.int32, device=DEV)
    idx = selection(g, end.tolist(), 200, 600)
    q = query(g, 2, 128)
    o, lse = mla.mla_sparse_attend_fp8(*q, c, end, idx, SCALE)
    for b in range(2):
        rest = torch.ones(600, dtype=torch.bool, device=DEV)
        rest[idx[b].long()] = False
        c.kv[b, rest], c.pe[b, rest], c.scale[b, rest] = 0x7f, math.nan, math.nan
    o2, lse2 = mla.mla_sparse_attend_fp8(*q, c, end, idx, SCALE)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_attend_non_finite_query_stays_in_its_head(bad):
    g = gen(22)
    c = make_cache(g, 1, 300, 8)
    end = torch.tensor([300], dtype=torch.int32, device=DEV)
    idx = selection(g, [300], 260, 300)
    q_lat, q_pe = query(g, 1, 128)
    o, lse = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE)
    q_lat[0, 77, 5] = bad
    o2, lse2 = mla.mla_sparse_attend_fp8(q_lat, q_pe, c, end, idx, SCALE)
    hit = torch.zeros(128, dtype=torch.bool, device=DEV)
    hit[77] = True
    assert bool(torch.isnan(lse2[0, :, hit]).all()) and bool(torch.isnan(o2[0, :, hit]).all())
    # the others: the same limbs where the largest element of the head's CTA is still the same
    torch.testing.assert_close(o2[0, :, ~hit].float(), o[0, :, ~hit].float(), rtol=2.0 ** -7, atol=1e-3)
    assert bool(torch.isfinite(lse2[0, :, ~hit]).all())


def test_attend_offsets_past_32_bits():
    """A cache of 4.6 GB in one slot: its last rows lie behind byte 2^32."""
    g = gen(23)
    S, K = 9_000_000, 200
    c = mla.Fp8Cache(torch.zeros(1, S, 512, dtype=torch.uint8, device=DEV), torch.zeros(1, S, 64, dtype=bf, device=DEV),
                     torch.ones(1, S // 64 + 1, device=DEV)[:, :-(-S // 64)].contiguous(), 64)
    x, r = torch.randn(K, 512, generator=g, device=DEV).to(bf), torch.randn(K, 64, generator=g, device=DEV).to(bf)
    mla.mla_append_fp8(c, x, r, torch.tensor([0, K], dtype=torch.int32, device=DEV), torch.tensor([S - K], dtype=torch.int32, device=DEV))
    end = torch.tensor([S], dtype=torch.int32, device=DEV)
    idx = (S - 1 - torch.randperm(K, generator=g, device=DEV)).to(torch.int32)[None].contiguous()
    q = query(g, 1, 128)
    check_attend(*q, c, end, idx, None)
    _, lse = mla.mla_sparse_attend_fp8(*q, c, end, idx, SCALE)
    lse = torch.logsumexp(lse, 1).contiguous()
    acc = torch.zeros(1, S, device=DEV)
    mla.mla_accumulate_weights_fp8(*q, c, end, idx, SCALE, lse, acc)
    assert abs(float(acc.sum()) - 128) < 1e-2 and int((acc != 0).sum()) == K


def decode_inputs(g, R, h):
    qn = torch.randn(R, h, 128, generator=g, device=DEV).to(bf)
    qp = torch.randn(R, h, 64, generator=g, device=DEV).to(bf)
    w = (torch.randn(h * 256, 512, generator=g, device=DEV) * 512 ** -0.5).to(bf)
    return qn, qp, w


@pytest.mark.parametrize("R,h,K,S,block,slots", [(1, 128, 256, 1001, 1, 1), (5, 128, 333, 700, 16, 5), (90, 64, 200, 400, 1, 3),
                                                 (3, 17, 2048, 3000, 128, 3), (200, 128, 64, 300, 8, 2)])
def test_decode_matches_64_bits(R, h, K, S, block, slots):
    g = gen(R + h)
    c = make_cache(g, slots, S, block, loud=False)
    qn, qp, w = decode_inputs(g, R, h)
    end = torch.randint(0, S + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
    idx = selection(g, end.tolist(), K, S)
    slot = torch.randint(0, slots, (R,), generator=g, device=DEV, dtype=torch.int32) if slots < R else None
    lse = torch.empty(R, h, device=DEV)
    out = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE, cache_slot=slot, lse_out=lse)
    want, want_lse = ref.decode(qn, qp, parts(c), slot if slot is not None else torch.arange(R), end, idx, w, SCALE)
    assert float((out.double() - want).abs().max()) <= 1e-2 * float(want.abs().max()) + 1e-3
    some = torch.isfinite(want_lse)
    assert bool((lse[~some] == -math.inf).all()) and float((lse.double() - want_lse)[some].abs().max()) <= 1e-2


@pytest.mark.parametrize("up", [-100, -30, 0, 30, 100])
def test_decode_any_size_of_latent_query(up):
    """W_UK and the rotary queries 2^up larger, the scale 2^-up: the same attention, whatever size the latent queries have; and
    heads and 32-column chunks of very different sizes (absolute error of a score: of the largest chunk's)."""
    g = gen(91)
    R, h, K, S = 3, 70, 300, 400
    c = make_cache(g, R, S, 4, loud=False)
    qn, qp, w = decode_inputs(g, R, h)
    wk = w.view(h, 256, 512).float()
    wk[:, :128] *= torch.exp2(-torch.randint(0, 20, (h, 1, 16), generator=g, device=DEV).float()).repeat_interleave(32, 2)
    wk[3, :128] = 0
    end = torch.tensor([400, 257, 64], dtype=torch.int32, device=DEV)
    idx = selection(g, end.tolist(), K, S)
    plain = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, wk.to(bf).view(-1, 512), SCALE)
    wk[:, :128] *= 2.0 ** up
    out = mla.mla_sparse_decode_fp8(qn, (qp.float() * 2.0 ** up).to(bf), c, end, idx, wk.to(bf).view(-1, 512), SCALE * 2.0 ** -up)
    want, _ = ref.decode(qn, (qp.float() * 2.0 ** up).to(bf), parts(c), torch.arange(R), end, idx, wk.to(bf).view(-1, 512), SCALE * 2.0 ** -up)
    # 2^30 scales every factor exactly (the smallest weights are above 2^-30 2^-19 2^-5 2^-9 = 2^-63, the query's common power below
    # 2^(8 + 30 + 5)): the same steps on the same digits.  2^-100 takes weights below bf16's 2^-126, which then have fewer digits.
    assert abs(up) > 30 or torch.equal(out, plain)
    assert float((out.double() - want).abs().max()) <= 1e-2 * float(want.abs().max()) + 1e-3


@pytest.mark.parametrize("big", [2.0 ** 10, 2.0 ** 20])
def test_decode_large_factors_that_meet_no_weight(big):
    """Query columns far larger than the others whose weights are zero, in some heads, change nothing: bounds on the latent queries
    that are 2^17 and 2^27 too large."""
    g = gen(93)
    c = make_cache(g, 2, 200, 8)
    qn, qp, w = decode_inputs(g, 2, 70)
    wk = w.view(70, 256, 512).clone()
    wk[::3, 5] = 0
    quiet, loud = qn.clone(), qn.clone()
    quiet[:, ::3, 5], loud[:, ::3, 5] = 0, big
    end = torch.tensor([200, 77], dtype=torch.int32, device=DEV)
    idx = selection(g, [200, 77], 150, 200)
    a, b = (mla.mla_sparse_decode_fp8(q, qp, c, end, idx, wk.view(-1, 512), SCALE) for q in (quiet, loud))
    # fp16 below its normal numbers at worst: 2^-25 in units that put the bound, 2^7 big times the usual size, at 2^15: 2^-13 of the
    # usual size at 2^20, less than the 2^-9 that a bf16 query would be off
    torch.testing.assert_close(b.float(), a.float(), rtol=2.0 ** -6, atol=4e-3 * float(a.float().abs().max()))
    want, _ = ref.decode(loud, qp, parts(c), torch.arange(2), end, idx, wk.view(-1, 512), SCALE)
    assert float((b.double() - want).abs().max()) <= 1e-2 * float(want.abs().max()) + 1e-3


def test_decode_infinite_weights_stay_in_their_head():
    g = gen(92)
    c = make_cache(g, 2, 90, 1)
    qn, qp, w = decode_inputs(g, 2, 66)
    end = torch.tensor([90, 90], dtype=torch.int32, device=DEV)
    idx = selection(g, [90, 90], 80, 90)
    want = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE)
    bad = w.clone()
    bad.view(66, 256, 512)[65, 5, 7] = math.inf
    qn = qn.clone()
    qn[0, 2, 9] = math.nan
    out = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, bad, SCALE)
    assert bool(torch.isnan(out[:, 65]).all()) and bool(torch.isnan(out[0, 2]).all())
    out[:, 65], out[0, 2] = 0, 0
    want[:, 65], want[0, 2] = 0, 0
    torch.testing.assert_close(out.float(), want.float(), rtol=2.0 ** -6, atol=1e-3)  # without those heads, another common power


def test_decode_graph_streams_and_repeats():
    """Captured and replayed on a side stream beside an eager call of other sizes; repeats are bit-identical."""
    g = gen(31)
    c = make_cache(g, 8, 800, 16)
    qn, qp, w = decode_inputs(g, 8, 128)
    end = torch.full((8,), 800, dtype=torch.int32, device=DEV)
    idx = selection(g, end.tolist(), 600, 800)
    first = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE)
    out = torch.zeros_like(first)
    ws = torch.empty(mla.workspace_size_fp8(8, 600, 800), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE, out=out, workspace=ws)
    other = None
    for _ in range(5):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        other = mla.mla_sparse_decode_fp8(qn[:3].contiguous(), qp[:3].contiguous(), c, end[:3].contiguous(), idx[:3].contiguous(), w, SCALE)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, first)
    torch.testing.assert_close(other.float(), first[:3].float(), rtol=2.0 ** -6, atol=1e-3)  # another split of the keys


def test_steps_at_once():
    """Calls on two streams that overlap on the GPU (pairs and single CTAs, totals, appends) answer as they do alone."""
    g = gen(77)
    c = make_cache(g, 4, 500, 8)
    end = torch.tensor([500, 300, 129, 7], dtype=torch.int32, device=DEV)
    idx = selection(g, end.tolist(), 400, 500)
    args = []
    for h in (128, 40):
        q, w = torch.randn(4, h, 128, generator=g, device=DEV).to(bf), (torch.randn(h * 256, 512, generator=g, device=DEV) * 512 ** -0.5).to(bf)
        args.append((q, torch.randn(4, h, 64, generator=g, device=DEV).to(bf), w, torch.empty(4, h, device=DEV)))
    x, r = torch.randn(4, 512, generator=g, device=DEV).to(bf), torch.randn(4, 64, generator=g, device=DEV).to(bf)
    cu, at = torch.arange(5, dtype=torch.int32, device=DEV), torch.tensor([499, 300, 130, 9], dtype=torch.int32, device=DEV)

    def step(i, cache):
        q, pe, w, lse = args[i]
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = mla.mla_sparse_decode_fp8(q, pe, c, end, idx, w, SCALE, lse_out=lse, d_status=status)
        acc = torch.zeros(4, 500, device=DEV)
        mla.mla_accumulate_weights_fp8((q.float() @ torch.ones(128, 512, device=DEV) / 128).to(bf), pe, c, end, idx, SCALE, lse, acc)
        mla.mla_append_fp8(cache, x, r, cu, at)
        return out, lse.clone(), acc, cache.kv.clone(), cache.scale.clone(), status

    def copy():
        return mla.Fp8Cache(c.kv.clone(), c.pe.clone(), c.scale.clone(), c.block)

    alone = [step(i, copy()) for i in range(2)]
    sides, copies = [torch.cuda.Stream(), torch.cuda.Stream()], [[copy() for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(6):
        for i in range(2):
            with torch.cuda.stream(sides[i]):
                got[i].append(step(i, copies[i][k]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert int(one[-1]) == 0
            for a, b in zip(one, alone[i]):
                assert torch.equal(a, b)


def test_decode_index_checks():
    g = gen(32)
    c = make_cache(g, 1, 100, 1)
    qn, qp, w = decode_inputs(g, 1, 128)
    idx = torch.tensor([[5, 6, 5, -1]], dtype=torch.int32, device=DEV)
    end = torch.tensor([100], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    was = mla.set_index_checks(True)
    try:
        mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, SCALE, d_status=status)
    finally:
        mla.set_index_checks(was)
    assert int(status) == 5


# ------------------------------------------------------------------- totals
@pytest.mark.parametrize("R,h,K,S,block", [(1, 128, 1, 1, 1), (2, 1, 40, 64, 0), (3, 127, 129, 300, 0), (3, 64, 300, 301, 8),
                                           (4, 128, 1000, 2000, 128), (160, 128, 300, 400, 0), (160, 33, 700, 800, 1)])
def test_totals_match_64_bits(R, h, K, S, block):
    g = gen(40 + K)
    if block:
        c = make_cache(g, R, S, block)
        cache = parts(c)
    else:
        cache = (torch.randn(R, S, 512, generator=g, device=DEV).to(bf), torch.randn(R, S, 64, generator=g, device=DEV).to(bf), None, 1)
    end = torch.randint(0, S + 1, (R,), generator=g, device=DEV, dtype=torch.int32)
    idx = selection(g, end.tolist(), K, S, holes=True)
    q_lat, q_pe = query(g, R, h)
    acc = torch.rand(R, S, generator=g, device=DEV)
    lse = torch.empty(R, h, device=DEV)
    want, bound = acc.double(), torch.zeros(R, S, dtype=torch.float64, device=DEV)
    for b in range(R):
        t = ref.selected(idx[b], end[b], S)
        x, _, l64 = ref.attend(q_lat[b], q_pe[b], cache, b, t, SCALE)
        lse[b] = l64.float()
        p = torch.exp(x - lse[b].double()[:, None])
        sb = score_bound(q_lat[b], q_pe[b], cache, b, t, 2.0 ** -19 if block else 0.0) if len(t) else x
        # the exponent's own rounding: x and lse in log2 units, to 24 bits
        rel = sb + 2.0 ** -22 * (x.abs() + l64.abs()[:, None] + 1) if len(t) else x
        want[b, t] += p.sum(0)
        bound[b, t] = (p * rel).sum(0) + 2.0 ** -22 * want[b, t]
    was = acc.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if block:
        got = mla.mla_accumulate_weights_fp8(q_lat, q_pe, c, end, idx, SCALE, lse, acc, d_status=status)
    else:
        got = mla.mla_accumulate_weights(q_lat, q_pe, cache[0], cache[1], end, idx, SCALE, lse, acc, d_status=status)
    assert got is acc and int(status) == 0
    assert bool(((acc.double() - want).abs() <= bound).all())
    assert torch.equal(acc[bound == 0], was[bound == 0])  # nothing but the selected positions


def test_totals_repeat_and_run_in_a_graph():
    g = gen(50)
    c = make_cache(g, 6, 500, 4)
    end = torch.full((6,), 500, dtype=torch.int32, device=DEV)
    idx = selection(g, end.tolist(), 400, 500)
    q = query(g, 6, 128)
    lse = torch.full((6, 128), 7.0, device=DEV)
    one = mla.mla_accumulate_weights_fp8(*q, c, end, idx, SCALE, lse, torch.zeros(6, 500, device=DEV))
    acc = torch.zeros(6, 500, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_accumulate_weights_fp8(*q, c, end, idx, SCALE, lse, acc)
    graph.replay()
    assert torch.equal(acc, one)
    graph.replay()
    assert torch.equal(acc, one + one)
    # a head's lse of -inf leaves its weights infinite, NaN makes them NaN: no other row is touched
    lse[2, 3] = math.nan
    two = mla.mla_accumulate_weights_fp8(*q, c, end, idx, SCALE, lse, torch.zeros(6, 500, device=DEV))
    rows = torch.arange(6, device=DEV) != 2
    assert torch.equal(two[rows], one[rows]) and bool(torch.isnan(two[2][idx[2].long()]).all())
