"""What the 8-bit cache's entry points, the totals and the eviction refuse, on
the host: bad arguments are answered before anything is launched, so no GPU is
needed."""
import ctypes

import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from sparse_latent_attention_absorb_b200 import binding, build

INVALID_ARG, WORKSPACE = 1, 2
A = 0x10000  # aligned, never dereferenced


def P(addr=A):
    return ctypes.c_void_p(addr)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def each_bad(args, pointers):
    """The argument lists with one pointer missing or misaligned."""
    for i in pointers:
        for bad in (None, P(A + 8)):
            a = list(args)
            a[i] = bad
            yield i, a


def with_(args, **at):
    a = list(args)
    for i, v in at.items():
        a[int(i[1:])] = v
    return a


def refused(fn, lists):
    for a in lists:
        assert fn(*a) == INVALID_ARG, a


def test_attend_and_decode(lib):
    f = ctypes.c_float(0.07)
    #            0    1    2    3    4   5   6    7    8   9  10   11  12  13  14  15   16
    dec = [P(), P(), P(), P(), P(), 16, P(), P(), P(), P(), f, P(), 4, 16, 64, 4, 128, P(), 1 << 30, None, None, None]
    refused(lib.mla_sparse_decode_fp8, [a for _, a in each_bad(dec, (0, 1, 2, 3, 4, 7, 8, 9, 11))])
    bad = [with_(dec, _5=b) for b in (0, -1, 3, 256, 48)] + [with_(dec, _6=P(A + 4)), with_(dec, _6=None, _15=3)]
    bad += [with_(dec, _12=0), with_(dec, _13=0), with_(dec, _14=0), with_(dec, _15=0), with_(dec, _16=0), with_(dec, _16=129)]
    bad += [with_(dec, _10=ctypes.c_float(v)) for v in (float("nan"), float("inf"))]
    bad += [with_(dec, _19=P(A + 2)), with_(dec, _20=P(A + 1))]
    refused(lib.mla_sparse_decode_fp8, bad)
    att = [P(), P(), P(), P(), P(), 1, None, P(), P(), f, P(), P(), 4, 16, 64, 4, 128, 1, None, None]
    refused(lib.mla_sparse_attend_fp8, [a for _, a in each_bad(att, (0, 1, 2, 3, 4, 7, 8, 10, 11))])
    refused(lib.mla_sparse_attend_fp8, [with_(att, _5=5), with_(att, _15=3), with_(att, _16=200)])


def test_sizes(lib):
    assert lib.mla_num_splits_fp8(0, 1, 1) == 0 and lib.mla_num_splits_fp8(1, 0, 1) == 0
    assert lib.mla_num_splits_fp8(1, 1, 0) == 0 and lib.mla_num_splits_fp8(1, 1, 129) == 0
    assert lib.mla_sparse_decode_fp8_workspace_size(1, 1, 0, 128) == 0
    for R in (1, 3, 64, 500):
        for K in (1, 128, 129, 2048, 8192):
            for h in (1, 64, 65, 128):
                n = lib.mla_num_splits_fp8(R, K, h)
                assert 1 <= n <= min(128, -(-K // 128))
                need = R * h * (512 * 2 + 4) + R * n * h * 512 * 2 + R * n * h * 4
                assert need <= lib.mla_sparse_decode_fp8_workspace_size(R, K, 9000, h) <= need + 4 * 256


def test_append(lib):
    app = [P(), P(), P(), P(), None, P(), P(), P(), 16, 100, 4, 64, 4, None]
    refused(lib.mla_append_fp8, [a for _, a in each_bad(app, (0, 1, 2, 3, 5, 6, 7))])
    refused(lib.mla_append_fp8, [with_(app, _8=24), with_(app, _9=0), with_(app, _10=0), with_(app, _11=0), with_(app, _12=0),
                                 with_(app, _12=3), with_(app, _4=P(A + 4))])


def test_totals(lib):
    f = ctypes.c_float(0.07)
    acc = [P(), P(), P(), P(), P(), P(), f, P(), P(), 4, 16, 64, 128, None, None]
    refused(lib.mla_accumulate_weights, [a for _, a in each_bad(acc, (0, 1, 2, 3, 4, 5, 7, 8))])
    refused(lib.mla_accumulate_weights, [with_(acc, _9=0), with_(acc, _10=0), with_(acc, _11=0), with_(acc, _12=0), with_(acc, _12=129),
                                         with_(acc, _13=P(A + 2)), with_(acc, _6=ctypes.c_float(float("nan")))])
    acc8 = [P(), P(), P(), P(), P(), 8, P(), P(), f, P(), P(), 4, 16, 64, 128, None, None]
    refused(lib.mla_accumulate_weights_fp8, [a for _, a in each_bad(acc8, (0, 1, 2, 3, 4, 6, 7, 9, 10))])
    refused(lib.mla_accumulate_weights_fp8, [with_(acc8, _5=7), with_(acc8, _13=0)])


def test_eviction(lib):
    big = 1 << 32
    ev = [P(), P(A + big), P(A + 2 * big), P(), P(A + 3 * big), P(A + 4 * big), P(A + 5 * big), P(), P(), 2, 64, 32, 8, None]
    refused(lib.mla_evict, [a for _, a in each_bad(ev, range(9))])
    refused(lib.mla_evict, [with_(ev, _9=0), with_(ev, _9=65536), with_(ev, _10=0), with_(ev, _11=0), with_(ev, _11=65),
                            with_(ev, _12=-1), with_(ev, _12=33)])
    refused(lib.mla_evict, [with_(ev, _6=ev[2]), with_(ev, _4=ev[0]), with_(ev, _4=P(A + 1024))])  # half in place, overlapping
    ev8 = [P(), P(A + big), P(A + 2 * big), 16, P(A + 3 * big), P(), P(A + 4 * big), P(A + 5 * big), P(A + 6 * big), P(A + 7 * big),
           P(), P(), 2, 64, 32, 8, None]
    refused(lib.mla_evict_fp8, [a for _, a in each_bad(ev8, (0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11))])
    refused(lib.mla_evict_fp8, [with_(ev8, _3=0), with_(ev8, _8=ev8[2]), with_(ev8, _6=P(A + 16))])


def test_binding_refuses_cpu_tensors_and_bad_blocks():
    kv, pe, sc = torch.zeros(1, 8, 512, dtype=torch.uint8), torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.ones(1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        mla.Fp8Cache(kv, pe, sc)
    for block in (0, 3, 256, True, 2.0):
        with pytest.raises(ValueError, match="block"):
            mla.Fp8Cache(kv, pe, sc, block)
    with pytest.raises(ValueError, match="kv"):
        mla.Fp8Cache(kv[0], pe, sc)
    with pytest.raises(ValueError):
        mla.mla_evict(kv, pe, torch.zeros(8), torch.zeros(1, dtype=torch.int32), 4, 1)


def test_binding_eviction_takes_all_outputs_or_none():
    """Out of place the totals move too: leaving their buffer out would drop them."""
    kv, pe, acc = torch.zeros(1, 8, 512), torch.zeros(1, 8, 64), torch.zeros(1, 8)
    end = torch.zeros(1, dtype=torch.int32)
    for outs in (dict(kv_out=kv, pe_out=pe), dict(acc_out=acc), dict(kv_out=kv, acc_out=acc), dict(pe_out=pe)):
        with pytest.raises(ValueError, match="all of them, or none"):
            mla.mla_evict(kv, pe, acc, end, 4, 1, **outs)
    cache = object.__new__(mla.Fp8Cache)
    for outs in (dict(cache_out=cache), dict(acc_out=acc)):
        with pytest.raises(ValueError, match="both, or neither"):
            mla.mla_evict_fp8(cache, acc, end, 4, 1, **outs)


def test_reference_rounding_is_torchs():
    """The tests' own E4M3 decoding and rounding against torch's cast: every code, its neighbours' midpoints, random numbers."""
    from tests import cache8_refs as ref
    codes = torch.arange(256, dtype=torch.uint8)
    v = ref.e4m3_values(codes)
    want = codes.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(v), torch.isnan(want)) and torch.equal(v.nan_to_num(), want.nan_to_num())
    fin = v[torch.isfinite(v)].sort().values
    x = torch.cat([fin, (fin[1:] + fin[:-1]) / 2, torch.randn(20000, generator=torch.Generator().manual_seed(1)).double() * 100])
    x = x[x.abs() <= 448].float().double()
    assert torch.equal(ref.e4m3_codes(x), x.float().to(torch.float8_e4m3fn).view(torch.uint8))
