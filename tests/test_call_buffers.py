"""Buffers that a call makes itself (outputs, workspaces) belong to the stream it
runs on: memory of another stream's pool may be handed to work of that stream
while the call's kernels still use it, or still be read by work queued there."""
import contextlib
import types

import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from sparse_latent_attention_absorb_b200 import binding

bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def cache8():
    c = object.__new__(mla.Fp8Cache)
    c.kv, c.pe, c.scale = z(2, 8, 512, dtype=torch.uint8), z(2, 8, 64), z(2, 8, dtype=f32)
    c.block, c.n_slots, c.S_max = 1, 2, 8
    return c


def calls():
    """Every wrapper that allocates, with the fewest arguments, and the number of buffers it makes."""
    q, qp, kv, pe = z(2, 128, 128), z(2, 128, 64), z(2, 8, 512), z(2, 8, 64)
    end, idx, w, ql = z(2, dtype=i32), z(2, 4, dtype=i32), z(128 * 256, 512), z(2, 128, 512)
    acc, wo, x = z(2, 8, dtype=f32), z(256, 128 * 128), z(2, 128 * 128)
    c = cache8()
    weight = types.SimpleNamespace(is_cuda=True, dtype=bf, dim=lambda: 2, stride=lambda i: 256 - 255 * i, shape=(256, 256), device="cpu",
                                   data_ptr=lambda: 16)
    return {
        "mla_prepare_wo": (1, lambda **k: mla.mla_prepare_wo(weight, **k)),
        "mla_sparse_decode": (2, lambda **k: mla.mla_sparse_decode(q, qp, kv, pe, end, idx, w, 0.1, **k)),
        "mla_absorb_q": (1, lambda **k: mla.mla_absorb_q(q, w, **k)),
        "mla_sparse_attend": (2, lambda **k: mla.mla_sparse_attend(ql, qp, kv, pe, end, idx, 0.1, **k)),
        "mla_combine_value_up": (1, lambda **k: mla.mla_combine_value_up(ql, z(2, 1, 128, dtype=f32), w, **k)),
        "mla_output_projection": (2, lambda **k: mla.mla_output_projection(x, wo, **k)),
        "mla_sparse_decode_project": (2, lambda **k: mla.mla_sparse_decode_project(q, qp, kv, pe, end, idx, w, 0.1, wo, **k)),
        "mla_sparse_prefill": (2, lambda **k: mla.mla_sparse_prefill(q, qp, kv, pe, end, end, idx, w, 0.1, **k)),
        "mla_check_topk_indices": (1, lambda **k: mla.mla_check_topk_indices(end, idx, 8, **k)),
        "mla_sparse_decode_heads": (2, lambda **k: mla.mla_sparse_decode_heads(q, qp, kv, pe, end, idx, w, 0.1, **k)),
        "mla_output_projection_shard": (2, lambda **k: mla.mla_output_projection_shard(z(2, 256), weight, **k)),
        "mla_output_projection_prepared": (
            2, lambda **k: mla.mla_output_projection_prepared(x, mla.PreparedWo(z(256 * 128 * 128), 256, 128 * 128), **k)),
        "mla_dequant_fp8_blocks": (1, lambda **k: mla.mla_dequant_fp8_blocks(z(128, 128, dtype=torch.uint8), z(1, 1, dtype=f32), **k)),
        "mla_sparse_decode_fp8": (2, lambda **k: mla.mla_sparse_decode_fp8(q, qp, c, end, idx, w, 0.1, **k)),
        "mla_sparse_attend_fp8": (2, lambda **k: mla.mla_sparse_attend_fp8(ql, qp, c, end, idx, 0.1, **k)),
        "mla_evict": (2, lambda **k: mla.mla_evict(kv, pe, acc, end, 4, 1, **k)),
        "mla_evict_fp8": (2, lambda **k: mla.mla_evict_fp8(c, acc, end, 4, 1, **k)),
    }


class Lib:
    """Every status is 0, every size 1024, and the stream handle of the last call is kept."""

    def __getattr__(self, name):
        def call(*args):
            self.stream = args[-1] if args else None
            return 1024 if "workspace_size" in name else (1 if "num_splits" in name else 0)
        return call


@pytest.fixture
def host(monkeypatch):
    """The wrappers without a GPU: returns the list of streams that buffers were made under, and the library."""
    lib, made, now = Lib(), [], [None]
    monkeypatch.setattr(binding, "load_library", lambda: lib)
    monkeypatch.setattr(binding, "_check", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_check_same_device", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_sizing_cache", {})
    monkeypatch.setattr(binding, "num_splits", lambda *a: 1)
    monkeypatch.setattr(binding, "num_splits_fp8", lambda *a: 1)
    monkeypatch.setattr(binding, "workspace_size_fp8", lambda *a: 1024)

    @contextlib.contextmanager
    def under(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    empty = torch.empty

    def recorded(*a, **k):
        made.append(now[-1])
        return empty(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: types.SimpleNamespace(cuda_stream=handle))
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return made, lib


@pytest.mark.parametrize("name", sorted(calls()))
def test_buffers_are_made_under_the_calls_stream(host, name):
    made, lib = host
    n, call = calls()[name]
    call(stream=types.SimpleNamespace(cuda_stream=7))
    assert made == [7] * n and lib.stream == 7
    made.clear()
    call()
    assert made == [None] * n and lib.stream == 1


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [128, 16])
def test_a_steps_buffers_are_not_handed_out_while_it_runs(heads):
    """A step on a side stream that starts late, while the current stream fills all the memory it can get again."""
    from sparse_latent_attention_absorb_b200 import build
    build.build()
    from tests import test_cache8 as t8
    g = t8.gen(3)
    c = t8.make_cache(g, 4, 400, 8)
    qn, qp, w = t8.decode_inputs(g, 4, heads)
    end = torch.full((4,), 400, dtype=i32, device=t8.DEV)
    idx = t8.selection(g, end.tolist(), 300, 400)
    want = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, t8.SCALE)
    size = mla.workspace_size_fp8(4, 300, 400, heads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        out = mla.mla_sparse_decode_fp8(qn, qp, c, end, idx, w, t8.SCALE, stream=side)
        for n in (size, size, out.numel() * 2):
            torch.empty(n, dtype=torch.uint8, device=t8.DEV).fill_(0x7f)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
        torch.cuda.synchronize()
