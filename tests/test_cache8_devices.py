"""Tensors of one call lie on one GPU, the current one: each of them is refused
elsewhere, on the host, before a kernel gets its address.  The GPUs here are
faked."""
import pytest
import torch

import sparse_latent_attention_absorb_b200 as mla
from sparse_latent_attention_absorb_b200 import binding

bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


class Fake(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    gpu = 0

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.gpu))

    def get_device(self):
        return self.gpu

    @property
    def shape(self):
        return torch.Tensor.size(self)


def t(*shape, dtype=bf, gpu=0):
    f = torch.zeros(shape, dtype=dtype).as_subclass(Fake)
    f.gpu = gpu
    return f


@pytest.fixture(autouse=True)
def one_gpu(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0
    monkeypatch.setattr(binding, "load_library", lambda: Lib())
    monkeypatch.setattr(binding, "num_splits_fp8", lambda *a: 1)
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def cache(**gpu):
    return mla.Fp8Cache(t(2, 8, 512, dtype=u8, gpu=gpu.get("kv", 0)), t(2, 8, 64, gpu=gpu.get("pe", 0)),
                        t(2, 8, dtype=f32, gpu=gpu.get("scale", 0)))


def test_a_cache_lies_on_one_gpu():
    cache()
    assert cache(kv=1, pe=1, scale=1).kv.get_device() == 1
    for part in ("pe", "scale"):
        with pytest.raises(ValueError, match=f"{part}: on cuda:1, expected cuda:0"):
            cache(**{part: 1})
    with pytest.raises(ValueError, match="expected cuda:1"):
        cache(kv=1)


def ev():
    return dict(acc=t(2, 8, dtype=f32), end_pos=t(2, dtype=i32), kept=t(2, 4, dtype=i32), new_end=t(2, dtype=i32))


def att():
    return dict(q_pe=t(2, 128, 64), end_pos=t(2, dtype=i32), topk_idx=t(2, 4, dtype=i32), d_status=t(1, dtype=i32))


CALLS = {
    "decode": lambda: (mla.mla_sparse_decode_fp8, dict(
        q_nope=t(2, 128, 128), cache=cache(), wkv_b=t(128 * 256, 512), scale=0.1, cache_slot=t(2, dtype=i32), out=t(2, 128, 128),
        workspace=t(1 << 10, dtype=u8), lse_out=t(2, 128, dtype=f32), **att())),
    "attend": lambda: (mla.mla_sparse_attend_fp8, dict(
        q_lat=t(2, 128, 512), cache=cache(), scale=0.1, cache_slot=t(2, dtype=i32), o_part=t(2, 1, 128, 512),
        lse_part=t(2, 1, 128, dtype=f32), **att())),
    "append": lambda: (mla.mla_append_fp8, dict(
        cache=cache(), kv_new=t(2, 512), pe_new=t(2, 64), cu_rows=t(3, dtype=i32), start_pos=t(2, dtype=i32), cache_slot=t(2, dtype=i32))),
    "totals": lambda: (mla.mla_accumulate_weights, dict(
        q_lat=t(2, 128, 512), kv_cache=t(2, 8, 512), pe_cache=t(2, 8, 64), scale=0.1, lse=t(2, 128, dtype=f32), acc=t(2, 8, dtype=f32), **att())),
    "totals8": lambda: (mla.mla_accumulate_weights_fp8, dict(
        q_lat=t(2, 128, 512), cache=cache(), scale=0.1, lse=t(2, 128, dtype=f32), acc=t(2, 8, dtype=f32), **att())),
    "evict": lambda: (mla.mla_evict, dict(
        kv_cache=t(2, 8, 512), pe_cache=t(2, 8, 64), keep=4, recent=1, kv_out=t(2, 8, 512), pe_out=t(2, 8, 64), acc_out=t(2, 8, dtype=f32),
        **ev())),
    "evict8": lambda: (mla.mla_evict_fp8, dict(cache=cache(), keep=4, recent=1, cache_out=cache(), acc_out=t(2, 8, dtype=f32), **ev())),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_every_tensor_of_a_call_is_looked_at(name):
    fn, args = CALLS[name]()
    fn(**args)
    for key in args:
        fn, args = CALLS[name]()
        if isinstance(args[key], mla.Fp8Cache):
            args[key] = cache(kv=1, pe=1, scale=1)
        elif isinstance(args[key], torch.Tensor):
            args[key].gpu = 1
        else:
            continue
        with pytest.raises(ValueError, match="cuda:1"):
            fn(**args)
