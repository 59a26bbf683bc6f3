"""The Python calls of the paged cache path take tensors of the cache's device alone, with that device current (tensors
that only have shapes, and a library that only counts: no GPU needed)."""
import types

import pytest
import torch

from dflash_draft_selection_gb300 import binding

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Shape:
    """What the calls ask of a tensor."""

    def __init__(self, dt, *shape, dev=0):
        self.dtype, self.shape, self.dev = dt, torch.Size(shape), dev
        self.device, self.is_cuda = torch.device("cuda", dev), True

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()


def arguments():
    B, T, Hq, Hkv, d = 2, 3, 4, 2, 64
    lens = lambda: Shape(I32, B)  # noqa: E731
    cache = types.SimpleNamespace(dtype=BF, Hkv=Hkv, d=d, page_size=16, _dev=0, _ref=None)
    ws = lambda: types.SimpleNamespace(buf=Shape(U8, 1 << 20))  # noqa: E731
    table = lambda: Shape(I32, B, 4)  # noqa: E731
    return {
        "rope_append": dict(q=Shape(BF, B, T, Hq, d), k=Shape(BF, B, T, Hkv, d), v=Shape(BF, B, T, Hkv, d),
                            cos_sin=Shape(F32, 10, d), pos_ids=Shape(I32, 1, B, T), cache=cache, page_table=table(),
                            kv_len=lens(), pair_axis=Shape(U8, d // 2), q_norm=Shape(BF, d), k_norm=Shape(BF, d),
                            q_len=lens(), seq_pos=lens(), out=(Shape(BF, B, T, Hq, d), lens())),
        "paged_attn": dict(q=Shape(BF, B, T, Hq, d), cache=cache, page_table=table(), kv_len=lens(), q_len=lens(),
                           seq_pos=lens(), ws=ws(), out=(Shape(BF, B, T, Hq, d), Shape(F32, B, T, Hq))),
        "kv_evict": dict(cache=cache, page_table=table(), kv_len=lens(), budget=8, seq_len=lens(), ws=ws(), out=lens()),
    }


def tensors(a):
    for v in a.values():
        for t in v if isinstance(v, tuple) else (v,):
            t = getattr(t, "buf", t)
            if isinstance(t, Shape):
                yield t


@pytest.mark.parametrize("name", ["rope_append", "paged_attn", "kv_evict"])
def test_tensors_of_another_device_are_refused(monkeypatch, name):
    calls = []
    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(**{"dflash2_" + name: lambda *a: calls.append(a) or 0}))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 7 + dev, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call = getattr(binding, name)
    call(**arguments()[name])
    assert len(calls) == 1 and calls[0][-1] == 7            # the stream of the cache's device
    n = len(list(tensors(arguments()[name])))
    assert n >= 5
    for i in range(n):
        a = arguments()[name]
        list(tensors(a))[i].dev = 1
        with pytest.raises(ValueError):
            call(**a)
    a = arguments()[name]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError):                          # the cache's device is not the current one
        call(**a)
    assert len(calls) == 1


@pytest.mark.parametrize("name,number", [("paged_attn", "window"), ("kv_evict", "budget"), ("kv_evict", "recent"),
                                         ("kv_evict", "sink")])
def test_numbers_that_do_not_fit_are_refused(monkeypatch, name, number):
    """2^32 + 5 is not 5."""
    calls = []
    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(**{"dflash2_" + name: lambda *a: calls.append(a) or 0}))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call = getattr(binding, name)
    for n in (2 ** 31 - 1, 5):
        call(**{**arguments()[name], number: n})
        assert n in calls[-1]
    for n in (2 ** 32 + 5, 2 ** 32, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            call(**{**arguments()[name], number: n})
    assert len(calls) == 2
