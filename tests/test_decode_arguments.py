"""Arguments of the 4-bit and sampling calls that are taken or refused on the host (no GPU needed: the pointers are never
dereferenced)."""
import ctypes
import types

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from dflash_draft_selection_gb300 import binding

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
RECORD = dict(codes=4096, scale=8192, zero=None, N=40, K=200, code_stride=112, side_stride=2, group=128, side_dt=1)


def library():
    from dflash_draft_selection_gb300 import build
    build.build()
    return d2.load_library()


def record(**kw):
    return ctypes.byref(binding._Weight4Record(**{**RECORD, **kw}))


def quant(w=None, **kw):
    a = dict(W=4096, dt=1, ld=200, w=record(**(w or {})), stream=None)
    return library().dflash2_quant4(*{**a, **kw}.values())


def dequant(w=None, **kw):
    a = dict(w=record(**(w or {})), out=4096, dt=1, ld=200, stream=None)
    return library().dflash2_dequant4(*{**a, **kw}.values())


def linear(w=None, **kw):
    a = dict(x=4096, dt=1, rows=3, x_stride=200, w=record(**(w or {})), y=4096, y_dt=1, y_stride=40, ws=None, ws_bytes=0,
             stream=None)
    return library().dflash2_linear4(*{**a, **kw}.values())


def sample(**kw):
    a = dict(logits=4096, dt=1, rows=3, V=100, ld=104, params=None, min_p=None, rows_per_param=1, u=4, token=8, prob=12,
             stream=None)
    return library().dflash2_sample(*{**a, **kw}.values())


BAD_RECORDS = [dict(codes=None), dict(codes=4104), dict(scale=None), dict(scale=8193), dict(zero=8193),
               dict(scale=8194, side_dt=0), dict(zero=8194, side_dt=0), dict(N=-1), dict(N=1 << 31), dict(K=0),
               dict(K=-5), dict(K=(1 << 31) - 1), dict(code_stride=96), dict(code_stride=120), dict(side_stride=1),
               dict(group=0), dict(group=16), dict(group=96), dict(group=256), dict(group=32), dict(side_dt=2),
               dict(side_dt=-1)]


@pytest.mark.parametrize("bad", BAD_RECORDS, ids=str)
def test_records(bad):
    assert quant(bad) == dequant(bad) == linear(bad) == INVALID


def test_calls_on_records():
    for call in (quant, dequant, linear):
        assert call(w=None, dt=2) == INVALID
    for call in (quant, dequant):
        assert call(ld=199) == INVALID
        assert call(dict(N=0, codes=None, scale=None)) == OK
        assert call(dict(N=(1 << 31) - 1, K=1 << 20, code_stride=1 << 20, side_stride=1 << 20), ld=1 << 20) == UNSUPPORTED
    assert quant(W=None) == quant(W=4097) == dequant(out=None) == dequant(out=4097) == INVALID
    assert quant(W=4098, dt=0) == dequant(out=4098, dt=0) == INVALID
    for kw in (dict(x=None), dict(y=None), dict(x=4097), dict(y=4097), dict(rows=-1), dict(x_stride=199),
               dict(y_stride=39), dict(dt=0, y_dt=1), dict(y_dt=5), dict(x=4098, dt=0, y_dt=0), dict(y=4098, y_dt=0)):
        assert linear(**kw) == INVALID, kw
    assert linear(rows=0, x=None, y=None) == linear(dict(N=0, codes=None, scale=None)) == OK
    assert linear(dict(K=(1 << 17) + 1, code_stride=1 << 17, side_stride=1 << 17), x_stride=1 << 18) == UNSUPPORTED
    assert linear(rows=(1 << 19) + 1) == UNSUPPORTED
    long = dict(K=(1 << 13) + 1, code_stride=1 << 13, side_stride=65)
    assert linear({**long, "N": 2}, rows=(1 << 15) + 1, x_stride=1 << 14, dt=0, y_dt=0) == UNSUPPORTED
    assert linear({**long, "N": 3}, rows=(1 << 15) + 1, x_stride=1 << 14) == UNSUPPORTED
    assert linear(long, rows=(1 << 15) + 1, x_stride=1 << 14) == INVALID     # these take a workspace
    L = library()
    need = L.dflash2_linear4_workspace_bytes
    assert need(1, 1, 40, 200) == need(0, 8, 151936, 200) == need(1, 0, 40, 200) == need(1, 1 << 20, 1 << 20, 1) == 0
    assert need(0, 512, 151936, 200) >= 512 * 256 * 6
    big = dict(N=151936)
    assert need(1, 512, 151936, 200) >= 512 * 256 * 2
    assert linear(big, rows=512, y_stride=151936) == linear(big, rows=512, y_stride=151936, ws=4104, ws_bytes=1 << 40) == INVALID
    assert linear(big, rows=512, y_stride=151936, ws=4096, ws_bytes=need(1, 512, 151936, 200) - 1) == WORKSPACE
    assert L.dflash2_quant4(4096, 1, 200, None, None) == L.dflash2_dequant4(None, 4096, 1, 200, None) == INVALID
    assert L.dflash2_linear4(4096, 1, 3, 200, None, 4096, 1, 40, None, 0, None) == INVALID


def test_sample():
    for kw in (dict(logits=None), dict(logits=4104), dict(u=None), dict(token=None), dict(prob=None), dict(u=6),
               dict(token=2), dict(prob=1), dict(params=5), dict(min_p=7), dict(rows=-1), dict(V=0), dict(V=1 << 31),
               dict(V=105), dict(ld=101), dict(ld=100, dt=1), dict(rows_per_param=0), dict(dt=3)):
        assert sample(**kw) == INVALID, kw
    assert sample(rows=0, logits=None, u=None, token=None, prob=None) == OK
    assert sample(rows=0, V=0) == INVALID
    assert sample(rows=1 << 28) == UNSUPPORTED


class Shape:
    """What the Python calls ask of a tensor."""

    def __init__(self, dt, *shape, dev=0, stride=None):
        self.dtype, self.shape, self.dev = dt, torch.Size(shape), dev
        self.device, self.is_cuda = torch.device("cuda", dev), True
        self._stride = stride or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return self._stride == torch.empty(self.shape, device="meta").stride()

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


U8, BF, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def calls(monkeypatch):
    """Calls that reached the library, with the first GPU current."""
    made = []

    class Library:
        def __getattr__(self, name):
            return (lambda *a: 0) if name.endswith("_bytes") else lambda *a: made.append(name) or 0

    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "load_library", lambda: binding._lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return made


def w4(dev=0, **kw):
    a = dict(codes=Shape(U8, 40, 112, dev=dev), scale=Shape(BF, 40, 2, dev=dev), zero=Shape(BF, 40, 2, dev=dev), K=200,
             group=128)
    return d2.Weight4(**{**a, **kw})


def test_weights_are_checked_when_they_are_made():
    w4()
    w4(zero=None)
    w4(scale=Shape(F32, 40, 2), zero=Shape(F32, 40, 2))
    assert w4(codes=Shape(U8, 40, 112, stride=(4096, 1)))._rec.code_stride == 4096
    one = d2.Weight4(Shape(U8, 1, 112, stride=(1, 1)), Shape(BF, 1, 2, stride=(1, 1)), None, K=200)
    assert (one._rec.code_stride, one._rec.side_stride) == (112, 2)
    for kw in (dict(codes=Shape(I32, 40, 112)), dict(codes=Shape(U8, 40, 96)), dict(codes=Shape(U8, 4480)),
               dict(codes=Shape(U8, 40, 112, stride=(1, 40))), dict(scale=Shape(BF, 40, 3)), dict(scale=Shape(BF, 39, 2)),
               dict(zero=Shape(F32, 40, 2)), dict(zero=Shape(BF, 40, 1)), dict(scale=Shape(BF, 40, 2, dev=1)),
               dict(zero=Shape(BF, 40, 2, dev=1)), dict(zero=Shape(BF, 40, 2, stride=(4, 1))), dict(K=0), dict(K=300),
               dict(group=100), dict(scale=Shape(BF, 40, 2, stride=(1, 40)))):
        with pytest.raises(ValueError):
            w4(**kw)
    with pytest.raises(TypeError):
        w4(scale=Shape(torch.float16, 40, 2), zero=None)


def test_calls_take_the_weights_device_and_shapes(calls):
    w, far = w4(), w4(dev=1)
    d2.linear4(Shape(BF, 3, 200), w, out=Shape(BF, 3, 40))
    d2.quant4(Shape(F32, 40, 200, stride=(256, 1)), out=w)
    d2.dequant4(w, out=Shape(F32, 40, 200))
    assert calls == ["dflash2_linear4", "dflash2_quant4", "dflash2_dequant4"]
    bad = [lambda: d2.linear4(Shape(BF, 3, 199), w, out=Shape(BF, 3, 40)),
           lambda: d2.linear4(Shape(BF, 3, 200), w, out=Shape(BF, 3, 41)),
           lambda: d2.linear4(Shape(BF, 3, 200), w, out=Shape(BF, 2, 40)),
           lambda: d2.linear4(Shape(BF, 3, 200, stride=(1, 3)), w, out=Shape(BF, 3, 40)),
           lambda: d2.linear4(Shape(BF, 1, 3, 200), w, out=Shape(BF, 3, 40)),
           lambda: d2.linear4(Shape(BF, 3, 200, dev=1), w, out=Shape(BF, 3, 40)),
           lambda: d2.linear4(Shape(BF, 3, 200), w, out=Shape(BF, 3, 40, dev=1)),
           lambda: d2.linear4(Shape(BF, 3, 200, dev=1), far, out=Shape(BF, 3, 40, dev=1)),
           lambda: d2.quant4(Shape(F32, 40, 201), out=w), lambda: d2.quant4(Shape(F32, 40, 200, dev=1), out=w),
           lambda: d2.quant4(Shape(F32, 40, 200, dev=1), out=far), lambda: d2.quant4(Shape(F32, 8000), out=w),
           lambda: d2.dequant4(w, out=Shape(BF, 40, 200, stride=(1, 40))), lambda: d2.dequant4(far, out=Shape(BF, 40, 200))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        d2.linear4(Shape(torch.float16, 3, 200), w, out=Shape(BF, 3, 40))
    assert len(calls) == 3


def test_sample_takes_the_logits_device_and_shapes(calls, monkeypatch):
    monkeypatch.setattr(binding, "_params_from", lambda p, dev: p)
    ok = dict(logits=Shape(BF, 4, 104), u=Shape(F32, 4), params=Shape(U8, 48), min_p=Shape(F32, 4),
              out=(Shape(I32, 4), Shape(F32, 4)))
    d2.sample(**ok)
    d2.sample(**{**ok, "V": 100})
    d2.sample(**{**ok, "params": Shape(U8, 24), "min_p": Shape(F32, 2), "rows_per_param": 2})
    d2.sample(**{**ok, "params": None, "min_p": None})
    assert len(calls) == 4
    for kw in (dict(u=Shape(F32, 3)), dict(u=Shape(F32, 4, dev=1)), dict(u=Shape(BF, 4)), dict(params=Shape(U8, 47)),
               dict(params=Shape(U8, 48, dev=1)), dict(min_p=Shape(F32, 3)), dict(min_p=Shape(F32, 4, dev=1)),
               dict(logits=Shape(BF, 4, 104, dev=1)), dict(logits=Shape(BF, 416)), dict(V=105),
               dict(logits=Shape(BF, 4, 104, stride=(1, 4))), dict(out=(Shape(F32, 4), Shape(F32, 4))),
               dict(out=(Shape(I32, 4), Shape(F32, 5))), dict(out=(Shape(I32, 4, dev=1), Shape(F32, 4))),
               dict(rows_per_param=1 << 31), dict(u=Shape(F32, 4, stride=(2,)))):
        with pytest.raises(ValueError):
            d2.sample(**{**ok, **kw})
    assert len(calls) == 4
