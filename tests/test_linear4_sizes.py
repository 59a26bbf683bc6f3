"""Products that dflash2_linear4 and dflash2_linear4_rounded refuse for their size, and workspaces that they ask for (no GPU
needed: the pointers are never dereferenced)."""
import pytest

from tests.test_decode_arguments import BAD_RECORDS, INVALID, OK, UNSUPPORTED, WORKSPACE, library, record

F32, BF = 0, 1


def call(rounded, w=None, **kw):
    a = dict(x=4096, dt=BF, rows=3, x_stride=200, w=record(**(w or {})), y=4096, y_dt=BF, y_stride=40, ws=None, ws_bytes=0,
             stream=None)
    L = library()
    return (L.dflash2_linear4_rounded if rounded else L.dflash2_linear4)(*{**a, **kw}.values())


@pytest.mark.parametrize("rounded", [False, True])
def test_the_largest_products(rounded):
    """2^31 - 1 weight rows of 2^17 columns against 2^19 rows: more tiles than are counted."""
    big = dict(N=(1 << 31) - 1, K=1 << 17, code_stride=1 << 16, side_stride=1 << 10)
    kw = dict(rows=1 << 19, x_stride=1 << 17, y_stride=1 << 31)
    need = library().dflash2_linear4_workspace_bytes(BF, 1 << 19, big["N"], big["K"])
    assert need > 1 << 37
    assert call(rounded, big, **kw) == INVALID
    assert call(rounded, big, **kw, ws=4096, ws_bytes=need - 1) == WORKSPACE
    for out in (BF, F32):
        assert call(rounded, big, **kw, y_dt=out, ws=4096, ws_bytes=1 << 60) == UNSUPPORTED


@pytest.mark.parametrize("bad", BAD_RECORDS, ids=str)
def test_rounded_products_check_their_records(bad):
    assert call(True, bad) == INVALID


def test_rounded_products_check_their_arguments():
    for kw in (dict(x=None), dict(y=None), dict(x=4097), dict(y=4097), dict(rows=-1), dict(x_stride=199), dict(y_stride=39),
               dict(dt=F32, y_dt=BF), dict(y_dt=5), dict(dt=2), dict(y=4098, y_dt=F32)):
        assert call(True, **kw) == INVALID, kw
    assert call(True, rows=0, x=None, y=None) == call(True, dict(N=0, codes=None, scale=None)) == OK
    assert call(True, rows=(1 << 19) + 1) == UNSUPPORTED
