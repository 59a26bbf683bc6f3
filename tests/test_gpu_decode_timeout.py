"""Bounded waits of dflash2_linear4's kernel for many rows that run out, made on the host without a fault: the test hook keeps
the warp that copies x from its first copy until a word is set that nothing sets.  The kernel has to return, set the error
word, write NaN and leave the context usable."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._util import cuda_or_skip
from tests.test_gpu_wait_timeout import LIMIT, held
from tests.test_gpu_weight4 import check, gen, weights

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("rows,N,K,group", [(9, 4096, 64, 32), (40, 4200, 640, 64), (130, 25000, 520, 128)])
def test_products_give_up_and_recover(rows, N, K, group, out):
    """One block and many, one tile to a CTA and several."""
    dev = cuda_or_skip()
    w = weights(N, K, group, True, seed=1)
    x = torch.randn(rows, K, generator=gen(rows), device=dev, dtype=BF)
    ws = d2.Workspace.for_linear4(rows, N, K)
    assert ws.nbytes > 16
    y = torch.zeros(rows, N, device=dev, dtype=out)
    _, code = held(lambda: d2.linear4(x, w, ws=ws, out=y))
    assert code == 1   # DFLASH2_DEVERR_WAIT_TIMEOUT
    assert y.isnan().all()
    check(d2.linear4(x, w, ws=ws, out=y), x, w)
    assert d2.device_error() == 0


@pytest.mark.parametrize("rows", [16, 70])
def test_products_of_f32_rows_give_up_and_recover(rows):
    dev = cuda_or_skip()
    w = weights(11000, 640, 64, True, seed=1)
    x = torch.randn(rows, 640, generator=gen(rows), device=dev)
    ws = d2.Workspace.for_linear4(rows, 11000, 640, F32)
    assert ws.nbytes > 16
    y = torch.zeros(rows, 11000, device=dev)
    _, code = held(lambda: d2.linear4(x, w, ws=ws, out=y))
    assert code == 1   # DFLASH2_DEVERR_WAIT_TIMEOUT
    assert y.isnan().all()
    check(d2.linear4(x, w, ws=ws, out=y), x, w)
    assert d2.device_error() == 0


def test_a_hook_that_is_set_in_time_changes_nothing():
    dev = cuda_or_skip()
    w = weights(5000, 300, 128, False, seed=1)
    x = torch.randn(33, 300, generator=gen(2), device=dev, dtype=BF)
    want = d2.linear4(x, w)
    flag = torch.ones(1, dtype=torch.int32, device=dev)
    d2.test_hold(flag, LIMIT)
    try:
        got = d2.linear4(x, w)
    finally:
        d2.test_hold(None)
    assert torch.equal(got, want) and d2.device_error() == 0
