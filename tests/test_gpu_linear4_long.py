"""dflash2_linear4 for as many and as long rows as it takes: calls that bring a workspace are taken."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._util import cuda_or_skip
from tests.test_gpu_linear4_rows import BF, F32, products, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out,side", [(BF, BF), (F32, BF), (BF, F32)])
def test_few_weight_rows_for_many_long_rows(out, side):
    """2^16 rows of 2^14 columns against two weight rows: a workspace is asked for, and the kernel for few rows does not
    count as many blocks."""
    cuda_or_skip()
    rows, K = 1 << 16, 1 << 14
    x, w = whole(rows, 2, K, 128, False, side)
    want = products(x, w)
    ws = d2.Workspace.for_linear4(rows, 2, K)
    assert ws.nbytes > rows * K * 2
    assert torch.equal(d2.linear4(x.to(BF), w, dtype=out, ws=ws), want.to(out))
    assert d2.device_error() == 0


@pytest.mark.parametrize("N", [9800, 1 << 21])
def test_the_longest_columns_on_the_tensor_cores(N):
    """K next to 2^17, and weight rows past 2^21 of fewer columns."""
    cuda_or_skip()
    K = (1 << 17) - 5 if N == 9800 else 72
    x, w = whole(20, N, K, 128 if N == 9800 else 32, True)
    x[:, 20000:] = 0     # so that sums stay within 24 bits; the codes are read all the same
    want = products(x, w)
    assert torch.equal(d2.linear4(x.to(BF), w), want.to(BF))
    assert torch.equal(d2.linear4(x.to(BF), w, dtype=F32), want.float())
    assert d2.device_error() == 0
