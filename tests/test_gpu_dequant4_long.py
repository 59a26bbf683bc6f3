"""dflash2_dequant4 of few long rows, which are cut over warps: every value once, and nothing beside them."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests import _decode as ref
from tests._util import cuda_or_skip
from tests.test_gpu_weight4 import weights

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("N,K", [(1, 1024), (1, 1025), (1, 20481), (16, 20480), (17, 20483), (3, 300007), (2, 1 << 20), (1300, 1031),
                                 (9700, 2049), (5, 100), (700, 40)])
def test_long_rows(N, K, group, zero, dt):
    cuda_or_skip()
    w = weights(N, K, group, zero, seed=K)
    z = torch.full_like(w.scale, 8.0) if w.zero is None else w.zero
    want = ((ref.unpack(w).float() - ref.per_column(z, K, group).float()) * ref.per_column(w.scale, K, group).float()).to(dt)
    assert torch.equal(d2.dequant4(w, dtype=dt), want)
    for ld, a in ((K + 7, 3), ((K + 23) // 8 * 8, 8)):      # rows that start anywhere, and on 16 bytes
        out = torch.full((N + 2, ld + 16), 77.0, device="cuda", dtype=dt)
        part = out[1:-1, a:a + K]
        assert d2.dequant4(w, out=part) is part
        assert torch.equal(part, want)
        part.fill_(77.0)
        assert (out == 77.0).all()
