"""dflash2_paged_attn over the row counts that the tensor-core kernels are built for (16, 32, 48, 64, 96 and 128 rows
per cached key), each with head dimensions 64, 128 and 256, with the attention weights.  Bounds as in
test_gpu_paged_attn."""
import math

import numpy as np
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case, attn64
from tests._util import cuda_or_skip
from tests.test_gpu_paged_attn import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(2, 8), (8, 4), (4, 6), (8, 6), (8, 8), (16, 4), (16, 6), (20, 4), (16, 8), (31, 4)])
def test_every_row_count(d, T, G):
    """Lengths of several tiles, so that both score buffers and both P buffers are used again, and a cut item."""
    check(Case(d + T + G, [T, 640 + T, 1500, 129], T, 2 * G, 2, d, 32), weights=True)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("T,G", [(8, 4), (8, 8), (16, 4), (16, 6), (16, 8)])
def test_every_row_count_with_positions_and_a_window(d, T, G):
    check(Case(d * T + G, [T, 700, 400], T, G, 1, d, 16, held=True), window=300, weights=True)
    check(Case(d * T + G, [T, 700, 400], T, G, 1, d, 16), window=130, causal=False, weights=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(8, 2), (8, 8), (16, 6), (16, 8)])
def test_values_that_are_not_finite_in_neighbouring_tiles(d, T, G):
    """The block's keys lie on both sides of a tile's edge and hold NaN and Inf that only later tokens see."""
    n = 256 + T // 2
    mk = lambda: Case(d + G, [n, 100], T, G, 1, d, 16)  # noqa: E731
    c, first = mk(), n - T
    nan_at, inf_at, col = first + 2, 256 + 1, d - 3          # tokens 2 and T / 2 + 1 are the first to see them
    pg, o = c.slot(0, nan_at)
    c.v[pg, 0, o, 5] = math.nan
    pg, o = c.slot(0, inf_at)
    c.v[pg, 0, o, col] = -math.inf
    c.v[pg, 0, o, 7] = math.inf
    dev = cuda_or_skip()
    out, lse = d2.paged_attn(c.q.to(dev), **c.on(dev))
    torch.cuda.synchronize()
    r_out, r_lse, _, pv, _ = attn64(mk(), d ** -0.5, True, 0)
    g = out.float().cpu().numpy()
    assert np.isnan(g[0, 2:, :, 5]).all()
    assert (g[0, T // 2 + 1:, :, col] == -math.inf).all() and (g[0, T // 2 + 1:, :, 7] == math.inf).all()
    fine = np.ones(g.shape, dtype=bool)
    fine[0, 2:, :, 5] = fine[0, T // 2 + 1:, :, col] = fine[0, T // 2 + 1:, :, 7] = False
    # two roundings to bf16 (p and the result) and the fp32 rest
    assert (np.abs(g - r_out)[fine] <= (2.0 ** -7 * pv + 1e-6)[fine]).all()
    np.testing.assert_allclose(lse.cpu().numpy(), r_lse, atol=1e-4)
    assert d2.device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("big", [1e15, 1e17, 1e18])
def test_scores_far_below_zero(dtype, d, big):
    """Scores of -1e30 and less are scores: equal ones give the mean of the values, whatever their size."""
    T, lens = 3, [3, 200, 700]
    c = Case(d, lens, T, 4, 2, d, 16, dtype)
    c.q[:] = big
    c.k[:] = -big
    dev = cuda_or_skip()
    out, lse = d2.paged_attn(c.q.to(dev), **c.on(dev))
    torch.cuda.synchronize()
    score = -float(c.q[0, 0, 0, 0]) * -float(c.k[0, 0, 0, 0]) * d * d ** -0.5
    assert torch.isfinite(lse).all() and (lse.double().cpu() / -abs(score) - 1).abs().max() <= 2.0 ** -18
    for b, n in enumerate(lens):
        for t in range(T):
            m = n - T + t + 1
            for h in range(4):
                V = c.gather(c.v, b, h // 2)[:m].double()
                lim = (2.0 ** -7 * (dtype == BF) + (m + 8) * 2.0 ** -24 + 2.0 ** -20) * V.abs().mean(0)
                assert ((out[b, t, h].double().cpu() - V.mean(0)).abs() <= lim).all()
    assert d2.device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("big", [3e3, 1e5, 1e8, 1e16])
def test_scores_far_apart(dtype, d, big):
    """Scores of 1e7 to 1e33 of either sign: the largest one takes it all, and its value comes out."""
    T, lens = 3, [40, 300, 700]
    c = Case(d + 1, lens, T, 4, 2, d, 16, dtype, sigma=big)
    c.q = (c.q.float() * big).to(dtype)
    dev = cuda_or_skip()
    out, lse = d2.paged_attn(c.q.to(dev), **c.on(dev))
    torch.cuda.synchronize()
    sure = 0
    for b, n in enumerate(lens):
        for t in range(T):
            m = n - T + t + 1
            for h in range(4):
                K, V = (c.gather(x, b, h // 2)[:m].double() for x in (c.k, c.v))
                x = K @ c.q[b, t, h].double() * d ** -0.5
                top = x.topk(2)
                off = float((K.abs() @ c.q[b, t, h].double().abs()).max()) * d ** -0.5 * (d + 4) * 2.0 ** -24
                assert abs(float(lse[b, t, h]) - float(top.values[0])) <= off + 2.0 ** -20 * abs(float(top.values[0])) + 1
                if float(top.values[0] - top.values[1]) <= 2 * off + 100:
                    continue               # two scores that fp32 may not tell apart
                sure += 1
                assert ((out[b, t, h].double().cpu() - V[top.indices[0]]).abs() <= 1e-6 * V.abs().max()).all()
    assert sure > 30 and d2.device_error() == 0


def test_a_block_of_more_outputs_than_31_bits():
    """127 tokens of 67000 heads of 256: the last row of a block lies more than 2^31 elements behind its first."""
    dev = cuda_or_skip()
    T, H, d, n, step = 127, 67000, 256, 8, 4000
    assert (T - 1) * H * d > 2 ** 31 - 1
    g = torch.Generator(device=dev).manual_seed(0)
    k, v = (torch.randn(1, H, n, d, generator=g, device=dev, dtype=BF) for _ in range(2))
    q = torch.randn(1, T, H, d, generator=g, device=dev, dtype=BF)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    out, lse = d2.paged_attn(q, d2.KVCache(k, v), i32(0)[None], i32(n), causal=False)
    for h in range(0, H, step):
        x = torch.einsum("thd,hsd->ths", q[0, :, h:h + step].float(), k[0, h:h + step].float()) * d ** -0.5
        want = torch.einsum("ths,hsd->thd", x.softmax(-1), v[0, h:h + step].float())
        big = torch.einsum("ths,hsd->thd", x.softmax(-1), v[0, h:h + step].float().abs())
        # p and the result rounded to bf16, and the fp32 rest
        assert ((out[0, :, h:h + step].float() - want).abs() <= 2.0 ** -7 * big + 2.0 ** -12).all()
        assert torch.allclose(lse[0, :, h:h + step], x.logsumexp(-1), rtol=2.0 ** -16, atol=2.0 ** -12)
    assert d2.device_error() == 0
