"""dflash2_linear4 at the widths of the library's models, from a few rows to thousands: the products of a row of x do not
depend on how many rows are beside it."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests import _decode as ref
from tests._util import cuda_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(rows, N, K, group, zero, side=BF, seed=0):
    """x and weights whose products and sums are exact in f32: x whole up to 4, scales odd multiples of 2^-7 (8 bits, so
    that few weights are bf16 numbers), zero points multiples of a half.  In units of 2^-8 a product stays below 2^17, a
    group's sum below 2^24, and the sums of K <= 20000 terms within 2^24 by more than 10 standard deviations (a term's is
    2^13 at most)."""
    g = gen(seed)
    G = -(-K // group)
    codes = torch.randint(0, 256, (N, -(-K // 32) * 16), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.randint(64, 128, (N, G), generator=g, device="cuda") * 2 + 1) / 128
    scale = (scale * (1 - 2 * torch.randint(0, 2, (N, G), generator=g, device="cuda"))).to(side)
    z = (torch.randint(0, 31, (N, G), generator=g, device="cuda") / 2).to(side) if zero else None
    x = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").float()
    return x, d2.Weight4(codes, scale, z, K=K, group=group)


def products(x, w):
    """x . W^T in 64 bits: exact."""
    want = torch.cat([x[a:a + 8192].double() @ ref.values(w).T for a in range(0, x.shape[0], 8192)])
    assert float(want.abs().max()) * 256 < 2 ** 24
    return want


@pytest.mark.parametrize("N,K,group,zero,side", [(20011, 5120, 32, True, BF), (20011, 5120, 64, False, BF),
                                                 (20011, 5120, 128, True, BF), (20011, 5120, 128, False, F32),
                                                 (20000, 17408, 128, False, BF), (20000, 17408, 32, True, BF)])
def test_a_row_has_the_same_products_beside_others(N, K, group, zero, side):
    """Few rows, and the tensor cores' kernel with blocks of 16, 64 and 128 rows: one rounding from the exact products."""
    cuda_or_skip()
    x, w = whole(512, N, K, group, zero, side)
    want = products(x, w)
    for rows in (1, 8, 9, 64, 65, 512):
        assert torch.equal(d2.linear4(x[:rows].to(BF), w), want[:rows].to(BF)), rows
        assert torch.equal(d2.linear4(x[:rows].to(BF), w, dtype=F32), want[:rows].float()), rows
    for rows in (8, 9, 64):
        assert torch.equal(d2.linear4(x[:rows], w), want[:rows].float()), rows
    assert d2.device_error() == 0


@pytest.mark.parametrize("group,zero", [(32, True), (64, True), (128, False)])
def test_thousands_of_rows(group, zero):
    cuda_or_skip()
    x, w = whole(2100, 1500, 5120, group, zero)
    want = products(x, w)
    assert torch.equal(d2.linear4(x.to(BF), w), want.to(BF))
    assert torch.equal(d2.linear4(x.to(BF), w, dtype=F32), want.float())
    assert torch.equal(d2.linear4(x, w), want.float())
    assert d2.device_error() == 0


def test_scales_of_any_size():
    """Scales from 2^-90 to 2^100 against rows that bring the results back into range."""
    cuda_or_skip()
    x, w = whole(70, 4096, 640, 64, True)
    want = products(x, w)
    for e in (-90, 40, 100):
        far = d2.Weight4(w.codes, w.scale * 2.0 ** e, w.zero, K=640, group=64)
        for rows in (1, 8, 9, 70):
            xs = (x[:rows] * 2.0 ** -(e // 2)).to(BF)
            # ^(e - e // 2) is left, an exact factor
            scaled = want[:rows] * 2.0 ** (e - e // 2)
            assert torch.equal(d2.linear4(xs, far), scaled.to(BF)), (e, rows)
            assert torch.equal(d2.linear4(xs, far, dtype=F32), scaled.float()), (e, rows)


# ------------------------------------------------- weights rounded to bf16 ----
@pytest.mark.parametrize("N,K,group,zero", [(4096, 200, 64, True), (20011, 5120, 32, True), (20011, 5120, 128, False),
                                            (4223, 31, 32, False)])
@pytest.mark.parametrize("rows", [1, 8, 9, 33, 64, 130, 512])
def test_rounded_weights_on_request(rows, N, K, group, zero):
    cuda_or_skip()
    from tests.test_gpu_weight4 import check, weights
    w = weights(N, K, group, zero, seed=N)
    x = torch.randn(rows, K, generator=gen(rows), device="cuda", dtype=BF)
    y, own = d2.linear4(x, w, rounded=True), d2.linear4(x, w)
    check(y, x, w, "rounded")
    assert torch.equal(y, d2.linear4(x, w, rounded=True))
    # few rows keep their bits, and whatever else is asked for
    if d2.Workspace.for_linear4(rows, N, K).nbytes <= 16:
        assert torch.equal(y, own)
    elif K == 5120:
        assert not torch.equal(y, own)
    assert torch.equal(d2.linear4(x, w, dtype=F32, rounded=True), d2.linear4(x, w, dtype=F32))
    side = d2.Weight4(w.codes, w.scale.float(), None if w.zero is None else w.zero.float(), K=K, group=group)
    assert torch.equal(d2.linear4(x, side, rounded=True), d2.linear4(x, side))
    if rows <= 64:
        assert torch.equal(d2.linear4(x.float(), w, rounded=True), d2.linear4(x.float(), w))
    assert d2.device_error() == 0


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("rows", [9, 24, 100])
def test_rounded_weights_refuse_scales_that_they_have_no_room_for(rows, zero):
    """Their weight rows alone are NaN; the range's ends and 0 are taken."""
    cuda_or_skip()
    from tests.test_gpu_weight4 import check, weights
    w = weights(4096, 512, 128, zero, seed=3)
    x = torch.randn(rows, 512, generator=gen(9), device="cuda", dtype=BF)
    w.scale[:, 1] = 0.0
    w.scale[::4] *= 2.0 ** -79
    w.scale[1::4] *= 2.0 ** 28
    w.scale[5, 0], w.scale[8, 2] = 2.0 ** 30, 2.0 ** -80
    y = d2.linear4(x, w, rounded=True)
    assert y.isfinite().all()
    check(y, x, w)
    want = y.clone()
    bad = {17: 2.0 ** 31, 100: -2.0 ** 90, 255: 2.0 ** -81, 256: 2.0 ** -133, 4000: float("inf"), 4095: float("nan")}
    for n, s in bad.items():
        w.scale[n, n % 4] = s
    if zero:
        w.zero[300, 2] = 2.0 ** 41
        bad[300] = None
    y = d2.linear4(x, w, rounded=True)
    for n in bad:
        assert y[:, n].isnan().all(), n
        y[:, n] = want[:, n]
    assert torch.equal(y, want)


def test_rounded_rows_that_are_not_finite():
    cuda_or_skip()
    from tests.test_gpu_weight4 import weights
    w = weights(4096, 384, 128, False, seed=4)
    x = torch.randn(70, 384, generator=gen(1), device="cuda", dtype=BF)
    x[5] = 0
    want = d2.linear4(x, w, rounded=True)
    assert (want[5] == 0).all()
    for v in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[1, 200] = v
        got = d2.linear4(y, w, rounded=True)
        assert got[1].isnan().all()
        got[1] = want[1]
        assert torch.equal(got, want)


def test_rounded_products_captured_and_with_a_workspace():
    dev = cuda_or_skip()
    from tests.test_gpu_weight4 import weights
    w = weights(9000, 640, 64, True, seed=1)
    x = torch.randn(40, 640, generator=gen(3), device=dev, dtype=BF)
    ws = d2.Workspace.for_linear4(40, 9000, 640)
    want, out = d2.linear4(x, w, rounded=True), torch.empty(40, 9000, device=dev, dtype=BF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d2.linear4(x, w, ws=ws, out=out, rounded=True)
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert d2.device_error() == 0


@pytest.mark.parametrize("rows,N,K,group", [(9, 4096, 64, 32), (130, 25000, 520, 128)])
def test_rounded_products_give_up_and_recover(rows, N, K, group):
    """A bounded wait that runs out on the host's hook: NaN, the error word, and a context that stays usable."""
    dev = cuda_or_skip()
    from tests.test_gpu_wait_timeout import held
    from tests.test_gpu_weight4 import check, weights
    w = weights(N, K, group, True, seed=1)
    x = torch.randn(rows, K, generator=gen(rows), device=dev, dtype=BF)
    ws = d2.Workspace.for_linear4(rows, N, K)
    y = torch.zeros(rows, N, device=dev, dtype=BF)
    _, code = held(lambda: d2.linear4(x, w, ws=ws, out=y, rounded=True))
    assert code == 1   # DFLASH2_DEVERR_WAIT_TIMEOUT
    assert y.isnan().all()
    check(d2.linear4(x, w, ws=ws, out=y, rounded=True), x, w)
    assert d2.device_error() == 0
