"""4-bit weights and their products against their definitions in 64 bits."""
import math

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests import _decode as ref
from tests._util import cuda_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(N, K, group, zero, dtype=BF, seed=0):
    """Codes and scales as a checkpoint holds them; what lies behind K in a row's last bytes is arbitrary."""
    g = gen(seed)
    G = -(-K // group)
    codes = torch.randint(0, 256, (N, -(-K // 32) * 16), generator=g, device="cuda", dtype=torch.uint8)
    scale = ((0.5 + torch.rand(N, G, generator=g, device="cuda")) * torch.where(
        torch.rand(N, G, generator=g, device="cuda") < 0.1, -1.0, 1.0)).to(dtype)
    z = torch.randint(0, 16, (N, G), generator=g, device="cuda").to(dtype) if zero else None
    return d2.Weight4(codes, scale, z, K=K, group=group)


def check(y, x, w, what=""):
    """y against x . W^T.  Sums are of codes and of zero points apart (B bounds what they add up); f32 sums of K terms
    lose at most K halfsteps, a product taken on bf16 weights 2^-8 of every term, a bf16 result 2^-8 of itself."""
    W = ref.values(w)
    want = x.double() @ W.T
    zero = torch.full_like(W, 8.0) if w.zero is None else ref.per_column(w.zero, w.K, w.group)
    B = x.double().abs() @ ((ref.unpack(w).double() + zero.abs()) * ref.per_column(w.scale, w.K, w.group).abs()).T
    tol = (w.K + 16) * 2.0 ** -24 * B
    if y.dtype is BF:
        tol += 2.0 ** -8 * (want.abs() + x.double().abs() @ W.abs().T)
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), ((y.double() - want).abs() / tol).max().item())
    # and the whole: independent roundings add up as squares do
    if want.numel() >= 64:
        rel = float((y.double() - want).norm() / want.norm())
        assert rel <= (2.0 ** -8 if y.dtype is BF else 2.0 ** -18), (what, rel)


# ------------------------------------------------------------------ quant ----
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("side", [BF, F32])
@pytest.mark.parametrize("group,zero", [(32, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (17, 33), (5, 128), (64, 321), (130, 2560), (2, 5120)])
def test_quant_is_the_definition(N, K, group, zero, dt, side):
    cuda_or_skip()
    W = (torch.randn(N, K, generator=gen(N + K), device="cuda") * 0.02).to(dt)
    W[0, : K // 2] = 0
    w = d2.quant4(W, group=group, zero=zero, dtype=side)
    code, scale, z = ref.quantised(W, group, zero, side)
    assert torch.equal(w.scale, scale) and (z is None) == (w.zero is None)
    assert z is None or torch.equal(w.zero, z)
    assert torch.equal(ref.unpack(w), code)
    assert (w.codes[:, (K + 1) // 2:] == 0x88).all() and (K % 2 == 0 or (w.codes[:, K // 2] >> 4 == 8).all())
    for out in (BF, F32):
        got = d2.dequant4(w, dtype=out)
        zf = torch.full_like(w.scale, 8.0) if z is None else z
        want = (code.float() - ref.per_column(zf, K, group).float()) * ref.per_column(scale, K, group).float()
        assert got.dtype is out and torch.equal(got, want.to(out))


def test_quant_extremes():
    cuda_or_skip()
    big = torch.finfo(F32).max
    rows = [[0.0] * 32, [1.0] * 32, [-2.0] * 32, [math.nan] + [1.0] * 31, [math.inf] + [1.0] * 31, [-math.inf] * 32,
            [big, -big] * 16, [1e-40, -1e-40] * 16, [2.0 ** -149] * 32, [7.0, -7.0, 0.5, -0.5] * 8, [-8.0] + [7.0] * 31]
    W = torch.tensor(rows, device="cuda")
    for zero in (False, True):
        for side in (BF, F32):
            w = d2.quant4(W, group=32, zero=zero, dtype=side)
            code, scale, z = ref.quantised(W, 32, zero, side)
            assert torch.equal(ref.unpack(w), code)
            assert torch.equal(w.scale.isnan(), scale.isnan())
            assert torch.equal(w.scale.nan_to_num(0), scale.nan_to_num(0)) and (z is None or torch.equal(w.zero, z))
            got = d2.dequant4(w, dtype=F32)
            assert torch.equal(got.isnan().any(1), torch.tensor([i in (3, 4, 5) for i in range(len(rows))], device="cuda"))


def test_quant_takes_strided_weights_and_fills_strided_records():
    cuda_or_skip()
    W = torch.randn(40, 300, generator=gen(1), device="cuda", dtype=BF)
    part = W[3:37, 5:261]
    codes = torch.full((40, 256), 0xAA, dtype=torch.uint8, device="cuda")
    scale = torch.full((40, 9), -1.0, dtype=BF, device="cuda")
    w = d2.Weight4(codes[2:36, 16:160], scale[2:36, 1:5], None, K=256, group=64)
    assert d2.quant4(part, out=w) is w
    want = d2.quant4(part.contiguous(), group=64)
    assert torch.equal(w.codes[:, :128], want.codes) and torch.equal(w.scale, want.scale)
    keep = torch.ones_like(codes, dtype=torch.bool)
    keep[2:36, 16:144] = False
    assert (codes[keep] == 0xAA).all()
    keep = torch.ones_like(scale, dtype=torch.bool)
    keep[2:36, 1:5] = False
    assert (scale[keep] == -1).all()
    out = torch.full((40, 300), -3.0, dtype=BF, device="cuda")
    d2.dequant4(w, out=out[3:37, 7:263])
    assert torch.equal(out[3:37, 7:263], d2.dequant4(want))
    out[3:37, 7:263] = -3.0
    assert (out == -3.0).all()


def test_any_zero_point_is_taken_back_with_one_rounding():
    cuda_or_skip()
    side = torch.tensor([[8.0, 0.0, -1.0, 15.0, 128.0, -128.0, 130.0, -130.0, 200.0, -255.0, 300.0, 7.5, 0.125, 1e20, -1e20,
                          math.inf, math.nan]], device="cuda", dtype=BF)
    G = side.shape[1]
    for dt in (BF, F32):
        w = d2.Weight4(torch.randint(0, 256, (5, 16 * G), generator=gen(1), device="cuda", dtype=torch.uint8),
                       (0.5 + torch.rand(5, G, generator=gen(2), device="cuda")).to(dt), side.to(dt).repeat(5, 1), K=32 * G,
                       group=32)
        want = (ref.unpack(w).float() - ref.per_column(w.zero, w.K, 32).float()) * ref.per_column(w.scale, w.K, 32).float()
        for out in (BF, F32):
            got = d2.dequant4(w, dtype=out)
            assert torch.equal(got.nan_to_num(nan=1e4), want.to(out).nan_to_num(nan=1e4))


def test_the_longest_row():
    """A row whose columns come next to 2^31."""
    cuda_or_skip()
    K, end = (1 << 31) - 129, (1 << 31) - 512
    W = torch.zeros(1, K, dtype=BF, device="cuda")
    tail = torch.randn(1, K - end, generator=gen(1), device="cuda", dtype=BF)
    W[:, end:] = tail
    w, last = d2.quant4(W), d2.quant4(tail)
    assert torch.equal(w.codes[:, end // 2:], last.codes) and torch.equal(w.scale[:, end // 128:], last.scale)
    assert (w.codes[:, :end // 2] == 0x88).all() and (w.scale[:, :end // 128] == 0).all()
    W.fill_(1.0)
    d2.dequant4(w, out=W)
    assert torch.equal(W[:, end:], d2.dequant4(last))
    assert (W[:, :end] == 0).all()


# --------------------------------------------------------------- products ----
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("N,K,group,zero", [(1, 1, 32, False), (15, 31, 32, True), (16, 64, 64, False), (130, 200, 64, True),
                                            (257, 1024, 128, False), (333, 1312, 32, True), (2560, 2560, 128, True),
                                            (48, 17408, 128, False)])
def test_products_bf16(rows, N, K, group, zero):
    cuda_or_skip()
    w = weights(N, K, group, zero, seed=N)
    x = torch.randn(rows, K, generator=gen(rows), device="cuda", dtype=BF)
    check(d2.linear4(x, w), x, w, "bf16")
    check(d2.linear4(x, w, dtype=F32), x, w, "f32 out")
    assert d2.device_error() == 0


@pytest.mark.parametrize("rows", [17, 31, 32, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K,group,zero,side", [(4096, 200, 64, True, BF), (4100, 1312, 32, True, F32), (4223, 31, 32, False, BF),
                                                 (8000, 2560, 128, False, BF), (25000, 520, 128, True, F32)])
def test_products_of_many_rows(rows, N, K, group, zero, side):
    """Wide enough for the tensor cores' tiles: one and several to a CTA, the last ones cut."""
    cuda_or_skip()
    w = weights(N, K, group, zero, side, seed=N)
    x = torch.randn(rows, K, generator=gen(rows), device="cuda", dtype=BF)
    check(d2.linear4(x, w), x, w, "bf16")
    check(d2.linear4(x, w, dtype=F32), x, w, "f32 out")
    assert d2.device_error() == 0


@pytest.mark.parametrize("rows", [1, 3, 8, 20, 70])
@pytest.mark.parametrize("N,K,group,zero,side", [(1, 5, 32, False, F32), (129, 264, 32, True, F32), (500, 1024, 128, False, BF),
                                                 (64, 9000, 64, True, BF)])
def test_products_f32(rows, N, K, group, zero, side):
    cuda_or_skip()
    w = weights(N, K, group, zero, side, seed=N)
    x = torch.randn(rows, K, generator=gen(rows), device="cuda")
    check(d2.linear4(x, w), x, w)


@pytest.mark.parametrize("rows", [9, 16, 17, 32, 33, 100, 300])
@pytest.mark.parametrize("N,K,group,zero,side", [(11000, 200, 64, True, BF), (10925, 1312, 32, True, F32), (11223, 31, 32, False, BF),
                                                 (12000, 2560, 128, False, BF), (25000, 520, 128, True, F32)])
def test_products_of_many_f32_rows(rows, N, K, group, zero, side):
    """Wide enough for the tensor cores' tiles: one and several to a CTA, the last ones cut."""
    cuda_or_skip()
    w = weights(N, K, group, zero, side, seed=N)
    x = torch.randn(rows, K, generator=gen(rows), device="cuda")
    check(d2.linear4(x, w), x, w)
    ws = d2.Workspace.for_linear4(rows, N, K, F32)
    assert ws.nbytes > 16
    check(d2.linear4(x, w, ws=ws), x, w)
    assert d2.device_error() == 0


@pytest.mark.parametrize("rows", [1, 8, 40, 200])
def test_products_of_a_wide_head(rows):
    """More weight rows than the GPU has warps; N odd, so that output rows are not aligned."""
    cuda_or_skip()
    w = weights(70001, 640, 128, False, seed=5)
    x = torch.randn(rows, 640, generator=gen(rows), device="cuda", dtype=BF)
    check(d2.linear4(x, w), x, w)


def test_long_rows():
    """More columns than a CTA's share of x holds."""
    cuda_or_skip()
    for rows, K, dt in ((1, 70016, BF), (8, 65536, BF), (3, 40000, F32)):
        w = weights(33, K, 128, True, seed=K)
        x = torch.randn(rows, K, generator=gen(K), device="cuda", dtype=dt)
        check(d2.linear4(x, w, dtype=F32), x, w, K)


@pytest.mark.parametrize("N", [193, 4097])
@pytest.mark.parametrize("rows", [1, 8, 30, 100])
def test_strides(rows, N):
    """x cut out of a wider matrix at an odd column, outputs into one, weight rows and columns of a larger record."""
    cuda_or_skip()
    for dt in (BF, F32):
        big = weights(N + 100, 1024, 64, True, seed=2)
        at = slice(7, 7 + N)
        w = d2.Weight4(big.codes[at, 64:384], big.scale[at, 2:12], big.zero[at, 2:12], K=640, group=64)
        for a in (0, 1, 8):
            x = torch.randn(rows, 700, generator=gen(rows), device="cuda", dtype=dt)[:, a:a + 640]
            out = torch.full((rows + 2, N + 37), 77.0, device="cuda", dtype=dt)
            got = out[1:-1, 3:3 + N]
            assert d2.linear4(x, w, out=got) is got
            check(got, x, w, (rows, dt, a))
            got.fill_(77.0)
            assert (out == 77.0).all()


@pytest.mark.parametrize("N", [100, 4096])
@pytest.mark.parametrize("rows", [1, 8, 24, 100])
def test_magnitudes(rows, N):
    """Rows of every magnitude, with entries far smaller than their largest; a row of zeros; one huge entry."""
    cuda_or_skip()
    w = weights(N, 512, 128, True, seed=3)
    g = gen(9)
    x = torch.randn(rows, 512, generator=g, device="cuda")
    x *= 10.0 ** (torch.arange(rows, device="cuda")[:, None] * 61 % 60 - 30).float()
    x[:, ::7] *= 2.0 ** -30
    if rows > 2:
        x[1] = 0
        x[2, 5] = 2.0 ** 100
    for y, xx in ((d2.linear4(x.bfloat16(), w, dtype=F32), x.bfloat16()), (d2.linear4(x, w), x)):
        W = ref.values(w)
        want = xx.double() @ W.T
        zero = ref.per_column(w.zero, w.K, w.group)
        B = xx.double().abs() @ ((ref.unpack(w).double() + zero) * ref.per_column(w.scale, w.K, w.group).abs()).T
        # Rows are scaled so that their largest entry lies in 2^125 .. 2^127 and codes are taken times 2^-133, so a
        # product's f32 (units of 2^-149) drops entries below 2^-16 of those: 2^-141 of the largest, for each of the
        # 512 terms, with codes and scales beside them.
        drop = 512 * 2.0 ** -140 * xx.double().abs().amax(1, keepdim=True) * w.scale.double().abs().amax(1)
        assert ((y.double() - want).abs() <= (512 + 16) * 2.0 ** -24 * B + drop + 2.0 ** -149).all()
        if rows > 2:
            assert (y[1] == 0).all()


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("rows", [9, 24, 100])
def test_magnitudes_of_bf16_results(rows, zero):
    """Rows from 2^-120 to 2^90 against weights of the tensor cores' tiles, scales from 2^-80 to 2^20."""
    cuda_or_skip()
    w = weights(4096, 512, 128, zero, seed=3)
    w.scale.mul_(torch.tensor([2.0 ** -80, 2.0 ** -20, 1.0, 2.0 ** 20], device="cuda")[torch.arange(4096, device="cuda") % 4][:, None])
    x = torch.randn(rows, 512, generator=gen(9), device="cuda")
    x *= torch.exp2((torch.arange(rows, device="cuda")[:, None] * 61 % 211 - 120).float())
    x = x.bfloat16()
    x[1] = 0
    W = ref.values(w)
    want = x.double() @ W.T
    z = torch.full_like(W, 8.0) if w.zero is None else ref.per_column(w.zero, w.K, w.group)
    B = x.double().abs() @ ((ref.unpack(w).double() + z) * ref.per_column(w.scale, w.K, w.group).abs()).T
    # f32 sums, bf16 weights, a bf16 result as elsewhere; results next to bf16's least are whole multiples of 2^-133, and
    # what f32 drops in between (2^-149) is less than 2^-140 of that
    tol = (512 + 16) * 2.0 ** -24 * B + 2.0 ** -8 * (want.abs() + x.double().abs() @ W.abs().T) + 2.0 ** -133
    got = d2.linear4(x, w)
    assert ((got.double() - want).abs() <= tol).all()
    assert (got[1] == 0).all()


@pytest.mark.parametrize("N", [200, 4096])
@pytest.mark.parametrize("rows", [2, 8, 24, 100])
def test_a_row_with_nan_or_infinity_is_nan_alone(rows, N):
    cuda_or_skip()
    w = weights(N, 384, 128, False, seed=4)
    for dt in (BF, F32):
        x = torch.randn(rows, 384, generator=gen(rows), device="cuda", dtype=dt)
        want = d2.linear4(x, w)
        for v in (math.nan, math.inf, -math.inf):
            y = x.clone()
            y[1, 200] = v
            got = d2.linear4(y, w)
            assert got[1].isnan().all()
            got[1] = want[1]
            assert torch.equal(got, want)


def test_a_nan_scale_is_its_weight_rows_alone():
    cuda_or_skip()
    for rows, N in ((1, 200), (8, 200), (100, 200), (100, 4096)):
        w = weights(N, 384, 128, False, seed=4)
        x = torch.randn(rows, 384, generator=gen(rows), device="cuda", dtype=BF)
        want = d2.linear4(x, w)
        w.scale[17, 1] = math.nan
        got = d2.linear4(x, w)
        assert got[:, 17].isnan().all()
        got[:, 17] = want[:, 17]
        assert torch.equal(got, want)


def test_empty_products():
    cuda_or_skip()
    w = weights(20, 64, 64, False)
    assert d2.linear4(torch.empty(0, 64, device="cuda", dtype=BF), w).shape == (0, 20)
    none = d2.Weight4(w.codes[:0], w.scale[:0], None, K=64, group=64)
    assert d2.linear4(torch.zeros(3, 64, device="cuda", dtype=BF), none).shape == (3, 0)
    assert d2.dequant4(none).shape == (0, 64)
    d2.quant4(torch.empty(0, 64, device="cuda"), out=none)


def test_offsets_past_32_bits():
    """Rows of codes, of x and of outputs that lie more than 2^32 bytes apart in all."""
    cuda_or_skip()
    N, K, rows = 70, 96, 40
    ref_w = weights(N, K, 32, False, seed=6)
    codes = torch.zeros(N, 1 << 26, dtype=torch.uint8, device="cuda")
    codes[:, :48] = ref_w.codes
    w = d2.Weight4(codes, ref_w.scale, None, K=K, group=32)
    x = torch.randn(rows, K, generator=gen(1), device="cuda", dtype=BF)
    want, one = d2.linear4(x, ref_w), d2.linear4(x[:1], ref_w)
    assert torch.equal(d2.linear4(x, w), want) and torch.equal(d2.linear4(x[:1], w), one)
    del codes, w
    far = torch.zeros(rows, 1 << 26, dtype=BF, device="cuda")
    far[:, :K] = x
    assert torch.equal(d2.linear4(far[:, :K], ref_w), want)
    d2.linear4(x, ref_w, out=far[:, 100:100 + N])
    assert torch.equal(far[:, 100:100 + N], want)


@pytest.mark.parametrize("rows", [1, 8, 64, 300])
def test_calls_are_repeatable_and_captured(rows):
    """The same bits every time, from a graph and from another stream too; a row's outputs do not depend on NaNs beside
    it or on what the outputs held."""
    dev = cuda_or_skip()
    w = weights(5000, 1280, 64, True, seed=8)
    x = torch.randn(rows, 1280, generator=gen(rows), device=dev, dtype=BF)
    want = d2.linear4(x, w)
    out = torch.full_like(want, math.nan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d2.linear4(x, w, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.fill_(math.nan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d2.linear4(x, w, out=out)
    for _ in range(3):
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    x2 = torch.randn(rows, 1280, generator=gen(77), device=dev, dtype=BF)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, d2.linear4(x2, w))
    assert d2.device_error() == 0


@pytest.mark.parametrize("dt", [BF, F32])
def test_two_streams_and_two_graphs(dt):
    """Calls at one time, each with its workspace; two graphs that share one, replayed in turn."""
    dev = cuda_or_skip()
    w = [weights(9000, 640, 64, True, seed=s) for s in (1, 2)]
    x = [torch.randn(40, 640, generator=gen(s), device=dev, dtype=dt) for s in (3, 4)]
    want = [d2.linear4(a, b) for a, b in zip(x, w)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [d2.Workspace.for_linear4(40, 9000, 640, dt) for _ in range(2)]
    out = [torch.full_like(want[0], math.nan) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d2.linear4(x[i], w[i], ws=ws[i], out=out[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        out[i].fill_(math.nan)
        with torch.cuda.graph(g):
            d2.linear4(x[i], w[i], ws=ws[0], out=out[i])
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert d2.device_error() == 0
