"""Sampling from given uniforms against its definition in 64 bits, and with the calls around it."""
import math

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from dflash_draft_selection_gb300 import synth
from tests import _decode as ref
from tests._util import cuda_or_skip, padded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# A draw whose uniform lies this close to a border of the distribution (or whose top_p lies as close to a running
# mass) is not compared: masses are held to 2^-45 of the largest and summed over at most 2^19 tokens.
NEAR = 1e-9


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check(z, u, T, k, p, mp, **kw):
    """One call against the definition, row by row.  T, k, p, mp: one entry per row."""
    rows = z.shape[0]
    params = d2.sampling_params(T, k, p, n=rows)
    token, prob = d2.sample(padded(z), u, params=params, min_p=torch.tensor(mp, device="cuda", dtype=F32), **kw)
    assert token.dtype is torch.int32 and prob.dtype is F32
    token, prob, us = token.tolist(), prob.tolist(), u.double().tolist()
    f = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
    compared = 0
    for r in range(rows):
        t, q, margin = ref.draw(z[r], us[r], f(T[r]), k[r], f(p[r]), f(mp[r]))
        if margin < NEAR:
            continue
        compared += 1
        assert token[r] == t, (r, token[r], t, margin, T[r], k[r], p[r], mp[r])
        # one rounding to f32, and the masses' units
        assert math.isnan(prob[r]) if math.isnan(q) else abs(prob[r] - q) <= (2.0 ** -24 + 2.0 ** -26) * q, (r, prob[r], q)
    assert compared >= 0.9 * rows
    return compared


KINDS = [(1.0, 0, 1.0, 0.0), (0.7, 20, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 100, 1.0, 0.05), (0.0, 0, 1.0, 0.0),
         (0.9, 0, 0.5, 0.02), (1.0, 1, 0.95, 0.0), (2.0, 700, 0.8, 0.001), (0.3, 0, 1.0, 0.3), (1.0, 0, 1.0, 1.0),
         (0.05, 5, 0.3, 0.0), (1.0, 3000, 0.999, 0.0), (8.0, 0, 0.7, 0.0)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 17, 100, 1000, 4096, 8205, 40000, 151936, 262151, 1 << 20])
def test_every_kind_of_request(V, dt):
    cuda_or_skip()
    g = gen(V)
    n = len(KINDS) * (3 if V < 200000 else 1)
    z = torch.randn(n, V, generator=g, device="cuda") * 2
    z[1::3] = synth.spike_logits(len(z[1::3]), V, g, "cuda") if V > 16 else z[1::3]
    z = z.to(dt)
    if V > 2:
        z[2::3] = z[2::3].masked_fill(torch.rand(len(z[2::3]), V, generator=g, device="cuda") < 0.4, -math.inf)
        z[2::3, V // 2] = 1.0
    u = torch.rand(n, generator=g, device="cuda")
    kinds = [KINDS[i % len(KINDS)] for i in range(n)]
    check(z, u, *[list(c) for c in zip(*kinds)])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 5, 40, 153, 400])
def test_batches(rows, dt):
    cuda_or_skip()
    g = gen(rows)
    z = (torch.randn(rows, 3001, generator=g, device="cuda") * 3).to(dt)
    u = torch.rand(rows, generator=g, device="cuda")
    kinds = [KINDS[(i * 5 + rows) % len(KINDS)] for i in range(rows)]
    check(z, u, *[list(c) for c in zip(*kinds)])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [64, 5000, 70000])
def test_ties(V, dt):
    """Rows of one value, of two and of few; zeros of both signs.  Ties are ranked by id."""
    cuda_or_skip()
    g = gen(V)
    rows = []
    for i in range(4):
        rows += [torch.full((V,), 2.5), torch.where(torch.rand(V) < 0.5, 1.0, 0.0), torch.randint(0, 4, (V,)).float(),
                 torch.where(torch.rand(V) < 0.5, 0.0, -0.0), torch.cat([torch.zeros(V - 1), torch.ones(1)])]
    z = torch.stack(rows).to("cuda").to(dt)
    n = len(rows)
    # uniforms in the middle between the borders of the evenly weighted rows
    u = (torch.randint(0, V, (n,), generator=g, device="cuda").float() + 0.5) / V
    for T, k, p, mp in [(1.0, 0, 1.0, 0.0), (1.0, V // 2, 1.0, 0.0), (1.0, 0, 0.777, 0.0), (0.5, V // 3, 0.6, 0.9),
                        (0.0, 0, 1.0, 0.0)]:
        check(z, u, [T] * n, [k] * n, [p] * n, [mp] * n)


@pytest.mark.parametrize("dt", [BF, F32])
def test_values_close_together_and_far_apart(dt):
    """Logits that differ in their last bits, of every magnitude, and rows whose best token holds nearly all."""
    cuda_or_skip()
    V, g = 9000, gen(3)
    base = torch.randn(V, generator=g, device="cuda")
    rows = [100 + base * 1e-3, -3e4 + base * 50, base * 1e-30, base * 1e30, base * 2.0 ** -130,
            torch.arange(V, device="cuda") * -1e-4, torch.cat([torch.full((1,), 30.0, device="cuda"), base[1:]]),
            base.sign() * 10.0 ** (torch.rand(V, generator=g, device="cuda") * 12 - 8)]
    z = torch.stack(rows).to(dt)
    n = len(rows)
    for i, (T, k, p, mp) in enumerate([(1.0, 0, 1.0, 0.0), (0.01, 0, 0.9, 0.0), (1.0, 50, 0.9, 0.1), (30.0, 0, 0.99, 0.0),
                                       (1e-30, 0, 0.9, 0.0), (1e30, 0, 0.9, 0.0)]):
        u = torch.rand(n, generator=gen(50 + i), device="cuda")
        check(z, u, [T] * n, [k] * n, [p] * n, [mp] * n)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [50, 40000])
def test_uniforms_at_the_ends(V, dt):
    cuda_or_skip()
    u = torch.tensor([0.0, 2.0 ** -149, 1.0 - 2.0 ** -24, 1.0, -1.0, 2.0, math.inf, -math.inf, math.nan], device="cuda")
    n = len(u)
    z = (torch.randn(1, V, generator=gen(V), device="cuda") * 2).to(dt).expand(n, V).contiguous()
    z[:, 7] = 9.0                # the first token of the ranking
    for kind in ((1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 13, 1.0, 0.0)):
        params = d2.sampling_params(*kind[:3], n=n)
        token, prob = d2.sample(padded(z), u, params=params)
        token = token.tolist()
        first, last = ref.draw(z[0], 0.0, *kind)[0], ref.draw(z[0], 2.0, *kind)[0]
        assert token[:2] == [first, first] and token[4] == token[7] == first == 7
        assert token[3] == token[5] == token[6] == last
        if V == 50:                              # the last token's share is well above 2^-24
            assert token[2] == last and (kind[2] < 1 or last != first)
        assert token[8] == -1 and prob[8].isnan()
        assert prob[:8].isfinite().all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [300, 50000])
def test_bad_rows_alone_are_refused(V, dt):
    cuda_or_skip()
    nan, inf = math.nan, math.inf
    z = (torch.randn(16, V, generator=gen(1), device="cuda") * 2).to(dt)
    z[0, V - 1] = nan
    z[1, 0] = inf
    z[2] = -inf
    z[3, :] = -inf
    z[3, V // 3] = -5.0
    z[15, 3] = nan
    T = [1.0] * 4 + [-1.0, nan, inf, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.0]
    k = [0] * 7 + [-1] + [0] * 8
    p = [1.0] * 8 + [0.0, 1.5, nan] + [1.0] * 5
    mp = [0.0] * 11 + [-0.1, 1.5, nan, 0.0, 0.0]
    u = torch.rand(16, generator=gen(2), device="cuda")
    token, prob = d2.sample(padded(z), u, params=d2.sampling_params(T, k, p), min_p=torch.tensor(mp, device="cuda"))
    good = [3, 14]
    for r in range(16):
        if r in good:
            assert token[r] == ref.draw(z[r], float(u[r]))[0]
        else:
            assert token[r] == -1 and prob[r].isnan(), r
    assert token[3] == V // 3 and prob[3] == 1
    # without parameters every row is greedy
    token, prob = d2.sample(padded(z), u)
    assert token[4:15].tolist() == z[4:15].float().argmax(1).tolist() and (prob[3:15] == 1).all()
    assert token[:3].tolist() == [-1, -1, -1]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [17, 1003, 70001])
def test_only_the_first_V_entries_of_a_row_count(V, dt):
    """Rows further apart than they are long, with NaN between; a slice's V; a single row at the end of its memory."""
    cuda_or_skip()
    g = gen(V)
    z = (torch.randn(6, V, generator=g, device="cuda") * 2).to(dt)
    wide = torch.full((6, (V + 95) // 64 * 64 + 64), math.nan, device="cuda", dtype=dt)
    wide[:, :V] = z
    u = torch.rand(6, generator=g, device="cuda")
    params = d2.sampling_params([1.0], [0], [0.9])
    want = d2.sample(padded(z), u, params=params, rows_per_param=6)
    for got in (d2.sample(wide[:, :V], u, params=params, rows_per_param=6),
                d2.sample(wide, u, params=params, rows_per_param=6, V=V)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for r in range(6):
        one = d2.sample(z[r:r + 1].clone(), u[r:r + 1].clone(), params=params)
        assert one[0] == want[0][r] and one[1] == want[1][r]


def test_a_row_does_not_depend_on_its_batch():
    """The same bits alone, in batches of every size and from either end."""
    cuda_or_skip()
    V, g = 151936, gen(11)
    z = synth.spike_logits(200, V, g, "cuda").bfloat16()
    u = torch.rand(200, generator=g, device="cuda")
    kinds = [KINDS[i % len(KINDS)] for i in range(200)]
    T, k, p, mp = [list(c) for c in zip(*kinds)]
    mp = torch.tensor(mp, device="cuda")
    rec = lambda a, b: d2.sampling_params(T[a:b], k[a:b], p[a:b])  # noqa: E731
    token, prob = d2.sample(z, u, params=rec(0, 200), min_p=mp)
    for a, b in ((0, 1), (3, 4), (0, 2), (5, 12), (13, 50), (100, 200), (199, 200), (64, 141)):
        t, q = d2.sample(z[a:b], u[a:b].clone(), params=rec(a, b), min_p=mp[a:b].clone())
        assert torch.equal(t, token[a:b]) and torch.equal(q, prob[a:b])


def test_rows_that_share_parameters():
    cuda_or_skip()
    g = gen(12)
    z = (torch.randn(10, 999, generator=g, device="cuda") * 2).bfloat16()
    u = torch.rand(10, generator=g, device="cuda")
    T, k, p, mp = [0.5, 1.0, 0.0, 1.5], [0, 30, 0, 0], [0.9, 1.0, 1.0, 0.8], [0.0, 0.02, 0.0, 0.1]
    mpt = torch.tensor(mp, device="cuda")
    a = d2.sample(padded(z), u, params=d2.sampling_params(T, k, p), min_p=mpt, rows_per_param=3)
    at = [r // 3 for r in range(10)]
    b = d2.sample(padded(z), u, params=d2.sampling_params([T[i] for i in at], [k[i] for i in at], [p[i] for i in at]),
                  min_p=mpt[at].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    cuda_or_skip()
    z = torch.zeros(5, 1 << 30, dtype=BF, device="cuda")
    part = (torch.randn(5, 1000, generator=gen(1), device="cuda") * 2).bfloat16()
    z[:, :1000] = part
    u = torch.rand(5, generator=gen(2), device="cuda")
    params = d2.sampling_params([1.0] * 5, [40] * 5, [0.9] * 5)
    a, b = d2.sample(z, u, params=params, V=1000), d2.sample(padded(part), u, params=params)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_frequencies():
    """Evenly spread uniforms give every token its share."""
    cuda_or_skip()
    n, V = 20000, 24
    z = torch.linspace(0, 3, V, device="cuda").bfloat16().expand(n, V).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    token, prob = d2.sample(z, u, params=d2.sampling_params([0.8], [0], [0.9]), rows_per_param=n)
    w = torch.softmax(z[0].double() / 0.8, 0)
    order = w.sort(descending=True)
    kept = order.indices[:int((order.values.cumsum(0) < float(torch.tensor(0.9))).sum()) + 1]
    share = torch.zeros(V, dtype=torch.float64, device="cuda")
    share[kept] = w[kept] / w[kept].sum()
    got = torch.bincount(token.long(), minlength=V).double() / n
    assert (got - share).abs().max() <= 1.0 / n       # a token's stretch holds its share of the points, one more or less
    assert ((prob.double() - share[token.long()]).abs() <= 2.0 ** -23 * prob).all()


def test_captured_and_on_another_stream():
    dev = cuda_or_skip()
    g = gen(5)
    z = (torch.randn(20, 30000, generator=g, device=dev) * 2).bfloat16()
    u = torch.rand(20, generator=g, device=dev)
    params = d2.sampling_params([1.0] * 20, [0, 20] * 10, [0.9] * 20)
    want = d2.sample(z, u, params=params)
    out = torch.full((20,), -7, dtype=torch.int32, device=dev), torch.full((20,), -7.0, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert d2.sample(z, u, params=params, out=out) is out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = d2.sample(z, u, params=params)
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    for got in (out, other):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    u2 = torch.rand(20, generator=g, device=dev)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], d2.sample(z, u2, params=params)[0])


def test_no_rows():
    cuda_or_skip()
    token, prob = d2.sample(torch.empty(0, 64, device="cuda"), torch.empty(0, device="cuda"))
    assert token.shape == prob.shape == (0,)
