"""Sampling where the rows' values leave the usual range, against the definition in 64 bits."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests import _decode as ref
from tests._util import cuda_or_skip, padded
from tests.test_gpu_sample import check, gen

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("M", [2.0 ** 39, 1e12, 1e13, 2.0 ** 60, 1e30])
@pytest.mark.parametrize("V", [1000, 40000])
def test_small_values_beside_a_huge_one(V, M, dt):
    """The largest logit is so large that values next to zero are past 6144 steps of bf16 from it; a temperature of its
    size gives them their mass all the same."""
    cuda_or_skip()
    g = gen(V)
    zeros = torch.zeros(V, device="cuda")
    tiny = torch.randn(V, generator=g, device="cuda") * 1e-3
    mixed = torch.where(torch.rand(V, generator=g, device="cuda") < 0.5, tiny, -M / 2)
    spread = torch.randn(V, generator=g, device="cuda") * M / 8
    base = torch.stack([zeros, tiny, mixed, torch.where(tiny > 0, spread, tiny)]).repeat(3, 1)
    base[:, V // 3] = M
    n = base.shape[0]
    for i, (T, k, p, mp) in enumerate([(M, 0, 1.0, 0.0), (M, 0, 0.9, 0.0), (M, 600, 1.0, 0.0), (M, 700, 0.9, 0.0),
                                       (M, 0, 0.95, 0.1), (M, 0, 0.95, 0.5), (M / 4, 0, 1.0, 0.0), (M, V - 1, 0.99, 0.0),
                                       (4 * M, 0, 0.5, 0.01)]):
        u = torch.rand(n, generator=gen(20 + i), device="cuda")
        check(base.to(dt), u, [T] * n, [k] * n, [p] * n, [mp] * n)


@pytest.mark.parametrize("dt", [BF, F32])
def test_differences_that_f32_does_not_hold(dt):
    """A logit of 16 and many whose difference from it takes 25 bits (a tie in f32): their masses are those of the exact
    difference.  Rounded it would move the mass by 2^-21 / T of itself."""
    cuda_or_skip()
    V, n = 150000, 8
    z = torch.full((n, V), 2.0 ** -14 + 2.0 ** -21, device="cuda")
    z[:, V // 2] = 16.0
    assert torch.equal(z.to(dt).float(), z)
    for i, (T, k, p, mp) in enumerate([(1.0, 0, 1.0, 0.0), (2.0, 0, 1.0, 0.0), (2.0, 0, 0.9, 0.0), (4.0, 0, 1.0, 0.0),
                                       (4.0, 0, 0.7, 0.0), (2.0, 5000, 1.0, 0.0), (4.0, 100, 1.0, 0.0)]):
        # uniforms in the middle of a token's share
        u = (torch.randint(0, 4096, (n,), generator=gen(i), device="cuda").float() + 0.5) / 4096
        check(z.to(dt), u, [T] * n, [k] * n, [p] * n, [mp] * n)


@pytest.mark.parametrize("dt", [BF, F32])
def test_temperatures_next_to_zero(dt):
    """Above 0 the least one is 2^-127: what lies between counts as that.  The logits are its size."""
    cuda_or_skip()
    V, n, least = 90, 24, 2.0 ** -127
    z = (torch.arange(V, device="cuda") * -2.0 ** -133).flip(0).expand(n, V).contiguous().to(dt)
    assert z.float().unique().numel() == V
    u = torch.rand(n, generator=gen(4), device="cuda")
    for k, p, mp in ((0, 1.0, 0.0), (30, 0.9, 0.0), (0, 0.8, 0.0), (0, 1.0, 0.5)):
        check(z, u, [least] * n, [k] * n, [p] * n, [mp] * n)
        rec = lambda T: d2.sampling_params([T] * n, [k] * n, [p] * n)  # noqa: E731
        m = torch.full((n,), mp, device="cuda")
        want = d2.sample(padded(z), u, params=rec(least), min_p=m)
        for T in (5e-39, 1e-40, 2.0 ** -149):
            got = d2.sample(padded(z), u, params=rec(T), min_p=m)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows,V", [(1, 151936), (40, 20000), (300, 9000), (64, 151936)])
@pytest.mark.parametrize("k", [513, 1000, 2100, 4096])
def test_top_k_past_the_short_list(k, rows, V):
    """f32 rows over several CTAs whose top_k is no short list: a floor, then bins."""
    cuda_or_skip()
    z = torch.randn(rows, V, generator=gen(k), device="cuda") * 2
    u = torch.rand(rows, generator=gen(rows), device="cuda")
    for p in (1.0, 0.9):
        for dt in (F32, BF):
            check(z.to(dt), u, [1.0] * rows, [k] * rows, [p] * rows, [0.0] * rows)
