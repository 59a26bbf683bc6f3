"""Every form of dflash2_kv_evict: the keys in shared memory or not (tables up to 50000 slots, and longer ones), the
moves made by the selecting launch or by one of their own (more than 128 moves per head, or lengths updated in place),
over several heads, both types, narrow and wide rows.  Evictions only move what is there: compared bit for bit."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case, evict64
from tests._util import cuda_or_skip

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIDES = ("k", "v", "weight", "pos")


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


def check_case(c, budget, recent, sink, in_place):
    dev = cuda_or_skip()
    seq = [s + c.T for s in c.seq_pos]
    on = c.on(dev)
    cache, page = on["cache"], c.page
    want = {n: getattr(cache, n).clone() for n in SIDES}
    for (b, h), f in evict64(c, budget, recent, sink, seq).items():
        s, f = torch.arange(budget), torch.as_tensor(f)
        to, of = (c.table[b].long()[s // page], s % page), (c.table[b].long()[f // page], f % page)
        for n in SIDES:
            old = getattr(cache, n)
            want[n][to[0], h, to[1]] = old[of[0].to(dev), h, of[1].to(dev)]
    lens = on["kv_len"]
    n = d2.kv_evict(cache, on["page_table"], lens, budget, recent, sink,
                    seq_len=torch.tensor(seq, dtype=torch.int32, device=dev), out=lens if in_place else None)
    torch.cuda.synchronize()
    assert n.tolist() == [min(x, budget) for x in c.lens]
    for name in SIDES:
        assert torch.equal(bits(getattr(cache, name)), bits(want[name])), name


@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 64), (BF, 256), (F32, 36)])
@pytest.mark.parametrize("budget,recent,sink", [(1, 1, 1), (50, 10, 4), (120, 30, 2)])
def test_lengths_in_place(dtype, d, budget, recent, sink):
    """Few moves in two launches: the lengths are read by the first and written by the second."""
    c = Case(budget + d, [0, 1, 49, 50, 51, 130, 300, 64], 1, 2, 2, d, 16, dtype, held=True)
    check_case(c, budget, recent, sink, True)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64), (F32, 256), (BF, 40)])
@pytest.mark.parametrize("Hkv", [1, 3])
@pytest.mark.parametrize("kind", ["random", "equal", "odd"])
def test_many_moves(dtype, d, Hkv, kind):
    """Several hundred moves per head, ragged requests, some within the budget."""
    c = Case(d + Hkv, [1500, 700, 0, 701, 1033, 1400], 1, Hkv, Hkv, d, 24, dtype, held=True)
    g = torch.Generator().manual_seed(Hkv)
    if kind == "equal":
        c.weight[:] = 0.25
    elif kind == "odd":
        c.weight = torch.randn(c.weight.shape, generator=g) * 1e30
        c.weight[torch.rand(c.weight.shape, generator=g) < 0.3] = float("nan")
        c.weight[torch.rand(c.weight.shape, generator=g) < 0.1] = -float("inf")
    check_case(c, 700, 100, 4, Hkv == 3)


@pytest.mark.parametrize("dtype,d,budget,most", [(BF, 8, 52000, 52096), (F32, 4, 60000, 60112), (BF, 64, 20000, 60000),
                                                 (F32, 256, 12345, 51200)])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_tables(dtype, d, budget, most, in_place):
    """Tables of more than 50000 slots, several heads: up to 128 moves per head, and many."""
    dev = cuda_or_skip()
    B, Hkv, page = 3, 2, 16
    lens = [most, budget, (budget + most) // 2 + 1]
    g = torch.Generator(device=dev).manual_seed(budget)
    pages = B * (most // page)
    k, v = (torch.randn(pages, Hkv, page, d, generator=g, device=dev).to(dtype) for _ in range(2))
    w = (torch.rand(pages, Hkv, page, generator=g, device=dev) * 500).floor()
    pos = torch.randint(0, 2 * most, (pages, Hkv, page), generator=g, device=dev, dtype=torch.int32)
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, -1).contiguous()
    cache = d2.KVCache(k, v, weight=w, pos=pos)
    seq, recent, sink = 2 * most, 3000, 5
    want = [x.clone() for x in (k, v, w, pos)]
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        s = torch.arange(n, device=dev)
        pg, off = table[b].long()[s // page], s % page
        for h in range(Hkv):
            p = pos[pg, h, off]
            x = torch.where((p >= seq - recent) | (p < sink), float("inf"), w[pg, h, off].double())
            kept = torch.zeros(n, dtype=torch.bool, device=dev)
            kept[torch.argsort(x, descending=True, stable=True)[:budget]] = True
            to, of = torch.nonzero(~kept[:budget])[:, 0], budget + torch.nonzero(kept[budget:])[:, 0]
            for y, z in zip(want, (k, v, w, pos)):
                y[pg[to], h, off[to]] = z[pg[of], h, off[of]]
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    got = d2.kv_evict(cache, table, n, budget, recent, sink, out=n if in_place else None,
                      seq_len=torch.full((B,), seq, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert got.tolist() == [budget] * B
    for name, x, y in zip(SIDES, want, (k, v, w, pos)):
        assert torch.equal(bits(x), bits(y)), name
