"""dflash2_rope_append and dflash2_kv_evict against plain implementations in 64 bits.

Bounds of the append: fp32 arithmetic on a pair (x, y) turned by (cos, sin): 4 u (|x| + |y|), u = 2^-24; with the norm
the factor is off by (d + 8) u relatively.  bf16 results (8 significant bits) are rounded once: 2^-8 of the value,
half an ulp at most, plus the same terms.  Values are copies, and evictions only move what is there: both are compared bit for bit."""
import ctypes

import numpy as np
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case, evict64, rope64
from tests._util import cuda_or_skip

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


def append_inputs(c, seed, axes=1, rot=None, norm=False, n_pos=500, fused=True):
    g = torch.Generator().manual_seed(seed)
    B, T, H = c.B, c.T, c.Hq + 2 * c.Hkv
    rot = rot or c.d
    qkv = (torch.randn(B, T, H, c.d, generator=g) * 2).to(c.dtype)
    ang = torch.arange(n_pos)[:, None].double() * (1e4 ** (-torch.arange(0, rot, 2).double() / rot))
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos_ids = torch.randint(0, n_pos, (axes, B, T), generator=g, dtype=torch.int32)
    pair_axis = torch.randint(0, axes, (rot // 2,), generator=g).to(torch.uint8) if axes > 1 else None
    w = lambda: (1 + 0.2 * torch.randn(c.d, generator=g)).to(c.dtype) if norm else None  # noqa: E731
    return dict(qkv=qkv, cos_sin=cos_sin, pos_ids=pos_ids, pair_axis=pair_axis, q_norm=w(), k_norm=w())


def check_append(c, lens, a, interleaved=False, seq_pos=None, held=True, eps=1e-6, split=True):
    dev = cuda_or_skip()
    on = c.on(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    cache = on["cache"]
    to = lambda x: None if x is None else x.to(dev)  # noqa: E731
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "weight", "pos")}
    Hq, Hkv = c.Hq, c.Hkv
    parts = (a["qkv"][:, :, :Hq], a["qkv"][:, :, Hq:Hq + Hkv], a["qkv"][:, :, Hq + Hkv:])
    if split:                          # slices of one fused projection
        x = to(a["qkv"])
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:
        q, k, v = (p.contiguous().to(dev) for p in parts)
    got_q, got_n = d2.rope_append(q, k, v, to(a["cos_sin"]), to(a["pos_ids"]), cache, on["page_table"], i32(lens),
                                  pair_axis=to(a["pair_axis"]), interleaved=interleaved, q_norm=to(a["q_norm"]),
                                  k_norm=to(a["k_norm"]), eps=eps, q_len=i32(c.q_lens),
                                  seq_pos=None if seq_pos is None else i32(seq_pos))
    torch.cuda.synchronize()
    nq = [min(max(n, 0), c.T) for n in c.q_lens]
    assert got_n.tolist() == [n + m for n, m in zip(lens, nq)]
    r_q, stored = rope64(c, *parts, a["cos_sin"], a["pos_ids"], a["pair_axis"], interleaved, a["q_norm"], a["k_norm"],
                         eps, lens, c.q_lens)

    def near(g, r, x, w):
        x = np.abs(x.double().numpy())
        if w is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.abs(w.double().numpy())
        rot = a["cos_sin"].shape[1]
        s = np.zeros_like(x)
        half = rot // 2
        if interleaved:
            s[..., :rot] = np.repeat(x[..., 0:rot:2] + x[..., 1:rot:2], 2, -1)
        else:
            s[..., :rot] = np.tile(x[..., :half] + x[..., half:rot], 2)
        s[..., rot:] = x[..., rot:]
        lim = (4 + (c.d + 8 if w is not None else 0)) * U * s + 1e-30
        if c.dtype == BF:
            lim = lim + 2.0 ** -8 * (np.abs(r) + lim)
        elif w is None:
            lim[..., rot:] = 0
        g = g.float().cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(g), np.isnan(r))
        f = np.isfinite(r)
        assert (np.abs(g - r)[f] <= lim[f]).all(), (np.abs(g - r) - lim)[f].max()

    near(got_q, r_q, parts[0], a["q_norm"])
    want = {n: x.clone() for n, x in before.items()}
    for b, t, s, pg, k64, v1 in stored:
        off = s % c.page
        near(cache.k[pg, :, off], k64, parts[1][b, t], a["k_norm"])
        want["k"][pg, :, off] = cache.k[pg, :, off]
        want["v"][pg, :, off] = v1.to(dev)
        want["weight"][pg, :, off] = 0
        want["pos"][pg, :, off] = (seq_pos[b] if seq_pos else lens[b]) + t
    for n in want:
        assert torch.equal(bits(getattr(cache, n)), bits(want[n])), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 64), (128, 32), (80, 80), (96, 48), (40, 10), (24, 2),
                                   (512, 512), (1024, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, d, rot, interleaved):
    lens = [0, 17, 47]
    c = Case(d + rot, [64] * 3, 5, 6, 2, d, 16, dtype, q_lens=[5, 3, 0], held=True)
    for axes, norm in ((1, False), (3, True)):
        check_append(c, lens, append_inputs(c, rot, axes, rot, norm), interleaved, seq_pos=[0, 90, 47])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 20, 4), (3, 1, 8, 8), (2, 33, 5, 1), (40, 8, 10, 2)])
@pytest.mark.parametrize("nhd", [False, True])
def test_append_shapes(dtype, B, T, Hq, Hkv, nhd):
    rng = np.random.default_rng(B)
    c = Case(B + T, [100] * B, T, Hq, Hkv, 64, 24, dtype, held=True, nhd=nhd)
    lens = [int(x) for x in rng.integers(0, 100 - T, B)]
    check_append(c, lens, append_inputs(c, 1, 1, 64, True))
    check_append(c, lens, append_inputs(c, 2, 2, 32), split=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,d,rot,nhd", [(20, 4, 128, 128, False), (14, 2, 256, 64, True), (50, 10, 80, 48, False),
                                              (32, 16, 64, 64, False), (50, 25, 256, 256, False), (1, 20, 48, 16, True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_long_blocks(dtype, Hq, Hkv, d, rot, nhd, interleaved):
    """Blocks of many tokens: ragged, one without a token, one that its page table ends in, pages that are nowhere."""
    T, lens = 925, [0, 17, 60, 5]
    c = Case(Hq + d, [985, 985, 985, 400], T, Hq, Hkv, d, 24, dtype, q_lens=[925, 700, 925, 0], held=True, nhd=nhd)
    c.table[0, 3] = -1
    c.table[2, 14] = c.k.shape[0] + 2
    lens[1] = c.table.shape[1] * 24 - 200
    for axes, norm in ((1, False), (3, True)):
        check_append(c, lens, append_inputs(c, rot, axes, rot, norm), interleaved, split=norm)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128), (BF, 40)])
def test_append_bad_positions_and_pages(dtype, d):
    """Position ids outside the table, a full page table, page ids out of range: NaN queries, nothing else written."""
    c = Case(1, [64] * 4, 6, 4, 2, d, 16, dtype, held=True)
    a = append_inputs(c, 5, 3)
    a["pos_ids"][1, 0, 2] = -1
    a["pos_ids"][0, 1, 4] = 500
    c.table[2, 1] = c.k.shape[0] + 3
    a["pair_axis"][0] = 200                    # counts as the last axis
    lens = [3, 20, 12, c.table.shape[1] * 16 - 2]
    for b in range(4):
        c.table[b, -1] = int(c.table[b, 0]) if b == 3 else -1
    check_append(c, lens, a)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 64), (BF, 256), (F32, 36)])
@pytest.mark.parametrize("budget,recent,sink", [(1, 0, 0), (1, 1, 1), (50, 0, 0), (50, 10, 4), (64, 64, 0),
                                                (120, 30, 2), (50, 40, 30), (1000, 5, 5)])
@pytest.mark.parametrize("kind", ["random", "equal", "steps", "odd"])
def test_evict(dtype, d, budget, recent, sink, kind):
    dev = cuda_or_skip()
    lens = [0, 1, 49, 50, 51, 130, 300, 64]
    c = Case(budget + d, lens, 1, 2, 2, d, 16, dtype, held=True)
    g = torch.Generator().manual_seed(budget)
    if kind == "equal":
        c.weight[:] = 0.25
    elif kind == "steps":
        c.weight = torch.randint(0, 4, c.weight.shape, generator=g).float() - 1.0
        c.weight[c.weight == 0] *= -1.0        # -0 and 0 are one value
        c.weight[::2] = c.weight[::2].abs()
    elif kind == "odd":
        c.weight = torch.randn(c.weight.shape, generator=g) * 1e30
        c.weight[torch.rand(c.weight.shape, generator=g) < 0.2] = float("nan")
        c.weight[torch.rand(c.weight.shape, generator=g) < 0.1] = float("inf")
        c.weight[torch.rand(c.weight.shape, generator=g) < 0.1] = -float("inf")
    seq = [s + 1 for s in c.seq_pos]           # T = 1: the newest position is seq_pos
    on = c.on(dev)
    cache = on["cache"]
    want = {n: getattr(cache, n).clone() for n in ("k", "v", "weight", "pos")}
    src = evict64(c, budget, recent, sink, seq)
    for (b, h), f in src.items():
        s = torch.arange(budget)
        to, of = (c.table[b].long()[s // 16], s % 16), (c.table[b].long()[f // 16], torch.as_tensor(f) % 16)
        for n in want:
            old = getattr(cache, n)
            want[n][to[0], h, to[1]] = old[of[0].to(dev), h, of[1].to(dev)]
    n = d2.kv_evict(cache, on["page_table"], on["kv_len"], budget, recent, sink,
                    seq_len=torch.tensor(seq, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert n.tolist() == [min(x, budget) for x in lens]
    for name in want:
        assert torch.equal(bits(getattr(cache, name)), bits(want[name])), name


@pytest.mark.gpu
def test_evict_long_in_place_twice():
    """70000 slots of one head to 30000, lengths updated in place; a second call has nothing to do."""
    dev = cuda_or_skip()
    lens, budget = [70001, 30000, 30001], 30000
    pages = 3 * 547
    g = torch.Generator(device=dev).manual_seed(1)
    k, v = (torch.randn(pages, 1, 128, 64, generator=g, device=dev).to(BF) for _ in range(2))
    w = (torch.rand(pages, 1, 128, generator=g, device=dev) * 1000).floor()
    pos = torch.arange(pages * 128, dtype=torch.int32, device=dev).view(pages, 1, 128).contiguous()
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(3, -1).contiguous()
    cache = d2.KVCache(k, v, weight=w, pos=pos)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    flat = lambda x, b: x[table[b].long()].flatten(0, 2)  # noqa: E731
    old = [[flat(x, b).clone() for x in (k, v, w, pos)] for b in range(3)]
    seq = torch.full((3,), 2 ** 31 - 1, dtype=torch.int32, device=dev)
    out = d2.kv_evict(cache, table, n, budget, recent=10, seq_len=seq, out=n)
    assert out is n and n.tolist() == [30000, 30000, 30000]
    for b in range(3):
        m = lens[b]
        if m <= budget:
            assert all(torch.equal(flat(x, b), y) for x, y in zip((k, v, w, pos), old[b]))
            continue
        order = torch.argsort(old[b][2][:m].double(), descending=True, stable=True)
        kept = torch.zeros(m, dtype=torch.bool, device=dev)
        kept[order[:budget]] = True
        f = torch.arange(budget, device=dev)
        f[~kept[:budget]] = budget + torch.nonzero(kept[budget:])[:, 0]
        for x, y in zip((k, v, w, pos), old[b]):
            assert torch.equal(flat(x, b)[:budget], y[f])
            assert torch.equal(flat(x, b)[budget:], y[budget:])
    again = [x.clone() for x in (k, v, w, pos)]
    d2.kv_evict(cache, table, n, budget, out=n)
    assert all(torch.equal(x, y) for x, y in zip((k, v, w, pos), again)) and n.tolist() == [30000] * 3


@pytest.mark.gpu
def test_evict_bad_page_ids():
    """Slots without a page are the first to go; when they have to stay they are not copied."""
    dev = cuda_or_skip()
    c = Case(2, [96], 1, 2, 1, 64, 16, held=True)
    on = c.on(dev)
    table = c.table.clone()
    table[0, 1], table[0, 4] = -1, c.k.shape[0]
    cache = on["cache"]
    old = [x.clone() for x in (cache.k, cache.v, cache.weight, cache.pos)]
    n = d2.kv_evict(cache, table.to(dev), on["kv_len"], 64, seq_len=torch.tensor([10 ** 6], dtype=torch.int32,
                                                                                device=dev))
    assert n.tolist() == [64] and d2.device_error() == 0
    # 64 slots with a page, 64 kept: all of them; the 16 past the budget have nowhere to go but slots 16 .. 31
    for x, y in zip((cache.k, cache.v, cache.weight, cache.pos), old):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Appends to and evictions in pages at the end of a pool of more than 2^31 elements."""
    dev = cuda_or_skip()
    c = Case(16, [60, 33], 3, 8, 2, 128, 32, held=True)
    m, extra = c.k.shape[0], 2 ** 31 // (2 * 32 * 128) + 64
    pools = [torch.zeros(extra, 2, 32, 128, dtype=BF, device=dev) for _ in range(2)]
    side = [torch.zeros(extra, 2, 32, dtype=t, device=dev) for t in (torch.float32, torch.int32)]
    small = c.on(dev)["cache"]
    for x, y in zip(pools + side, (small.k, small.v, small.weight, small.pos)):
        x[-m:] = y
    far = d2.KVCache(*pools, weight=side[0], pos=side[1])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    a = append_inputs(c, 1)
    x = a["qkv"].to(dev)
    tables = c.table.to(dev), (c.table.to(dev) + (extra - m)).to(torch.int32)
    got = [d2.rope_append(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], a["cos_sin"].to(dev), a["pos_ids"].to(dev), cache,
                          table, i32([57, 30])) for cache, table in zip((small, far), tables)]
    assert torch.equal(got[0][0], got[1][0])
    lens = [d2.kv_evict(cache, table, n, 40, recent=3, sink=1, seq_len=i32([200, 200]))
            for cache, table, (_, n) in zip((small, far), tables, got)]
    assert lens[0].tolist() == lens[1].tolist() == [40, 33]
    for y, z in zip((small.k, small.v, small.weight, small.pos), (far.k, far.v, far.weight, far.pos)):
        assert torch.equal(bits(y), bits(z[-m:]))


def test_refusals():
    """Bad arguments are refused before anything is launched (no GPU needed)."""
    from dflash_draft_selection_gb300 import build
    from dflash_draft_selection_gb300.binding import _CacheRecord
    build.build()
    L = d2.load_library()
    p, odd = ctypes.c_void_p(256), ctypes.c_void_p(258)
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
    ok = dict(k=256, v=256, weight=256, pos=256, num_pages=4, page_stride=2 * 16 * 64, head_stride=16 * 64,
              slot_stride=64, Hkv=2, page_size=16, d=64, dt=1)

    def append(rec=None, **kw):
        r = _CacheRecord(**{**ok, **(rec or {})})
        a = dict(cache=ctypes.byref(r), table=p, max_pages=4, kv_len=p, q_len=p, seq_pos=p, q=p, k=p, v=p, qs=256,
                 ks=128, vs=128, B=2, T=2, Hq=4, cos_sin=p, n_pos=10, rot=64, pos_ids=p, axes=1, pair_axis=None,
                 interleaved=0, q_norm=p, k_norm=p, eps=1e-6, q_out=p, kv_len_out=ctypes.c_void_p(512), stream=None)
        a.update(kw)
        return L.dflash2_rope_append(*a.values())

    assert append(B=0) == 0 and append(T=0) == 0
    for n in ("cache", "table", "kv_len", "q", "k", "v", "cos_sin", "pos_ids", "q_out"):
        assert append(**{n: None}) == INVALID, n
    for bad in (dict(k=None), dict(v=264), dict(d=60), dict(page_size=0), dict(Hkv=0), dict(dt=5), dict(pos=2)):
        assert append(bad) == INVALID, bad
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(rot=0), dict(rot=7), dict(rot=66), dict(axes=0), dict(n_pos=0),
               dict(qs=248), dict(ks=120), dict(vs=129), dict(q=ctypes.c_void_p(264)), dict(kv_len=odd),
               dict(q_norm=ctypes.c_void_p(264)), dict(kv_len_out=odd), dict(max_pages=0)):
        assert append(**kw) == INVALID, kw
    assert append(kv_len_out=p) == INVALID     # the lengths before and after in one array
    assert append(dict(d=1032, slot_stride=1032), qs=8192, ks=4096, vs=4096) == UNSUPPORTED
    assert append(B=2 ** 30, T=2) == UNSUPPORTED

    def evict(rec=None, **kw):
        r = _CacheRecord(**{**ok, **(rec or {})})
        a = dict(cache=ctypes.byref(r), table=p, max_pages=4, kv_len=p, seq_len=p, B=2, budget=8, recent=0, sink=0,
                 out=p, ws=p, ws_bytes=1 << 30, stream=None)
        a.update(kw)
        return L.dflash2_kv_evict(*a.values())

    assert evict(B=0) == 0
    for n in ("cache", "table", "kv_len", "out", "ws"):
        assert evict(**{n: None}) == INVALID, n
    for bad in (dict(weight=None), dict(pos=None), dict(k=None), dict(num_pages=0)):
        assert evict(bad) == INVALID, bad
    for kw in (dict(B=-1), dict(budget=0), dict(recent=-1), dict(sink=-1), dict(kv_len=odd), dict(out=odd)):
        assert evict(**kw) == INVALID, kw
    assert evict(max_pages=2 ** 27) == UNSUPPORTED
    assert evict(ws_bytes=64) == WORKSPACE
    assert L.dflash2_kv_evict_workspace_bytes(2, 2, 64, 0) == 0
    assert L.dflash2_kv_evict_workspace_bytes(2, 2, 64, 8) >= 2 * 2 * 8 * 8
