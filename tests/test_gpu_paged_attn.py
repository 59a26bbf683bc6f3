"""dflash2_paged_attn against the definition in 64 bits.

Bounds.  With u = 2^-24 (fp32) and D = |scale| max_s sum_i |q_i k_si| (d + 4) u, the error of a score x_s; a
probability then is off by at most e = 2 D + 2^-20 relatively (the exponential, itself good to 2^-21, of a rounded
argument; the sum's error is (n + 8) u, added).  out: (e + (n + 8) u) sum p |v|, plus, for bf16 (8 significant bits: a
rounding is off by up to 2^-8 relatively), 2^-8 sum p |v| (p may be rounded once) and 2^-8 |out| (the result is).  lse: D + 2^-20 + (n + 8) u + 2^-22 |lse|.  Weights: the sum over the
rows of p (e + the lse's bound), plus 2^-22 of the total."""
import ctypes
import math

import numpy as np
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case, attn64
from tests._util import cuda_or_skip

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def check(c, causal=True, window=0, scale=None, weights=False, got=None, blind=()):
    dev = cuda_or_skip()
    scale = c.d ** -0.5 if scale is None else scale
    on = c.on(dev)
    w0 = on["cache"].weight.clone()
    out, lse = got or d2.paged_attn(c.q.to(dev), scale=scale, causal=causal, window=window, add_weights=weights, **on)
    torch.cuda.synchronize()
    assert d2.device_error() == 0
    r_out, r_lse, added, pv, big = attn64(c, scale, causal, window, blind)
    n = max(max(c.lens), 1)
    D = big * (c.d + 4) * U
    e = 2 * D + 2.0 ** -20
    s = (n + 8) * U
    lim = (e + s)[..., None] * pv + 1e-30
    if c.dtype == BF:
        lim = lim + 2.0 ** -8 * pv + 2.0 ** -8 * np.abs(r_out)
    g_out, g_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(g_out).all()
    off = np.abs(g_out - r_out) - lim
    assert (off <= 0).all(), f"out: {off.max():.3g} over its bound at {np.unravel_index(off.argmax(), off.shape)}"
    assert np.array_equal(np.isneginf(g_lse), np.isneginf(r_lse))
    seen = ~np.isneginf(r_lse)
    l_lim = D + 2.0 ** -20 + s + 2.0 ** -22 * np.abs(np.where(seen, r_lse, 0))
    assert (np.abs(g_lse[seen] - r_lse[seen]) <= l_lim[seen]).all(), np.abs(g_lse[seen] - r_lse[seen]).max()
    w1 = on["cache"].weight
    if not weights:
        assert torch.equal(w1.nan_to_num(-1.0), w0.nan_to_num(-1.0))
        return out, lse
    rel = float((e + l_lim).max())
    w0, w1 = w0.cpu(), w1.cpu()
    left = torch.ones_like(w0, dtype=torch.bool)
    for b in range(c.B):
        for h in range(c.Hkv):
            before, after = c.gather(w0, b, h).double().numpy(), c.gather(w1, b, h).double().numpy()
            tot = before + added[b][h]
            assert (np.abs(after - tot) <= rel * added[b][h] + 2.0 ** -22 * np.abs(tot)).all()
        for t in range(c.lens[b]):
            pg, o = c.slot(b, t)
            left[pg, :, o] = False
    assert torch.equal(w1[left].nan_to_num(-1.0), w0[left].nan_to_num(-1.0))  # nobody else's weights
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 4), (1, 10, 2), (3, 6, 2), (8, 10, 2), (16, 12, 2), (20, 24, 3)])
def test_heads_and_block_lengths(dtype, d, T, Hq, Hkv):
    """One row to 160 rows per cached head: every row count's path, lengths around the tiles' edges."""
    lens = [T, T + 1, 127 + T, 128, 129, 300]
    check(Case(d + T + Hq, [max(n, T) for n in lens], T, Hq, Hkv, d, 16, dtype), weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 128, 1), (2, 128, 1), (3, 33, 1), (5, 94, 2), (1, 17, 17), (40, 3, 1)])
def test_many_heads_on_one_cached_head(dtype, T, Hq, Hkv):
    """Groups above a block's rows, groups that leave a block's rows unused, long blocks."""
    check(Case(T * Hq, [max(n, T) for n in (1, 90, 290)], T, Hq, Hkv, 128, 16, dtype, held=T == 3), weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 48, 64, 128, 192, 256, 1024])
@pytest.mark.parametrize("nhd", [False, True])
def test_page_sizes_and_layouts(dtype, page, nhd):
    check(Case(page, [1, 63, 64, 257, 500], 1, 6, 2, 64, page, dtype, nhd=nhd), weights=True)
    check(Case(page, [5, 130, 191], 4, 6, 2, 128, page, dtype, nhd=nhd))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 8), (BF, 40), (BF, 80), (BF, 96), (BF, 192), (F32, 4), (F32, 36),
                                     (F32, 100), (F32, 252)])
def test_other_head_dimensions(dtype, d):
    check(Case(d, [1, 40, 200], 3, 6, 2, d, 16, dtype), weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 5, 128, 129, 1000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("held", [False, True])
def test_windows(dtype, window, causal, held):
    check(Case(window, [6, 135, 400], 6, 4, 2, 64, 32, dtype, held=held), causal=causal, window=window, weights=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_requests_and_tokens(dtype):
    """No slots at all, no tokens, fewer tokens than T, a block longer than what is cached, positions before it."""
    c = Case(3, [0, 10, 0, 300, 5, 3], 4, 6, 2, 128, 16, dtype, q_lens=[4, 0, 0, 2, 9, -3])
    check(c, weights=True)
    check(c, causal=False)
    c = Case(4, [3, 200], 4, 6, 2, 64, 16, dtype, q_lens=[4, 4])     # 3 slots, 4 tokens: the first sees nothing
    assert c.seq_pos[0] == -1
    check(c, weights=True)
    c.seq_pos = [-100, 90]                                           # a request that sees nothing; one that sees half
    check(c, weights=True)
    c.seq_pos = [2 ** 31 - 8, -2 ** 31]
    check(c, causal=False, window=7, weights=True)
    check(c, causal=True, window=2 ** 31 - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_touch(dtype, d, bad):
    """Values of later tokens, of positions before the window and of unused slots (NaN in every case here)."""
    T = 8
    c = Case(11, [150, 9, 260], T, 4, 2, d, 16, dtype)
    for b, n in enumerate(c.lens):
        pg, o = c.slot(b, n - 1)
        c.k[pg, :, o] = bad
        c.v[pg, :, o] = bad
    c.q_lens = [T] * 3
    dev = cuda_or_skip()
    on = c.on(dev)
    out, lse = d2.paged_attn(c.q.to(dev), add_weights=True, **on)
    clean = Case(11, [150, 9, 260], T, 4, 2, d, 16, dtype)
    r_out, r_lse, _, pv, _ = attn64(clean, d ** -0.5, True, 0)
    o, z = out.float().cpu().numpy(), lse.cpu().numpy()
    np.testing.assert_allclose(z[:, :T - 1], r_lse[:, :T - 1], atol=1e-4)
    lim = (2.0 ** -7 if dtype == BF else 1e-4) * pv[:, :T - 1]
    assert (np.abs(o[:, :T - 1] - r_out[:, :T - 1]) <= lim).all()
    assert not np.isfinite(o[:, T - 1]).any()   # the last token sees it
    # the same for what lies before a window: here slots 0 .. 39, the window begins later for all but token 0
    c = Case(12, [140], T, 4, 2, d, 16, dtype)
    for s in range(40):
        pg, o = c.slot(0, s)
        c.v[pg, :, o] = bad
    n, W = 140, 140 - T - 39                     # token 0 (position 132) sees positions > 39
    check(c, window=W)
    c.v[c.slot(0, 40)[0], :, c.slot(0, 40)[1]] = bad     # seen by token 0 alone
    on = c.on(dev)
    out, _ = d2.paged_attn(c.q.to(dev), window=W, **on)
    assert not torch.isfinite(out[:, 0]).any() and torch.isfinite(out[:, 1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_scores(dtype):
    """A key of -Inf is a key with probability 0; rows that see nothing else come out empty; +Inf gives NaN."""
    c = Case(5, [200, 1], 1, 2, 1, 64, 16, dtype)
    c.q = c.q.abs() + 0.125
    for b, s in [(0, 7), (0, 150), (1, 0)]:
        pg, o = c.slot(b, s)
        c.k[pg, :, o] = -math.inf
    check(c, weights=True, blind=[(0, 7), (0, 150), (1, 0)])
    pg, o = c.slot(0, 60)
    c.k[pg, :, o] = math.inf
    dev = cuda_or_skip()
    out, lse = d2.paged_attn(c.q.to(dev), **c.on(dev))
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and (out[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sigma", [1e-3, 8.0, 60.0])
def test_range_of_scores(dtype, sigma):
    """From flat to one-hot softmax, maxima that grow along the cache."""
    c = Case(6, [700, 33], 4, 6, 2, 128, 16, dtype, sigma=sigma)
    if sigma > 1:
        for s in range(700):                     # growing towards the end: the running maximum moves often
            pg, o = c.slot(0, s)
            c.k[pg, :, o] = (c.k[pg, :, o].float() * (s / 700)).to(dtype)
    check(c, weights=True)
    check(c, scale=-0.01)
    check(c, scale=0.0, weights=True)


@pytest.mark.gpu
def test_one_long_request_is_split_and_joined():
    """A single cached head of 20000 slots over all CTAs: one row, and the rows of two blocks."""
    check(Case(8, [20011], 1, 1, 1, 64, 64), weights=True)
    check(Case(9, [5003], 1, 3, 1, 128, 16, F32), weights=True)
    check(Case(10, [9001, 40, 3000], 17, 8, 1, 64, 128, held=True))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (8, 10, 2), (8, 24, 4), (16, 24, 4), (16, 16, 2)])
@pytest.mark.parametrize("window", [0, 700])
def test_long_ragged_batches(d, T, Hq, Hkv, window):
    """Batches whose stretches hold many tiles, so that copies, products and the softmax run far apart: against 64 bits
    on the GPU, and the same bits each time.  bf16: 2^-8 sum p |v| + 2^-8 |out| as above, with e = 2^-14 for the rest."""
    dev = cuda_or_skip()
    B, page, G = 12, 64, Hq // Hkv
    g = torch.Generator(device=dev).manual_seed(d + T)
    lens = [T, 127, 9001, 300, 5003, 12288, 64, 2500, 7777, 1111, 4096, 10000]
    per = -(-max(lens) // page)
    k, v = (torch.randn(B * per, Hkv, page, d, generator=g, device=dev).bfloat16() for _ in range(2))
    q = torch.randn(B, T, Hq, d, generator=g, device=dev).bfloat16()
    table = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    cache = d2.KVCache(k, v)
    ws = d2.Workspace.for_paged_attn(B, T, Hq, Hkv, d, BF)
    out, lse = d2.paged_attn(q, cache, table, n, window=window, ws=ws)
    for b in range(B):
        s = torch.arange(lens[b], device=dev)
        K, V = (x[table[b].long()[s // page], :, s % page].double() for x in (k, v))       # [n, Hkv, d]
        x = torch.einsum("thgd,nhd->htgn", q[b].double().view(T, Hkv, G, d), K) * d ** -0.5
        far = (lens[b] - T + torch.arange(T, device=dev))[:, None] - s
        x = x.masked_fill(((far < 0) | (far >= (window or 2 ** 31)))[None, :, None], -math.inf)
        p = x.softmax(-1)
        r, pv = (torch.einsum("htgn,nhd->thgd", p, y).reshape(T, Hq, d) for y in (V, V.abs()))
        off = (out[b].double() - r).abs() - (2.0 ** -8 + 2.0 ** -14) * pv - 2.0 ** -8 * r.abs()
        assert (off <= 0).all(), (b, off.max().item())
        z = torch.logsumexp(x, -1).permute(1, 0, 2).reshape(T, Hq)
        assert ((lse[b].double() - z).abs() <= 2.0 ** -14 * (1 + z.abs())).all()
    for _ in range(6):
        again = d2.paged_attn(q, cache, table, n, window=window, ws=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert d2.device_error() == 0


@pytest.mark.gpu
def test_many_requests():
    """More requests than threads of a CTA: the split over CTAs sums them in several rounds."""
    rng = np.random.default_rng(0)
    lens = [int(n) for n in rng.integers(0, 40, 700)]
    check(Case(13, lens, 1, 2, 1, 64, 16))
    check(Case(14, lens, 1, 2, 1, 64, 16, F32))


@pytest.mark.gpu
def test_bad_page_ids_are_not_seen():
    for dtype in (BF, F32):
        c = Case(15, [200, 100], 2, 4, 2, 64, 16, dtype)
        c.table[0, 3] = -5
        c.table[0, 12] = c.k.shape[0]
        c.table[1, 0] = 2 ** 31 - 1
        blind = [(0, s) for s in [*range(48, 64), *range(192, 200)]] + [(1, s) for s in range(16)]
        keep = c.table.clone()
        c.table[c.table >= c.k.shape[0]] = 0     # for the 64-bit side's indexing; those slots are blind
        c.table[c.table < 0] = 0
        dev = cuda_or_skip()
        on = c.on(dev)
        on["page_table"] = keep.to(dev)
        got = d2.paged_attn(c.q.to(dev), causal=False, **on)
        check(c, causal=False, got=got, blind=blind)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^32 bytes."""
    dev = cuda_or_skip()
    c = Case(16, [300, 77], 3, 8, 2, 128, 32)
    pages = (2 ** 31 // (2 * 32 * 128)) + 64     # more than 2^31 elements
    for layout in range(2):
        shape = (pages, 2, 32, 128) if layout == 0 else (pages, 32, 2, 128)
        k, v = (torch.empty(shape, dtype=BF, device=dev) for _ in range(2))
        if layout:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        m = c.k.shape[0]
        k[-m:], v[-m:] = c.k.to(dev), c.v.to(dev)
        on = c.on(dev)
        on["cache"] = d2.KVCache(k, v)
        on["page_table"] = (c.table + (pages - m)).to(torch.int32).to(dev)
        got = d2.paged_attn(c.q.to(dev), **on)
        check(c, got=got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_each_time_on_any_stream_in_one_workspace(dtype):
    """Calls of different shapes share a workspace; a side stream and a captured graph give the same bits."""
    dev = cuda_or_skip()
    big, small = Case(20, [3000, 900, 4000], 4, 10, 2, 128, 16, dtype), Case(21, [257], 1, 2, 2, 64, 16, dtype)
    ws = d2.Workspace.for_paged_attn(3, 4, 10, 2, 128, dtype)
    runs = []
    on_b, on_s = big.on(dev), small.on(dev)
    qb, qs = big.q.to(dev), small.q.to(dev)
    for _ in range(3):
        runs.append([x.clone() for x in d2.paged_attn(qb, ws=ws, **on_b) + d2.paged_attn(qs, ws=ws, **on_s)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        runs.append([x.clone() for x in d2.paged_attn(qb, ws=ws, **on_b) + d2.paged_attn(qs, ws=ws, **on_s)])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = d2.paged_attn(qb, ws=ws, **on_b) + d2.paged_attn(qs, ws=ws, **on_s)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        runs.append([x.clone() for x in outs])
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))
    check(big, got=tuple(runs[0][:2]))
    check(small, got=tuple(runs[0][2:]))


def test_refusals():
    """Bad arguments are refused before anything is launched (no GPU needed)."""
    from dflash_draft_selection_gb300 import build
    from dflash_draft_selection_gb300.binding import _CacheRecord
    build.build()
    L = d2.load_library()
    p = ctypes.c_void_p(256)          # never dereferenced: the checks fail first
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
    ok = dict(k=256, v=256, weight=256, pos=None, num_pages=4, page_stride=2 * 16 * 64, head_stride=16 * 64,
              slot_stride=64, Hkv=2, page_size=16, d=64, dt=1)

    def call(cache=None, null=(), **kw):
        r = _CacheRecord(**{**ok, **(cache or {})})
        a = dict(cache=ctypes.byref(r), table=p, max_pages=4, kv_len=p, q_len=p, seq_pos=p, q=p, B=2, T=2, Hq=4,
                 scale=0.125, window=0, flags=1, out=ctypes.c_void_p(1024), lse=p, ws=p, ws_bytes=1 << 30, stream=None)
        a.update(kw)
        for n in null:
            a[n] = None
        return L.dflash2_paged_attn(*a.values())

    assert call(B=0) == 0 and call(T=0) == 0
    for n in ("cache", "table", "kv_len", "q", "out", "ws"):
        assert call(null=[n]) == INVALID, n
    for bad in (dict(k=None), dict(v=None), dict(k=264), dict(num_pages=0), dict(Hkv=0), dict(page_size=0), dict(d=0),
                dict(d=60), dict(slot_stride=56), dict(slot_stride=68), dict(head_stride=-8), dict(page_stride=4),
                dict(weight=258), dict(pos=257), dict(dt=7), dict(Hkv=3)):
        assert call(bad) == INVALID, bad
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hq=5), dict(scale=math.nan), dict(scale=math.inf),
               dict(window=-1), dict(flags=4), dict(out=ctypes.c_void_p(512), q=ctypes.c_void_p(512)), dict(max_pages=0), dict(q=ctypes.c_void_p(264)),
               dict(kv_len=ctypes.c_void_p(258))):
        assert call(**kw) == INVALID, kw
    assert call(flags=2, lse=None) == INVALID and call(dict(weight=None), flags=2) == INVALID
    assert call(dict(d=264, slot_stride=264)) == UNSUPPORTED
    assert call(Hq=2 * 129) == UNSUPPORTED
    assert call(max_pages=2 ** 27) == UNSUPPORTED
    assert call(ws_bytes=64) == WORKSPACE
    assert L.dflash2_paged_attn_workspace_bytes(2, 2, 5, 2, 64, 1) == 0
    for bad in (dict(k=torch.zeros(2, 2, 16, 64), v=torch.zeros(2, 2, 16, 64)),):
        with pytest.raises(ValueError):
            d2.KVCache(**bad)          # not on the GPU
