"""What the calls of the paged cache path promise beside their formulas: empty blocks and batches, arrays and workspaces
that several calls share."""
import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case
from tests._util import cuda_or_skip
from tests.test_gpu_kvcache import append_inputs, bits

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIDES = ("k", "v", "weight", "pos")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_of_no_tokens(dtype):
    """T = 0: nothing is appended and the lengths are what they were."""
    dev = cuda_or_skip()
    c = Case(1, [40, 0, 7], 1, 4, 2, 64, 16, dtype, held=True)
    on = c.on(dev)
    cache, lens = on["cache"], on["kv_len"]
    before = [getattr(cache, n).clone() for n in SIDES]
    x = torch.empty(3, 0, 8, 64, dtype=dtype, device=dev)
    ids = torch.empty(1, 3, 0, dtype=torch.int32, device=dev)
    out = (torch.empty(3, 0, 4, 64, dtype=dtype, device=dev), torch.full((3,), -99, dtype=torch.int32, device=dev))
    kw = dict(q_len=torch.tensor([5, 0, -1], dtype=torch.int32, device=dev))
    for o in (None, out):
        q, n = d2.rope_append(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], torch.ones(10, 64, device=dev), ids, cache,
                              on["page_table"], lens, out=o, **kw)
        assert q.shape == (3, 0, 4, 64) and n.tolist() == [40, 0, 7] == lens.tolist()
    for x, n in zip(before, SIDES):
        assert torch.equal(bits(x), bits(getattr(cache, n)))
    assert d2.paged_attn(q, cache, on["page_table"], lens)[0].shape == (3, 0, 4, 64)
    assert d2.device_error() == 0


def test_append_of_no_tokens_in_a_graph():
    """The copied lengths are part of a captured graph."""
    dev = cuda_or_skip()
    cache = d2.KVCache.empty(4, 2, 16, 64, device=dev)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    x = torch.empty(2, 0, 8, 64, dtype=BF, device=dev)
    n, table = i32(3, 9), torch.zeros(2, 2, dtype=torch.int32, device=dev)
    args = (x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], torch.ones(10, 64, device=dev),
            torch.empty(1, 2, 0, dtype=torch.int32, device=dev), cache, table, n)
    out = (torch.empty(2, 0, 4, 64, dtype=BF, device=dev), i32(-1, -1))
    d2.rope_append(*args, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d2.rope_append(*args, out=out)
    n += 5
    g.replay()
    torch.cuda.synchronize()
    assert out[1].tolist() == [8, 14]


@pytest.mark.parametrize("pages", [0, 3])
def test_no_requests(pages):
    """B = 0 is an empty batch, with a page table of no rows."""
    dev = cuda_or_skip()
    cache = d2.KVCache.empty(4, 2, 16, 64, weights=True, positions=True, device=dev)
    i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device=dev)  # noqa: E731
    x = torch.empty(0, 3, 8, 64, dtype=BF, device=dev)
    q, n = d2.rope_append(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], torch.ones(10, 64, device=dev), i32(1, 0, 3), cache,
                          i32(0, pages), i32(0))
    out, lse = d2.paged_attn(q, cache, i32(0, pages), n, add_weights=True)
    left = d2.kv_evict(cache, i32(0, pages), n, 8)
    assert q.shape == out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4) and n.shape == left.shape == (0,)
    x = torch.empty(2, 0, 4, 64, dtype=BF, device=dev)          # two requests, no tokens
    assert d2.paged_attn(x, cache, torch.zeros_like(i32(2, 3)), torch.zeros_like(i32(2)), add_weights=True)[0].shape == x.shape
    assert d2.device_error() == 0


@pytest.mark.parametrize("budget", [40, 700])      # the moves in the selecting launch, and in one of their own
def test_eviction_and_attention_in_one_workspace(budget):
    """Calls that follow each other share a workspace: each leaves it as the other needs it."""
    dev = cuda_or_skip()
    lens = [1500, 900, 1203] if budget == 700 else [100, 41, 112]
    c = Case(3, lens, 1, 4, 4, 64, 16, held=True)
    a = Case(4, [3000, 900, 4000], 4, 10, 2, 128, 16)
    seq = torch.tensor([s + 1 for s in c.seq_pos], dtype=torch.int32, device=dev)
    cap = c.table.shape[1] * 16
    L = d2.load_library()
    need = [L.dflash2_kv_evict_workspace_bytes(3, 4, cap, budget), L.dflash2_paged_attn_workspace_bytes(3, 4, 10, 2, 128, 1)]
    one = d2.Workspace(max(need), dev)
    qa, on_a = a.q.to(dev), a.on(dev)
    results = []
    for shared in (False, True):
        on = c.on(dev)
        for _ in range(3):
            on = {**on, **c.on(dev)}
            n = d2.kv_evict(on["cache"], on["page_table"], on["kv_len"], budget, 3, 1, seq_len=seq,
                            ws=one if shared else None)
            got = d2.paged_attn(qa, ws=one if shared else None, **on_a)
        results.append([n, *got] + [bits(getattr(on["cache"], x)) for x in SIDES])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert d2.device_error() == 0


def test_evicted_lengths_over_the_sequences_lengths():
    """kv_len_out may be kv_len or seq_len: every head reads both before either is written."""
    dev = cuda_or_skip()
    lens, budget = [60 + i % 5 for i in range(300)], 40
    c = Case(5, lens, 1, 8, 8, 8, 16, held=True)
    results = []
    for shared in (False, True):
        on = c.on(dev)
        seq = torch.tensor([s + 1 for s in c.seq_pos], dtype=torch.int32, device=dev)
        n = d2.kv_evict(on["cache"], on["page_table"], on["kv_len"], budget, 20, 2, seq_len=seq,
                        out=seq if shared else None)
        torch.cuda.synchronize()
        assert n.tolist() == [budget] * 300
        results.append([bits(getattr(on["cache"], x)) for x in SIDES])
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,rot", [(3, 5, 6, 2, 128, 128), (2, 3, 4, 2, 40, 10), (4, 1000, 20, 4, 128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_turned_in_place(dtype, B, T, Hq, Hkv, d, rot, interleaved):
    """q_out may be a contiguous q: in vectors, entry by entry and in long blocks."""
    dev = cuda_or_skip()
    c = Case(d + T, [T + 10] * B, T, Hq, Hkv, d, 24, dtype, held=True)
    a = append_inputs(c, T, 1, rot, True)
    x = a["qkv"].to(dev)
    k, v = x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    lens = torch.full((B,), 10, dtype=torch.int32, device=dev)
    results = []
    for in_place in (False, True):
        on, q = c.on(dev), x[:, :, :Hq].contiguous()
        out = (q if in_place else torch.empty_like(q), torch.empty_like(lens))
        d2.rope_append(q, k, v, a["cos_sin"].to(dev), a["pos_ids"].to(dev), on["cache"], on["page_table"], lens,
                       interleaved=interleaved, q_norm=a["q_norm"].to(dev), k_norm=a["k_norm"].to(dev), out=out)
        torch.cuda.synchronize()
        results.append([bits(out[0]), out[1]] + [bits(getattr(on["cache"], n)) for n in SIDES])
    assert all(torch.equal(y, z) for y, z in zip(*results))


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_token_of_more_entries_than_31_bits(interleaved):
    """2^24 + 9 query heads of 128: places within a token pass 2^31."""
    dev = cuda_or_skip()
    H, d, step = 2 ** 24 + 9, 128, 2 ** 21
    cache = d2.KVCache.empty(2, 1, 16, d, positions=True, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    q = torch.randn(1, 1, H, d, generator=g, device=dev, dtype=BF)
    k, v = (torch.randn(1, 1, 1, d, generator=g, device=dev, dtype=BF) for _ in range(2))
    angle = torch.arange(20, device=dev).double()[:, None] * 1e4 ** (-torch.arange(0, d, 2, device=dev).double() / d)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    out, n = d2.rope_append(q, k, v, cos_sin, i32(7).view(1, 1, 1), cache, i32(1, 0)[None], i32(3),
                            interleaved=interleaved)
    cs, sn = cos_sin[7].chunk(2)

    def turn(x):
        x = x.float()
        a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
        y, z = a * cs - b * sn, b * cs + a * sn
        return torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)

    for h in range(0, H, step):
        x = q[0, 0, h:h + step]
        pair = x.float().abs().amax(-1, keepdim=True)
        # the result rounded to bf16, and four fp32 roundings on entries no larger than the row's largest
        assert ((out[0, 0, h:h + step].float() - turn(x)).abs() <= 2.0 ** -8 * turn(x).abs() + 2.0 ** -20 * pair).all()
    assert n.tolist() == [4] and cache.pos[1, 0, 3].item() == 3 and torch.equal(cache.v[1, 0, 3], v[0, 0, 0])
    assert ((cache.k[1, 0, 3].float() - turn(k[0, 0, 0])).abs() <= 2.0 ** -7 * k.float().abs().max()).all()


def test_one_buffer_for_calls_of_every_kind():
    """Zero-filled before it goes to another kind of call, a workspace serves them all."""
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(3)
    z = torch.randn(3, 262144, generator=g, device=dev).bfloat16()       # rows split over the GPU
    a = Case(4, [3000, 900, 4000], 4, 10, 2, 128, 16)
    c = Case(3, [1500, 900, 1203], 1, 4, 4, 64, 16, held=True)
    qa, on_a = a.q.to(dev), a.on(dev)
    seq = torch.tensor([s + 1 for s in c.seq_pos], dtype=torch.int32, device=dev)
    one = d2.Workspace(64 << 20, dev)
    want, got = [], []
    for results, ws in ((want, lambda: None), (got, lambda: one)):
        for _ in range(2):
            results += d2.topk16(z, ws=ws())
            one.buf.zero_()
            results += d2.paged_attn(qa, ws=ws(), **on_a)
            on = c.on(dev)
            d2.kv_evict(on["cache"], on["page_table"], on["kv_len"], 700, 3, 1, seq_len=seq, ws=ws())
            results += [bits(getattr(on["cache"], x)) for x in SIDES]
            one.buf.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and d2.device_error() == 0
