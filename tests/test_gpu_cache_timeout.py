"""Bounded waits of the paged cache path's kernels that run out, made on the host without a fault: the test hook keeps the
warps that copy the values (for the weights' pass: the keys) from their first copy until a word is set that nothing sets.
The kernels have to return, set the error word and leave the context usable; with the workspace zero-filled again
the next call is as good as any."""
import math

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._cache import Case
from tests._util import cuda_or_skip
from tests.test_gpu_kvcache import append_inputs, bits, check_append
from tests.test_gpu_paged_attn import check
from tests.test_gpu_wait_timeout import LIMIT, held

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G,lens", [(8, 2, [300, 8, 1000]), (8, 8, [260]), (16, 6, [16, 100, 2000, 264]), (1, 5, [777]),
                                      (16, 8, [140] * 200)])
@pytest.mark.parametrize("weights", [False, True])
def test_attention_gives_up_and_recovers(d, T, G, lens, weights):
    """Whole and cut items, tiles that some rows see in part, values that are not finite among them."""
    dev = cuda_or_skip()
    c = Case(d + T, lens, T, 2 * G, 2, d, 16)
    for b, n in enumerate(lens):
        pg, o = c.slot(b, n - 1)
        c.v[pg, :, o] = math.nan
    ws = d2.Workspace.for_paged_attn(len(lens), T, 2 * G, 2, d, BF)
    q = c.q.to(dev)
    on = c.on(dev)
    _, code = held(lambda: d2.paged_attn(q, add_weights=weights, ws=ws, **on))
    assert code == 1   # DFLASH2_DEVERR_WAIT_TIMEOUT
    ws.buf.zero_()
    fresh = Case(d + T, lens, T, 2 * G, 2, d, 16)
    check(fresh, got=d2.paged_attn(q, ws=ws, **fresh.on(dev)))


def test_a_hook_that_is_set_in_time_changes_nothing():
    dev = cuda_or_skip()
    c = Case(2, [500, 20], 8, 8, 2, 128, 16)
    want = d2.paged_attn(c.q.to(dev), **c.on(dev))
    flag = torch.ones(1, dtype=torch.int32, device=dev)
    d2.test_hold(flag, LIMIT)
    try:
        got = d2.paged_attn(c.q.to(dev), add_weights=True, **c.on(dev))
    finally:
        d2.test_hold(None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and d2.device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G,lens", [(1, 4, [100, 3, 128, 77]), (8, 6, [120, 60, 8]), (1, 5, [1500]), (8, 8, [2000, 900])])
def test_attention_that_gave_up_is_nan(d, T, G, lens):
    """Items of one tile, whose sums are complete before the product that never comes, and cut ones."""
    dev = cuda_or_skip()
    c = Case(d + T, lens, T, 2 * G, 2, d, 16)
    on = c.on(dev)
    (out, lse), code = held(lambda: d2.paged_attn(c.q.to(dev), **on))
    assert code == 1 and torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 4), (8, 8), (16, 8)])
def test_weights_that_gave_up_are_nan(d, T, G):
    """The outputs of the first pass stand; every key that some row sees gets NaN, the others keep theirs."""
    dev = cuda_or_skip()
    c = Case(d + T, [T + 200, T, 900], T, 2 * G, 2, d, 16)
    want = d2.paged_attn(c.q.to(dev), **c.on(dev))
    on = c.on(dev)
    w0 = on["cache"].weight.clone()
    got, code = held(lambda: d2.paged_attn(c.q.to(dev), add_weights=True, **on))
    assert code == 1 and all(torch.equal(x, y) for x, y in zip(got, want))
    w1 = on["cache"].weight
    for b in range(3):
        for h in range(2):
            assert torch.isnan(c.gather(w1.cpu(), b, h)).all()
    used = torch.zeros_like(w0, dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for s in range(n):
            pg, o = c.slot(b, s)
            used[pg, :, o] = True
    assert torch.equal(w1[~used].nan_to_num(-1.0), w0[~used].nan_to_num(-1.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_long_appends_that_gave_up_are_nan(dtype, interleaved):
    """No token is turned: NaN queries, keys and values (zeros past q_len), nothing else in the cache."""
    dev = cuda_or_skip()
    mk = lambda: Case(7, [985] * 4, 925, 20, 4, 128, 24, dtype, q_lens=[925, 700, 0, 925], held=True)  # noqa: E731
    c, lens = mk(), [0, 17, 5, 60]
    c.table[3, 14] = c.k.shape[0] + 2                       # a page that is nowhere
    a = append_inputs(c, 128, 1, 128, True)
    on = c.on(dev)
    cache = on["cache"]
    want = {n: getattr(cache, n).clone() for n in ("k", "v", "weight", "pos")}
    x = a["qkv"].to(dev)
    kw = dict(interleaved=interleaved, q_norm=a["q_norm"].to(dev), k_norm=a["k_norm"].to(dev), q_len=on["q_len"])
    (q, n), code = held(lambda: d2.rope_append(x[:, :, :20], x[:, :, 20:24], x[:, :, 24:], a["cos_sin"].to(dev),
                                               a["pos_ids"].to(dev), cache, on["page_table"],
                                               torch.tensor(lens, dtype=torch.int32, device=dev), **kw))
    assert code == 1 and n.tolist() == [925, 717, 5, 985]
    for b, m in enumerate(c.q_lens):
        assert torch.isnan(q[b, :m]).all() and (q[b, m:] == 0).all()
        s = lens[b] + torch.arange(m)
        pg = c.table[b].long()[s // 24]
        at = pg < c.k.shape[0]
        pg, off, s = pg[at].to(dev), (s % 24)[at].to(dev), s[at].to(dev)
        want["k"][pg, :, off] = want["v"][pg, :, off] = math.nan
        want["weight"][pg, :, off] = 0.0
        want["pos"][pg, :, off] = s[:, None].to(torch.int32)
    for name in want:
        assert torch.equal(bits(getattr(cache, name)), bits(want[name])), name
    check_append(mk(), lens, append_inputs(c, 128, 1, 128, True), interleaved)
