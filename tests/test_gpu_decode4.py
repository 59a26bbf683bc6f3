"""A 4-bit head as it is used: quantised when it is loaded, its logits sampled for a first token, ranked for a draft and
verified, on one stream and in one graph."""
import importlib.util
import os

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests import _decode as ref
from tests._util import cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zero", [False, True])
def test_head_sample_verify(zero):
    dev = cuda_or_skip()
    g = torch.Generator(device=dev).manual_seed(3)
    B, K, V, hidden = 6, 3, 4096, 512
    head = (torch.randn(V, hidden, generator=g, device=dev) * 4 * hidden ** -0.5).bfloat16()
    w = d2.quant4(head, group=64, zero=zero)
    close = d2.dequant4(w)
    assert float((close - head).double().norm() / head.double().norm()) < 0.15
    h = torch.randn(B, hidden, generator=g, device=dev).bfloat16()
    u = torch.rand(B, generator=g, device=dev)
    params = d2.sampling_params(1.0, 20, 0.95, n=B)

    logits = d2.linear4(h, w)
    token, prob = d2.sample(logits, u, params=params)
    exact = h.double() @ ref.values(w).T
    assert (logits.double() - exact).norm() <= 2.0 ** -8 * exact.norm()
    for b in range(B):
        t, q, _ = ref.draw(logits[b], float(u[b]), 1.0, 20, float(torch.tensor(0.95)))
        assert int(token[b]) == t and abs(float(prob[b]) - q) <= 2.0 ** -23 * q

    # a block of drafted tokens against the same head: the logits go where the verify reads them
    states = torch.randn(B * (K + 1), hidden, generator=g, device=dev).bfloat16()
    target = d2.linear4(states, w)
    cand, U, _ = d2.topk16(target)
    assert torch.equal(cand[:, 0].long(), target.float().argmax(1))
    blocks = cand.view(B, K + 1, 16)[:, :K].contiguous()
    path = blocks[:, :, 0].contiguous()
    slot = torch.zeros(B, K, dtype=torch.int32, device=dev)
    q_sel = torch.zeros(B, K, 16, device=dev)
    q_sel[:, :, 0] = 1
    accepted, out, status = d2.verify(target, path, blocks, q_sel, slot)
    assert (accepted == K).all() and (status == 0).all()
    assert torch.equal(out, target.float().argmax(1).view(B, K + 1).int())
    # the bonus token of a greedy verify is what greedy sampling of that row gives
    bonus, _ = d2.sample(target.view(B, K + 1, V)[:, K].contiguous(), u)
    assert torch.equal(bonus, out[:, K])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = d2.sample(d2.linear4(h, w), u, params=params)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step[0], token) and torch.equal(step[1], prob)
    assert d2.device_error() == 0


def test_the_serving_loop_on_a_4_bit_head():
    """examples/cached_decode.py: the first tokens are the sampler's, and every block is verified against the 4-bit
    head's logits."""
    dev = cuda_or_skip()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("cached_decode", os.path.join(root, "examples", "cached_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    m = example.Model(seed=2)
    m.hold_head_in_4_bits()
    assert torch.equal(m.head, d2.dequant4(m.head4))
    server = example.Server(m, 5, budget=512)
    start, u = server.last.clone(), torch.rand(5, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    prob = server.first(start, u, min_p=0.01)
    logits = m.logits(m.embed[start.long()])
    for b in range(5):
        t, q, _ = ref.draw(logits[b], float(u[b]), 1.0, 20, float(torch.tensor(0.95)), float(torch.tensor(0.01)))
        assert int(server.last[b]) == t and abs(float(prob[b]) - q) <= 2.0 ** -23 * q
    for _ in range(6):
        accepted, out, block, states = server.step()
        best = m.logits(states.view(-1, m.hidden)).float().argmax(1).view(5, -1)
        for b, n in enumerate(accepted.tolist()):
            assert out[b, :n].tolist() == block[b, 1:n + 1].tolist() == best[b, :n].tolist()
            assert int(out[b, n]) == int(best[b, n])
    assert d2.device_error() == 0
