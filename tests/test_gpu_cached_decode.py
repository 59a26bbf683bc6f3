"""The serving loop of examples/cached_decode.py: with room for everything, a block's hidden states are those of full
causal attention over the whole sequence (no cache); with a budget, every head keeps distinct positions, the newest
and the first among them, within the budget."""
import importlib.util
import os

import pytest
import torch

import dflash_draft_selection_gb300 as d2
from tests._util import cuda_or_skip

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("cached_decode", os.path.join(ROOT, "examples", "cached_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def full_states(m, tokens):
    """Hidden states of a sequence [n] by full causal attention in 64 bits."""
    n = tokens.shape[0]
    x = m.embed[tokens].double()
    qkv = (x @ m.qkv.double()).bfloat16().double().view(n, m.Hq + 2 * m.Hkv, m.d)
    cos, sin = m.cos_sin[:n].double().chunk(2, 1)

    def turn(y, w):
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.double()
        a, b = y.chunk(2, -1)
        return torch.cat([a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]], -1)

    G = m.Hq // m.Hkv
    q, k = turn(qkv[:, :m.Hq], m.q_norm), turn(qkv[:, m.Hq:m.Hq + m.Hkv], m.k_norm).repeat_interleave(G, 1)
    v = qkv[:, m.Hq + m.Hkv:].repeat_interleave(G, 1)
    s = torch.einsum("nhd,mhd->hnm", q, k) * m.d ** -0.5
    s = s.masked_fill(torch.ones(n, n, device=s.device).triu(1).bool(), float("-inf"))
    return x + torch.einsum("hnm,mhd->nhd", s.softmax(-1), v).reshape(n, -1) @ m.out.double()


def test_cached_states_equal_full_attention(example):
    cuda_or_skip()
    m = example.Model()
    server = example.Server(m, 3, budget=512)
    seqs = [[] for _ in range(3)]
    for _ in range(12):
        accepted, out, block, states = server.step()
        acc = accepted.tolist()
        for b in range(3):
            want = full_states(m, torch.tensor(seqs[b] + block[b].tolist(), device="cuda"))[len(seqs[b]):]
            got = states[b].double()
            # bf16 roundings of q, k, p, the output, the projection and the sum: 6 of 2^-8 on values of about 1
            assert (got - want).norm() <= 6 * 2.0 ** -8 * want.norm()
            seqs[b] += block[b, :acc[b] + 1].tolist()
            assert out[b, :acc[b]].tolist() == block[b, 1:acc[b] + 1].tolist()
    assert server.length.tolist() == [len(s) for s in seqs] == server.slots.tolist()
    assert max(len(s) for s in seqs) > 12      # drafted tokens were accepted, others rolled back
    assert d2.device_error() == 0


def test_a_budget_is_kept(example):
    cuda_or_skip()
    m = example.Model(seed=1)
    budget, recent, sink = 40, 12, 2
    server = example.Server(m, 4, budget, page=16, recent=recent, sink=sink)
    for _ in range(60):
        server.step()
    assert d2.device_error() == 0
    for b, (n, length) in enumerate(zip(server.slots.tolist(), server.length.tolist())):
        assert length >= 60 and n == min(budget, length)
        s = torch.arange(n, device="cuda")
        for h in range(m.Hkv):
            pos = server.cache.pos[server.table[b].long()[s // 16], h, s % 16].tolist()
            assert len(set(pos)) == n and max(pos) < length
            if length > budget:
                assert set(range(length - recent, length)) <= set(pos) and set(range(sink)) <= set(pos)
        w = server.cache.weight[server.table[b].long()[s // 16], :, s % 16]
        assert torch.isfinite(w).all() and (w >= 0).all()
