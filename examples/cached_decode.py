"""Speculative decoding over a paged cache with a budget, on one GPU: a one-layer model with random weights, run as a
serving loop would run it.

Every step drafts a block of K tokens per request (fused LM head, context gate, pair scores and walk), appends the
block's keys and values to the paged cache with their rotary positions, lets the K + 1 queries attend to the cache
causally while the cache collects the attention weights, verifies the block against the target logits, keeps the
accepted tokens' slots (the rejected ones are overwritten by the next block), and cuts a request that has outgrown its
budget down to its newest, first and most attended keys.  The requests' first tokens are sampled from given uniforms; the
target's head may be held in 4 bits.

  python examples/cached_decode.py [--requests 8] [--steps 64] [--budget 256] [--head4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dflash_draft_selection_gb300 as d2  # noqa: E402


class Model:
    """Weights of the layer, of the drafter's heads, and the rotation table."""

    def __init__(self, V=4096, hidden=512, Hq=8, Hkv=2, d=64, K=7, rank=256, max_pos=4096, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *n, s: (torch.randn(*n, generator=g, device=device) * s).bfloat16()  # noqa: E731
        self.V, self.hidden, self.Hq, self.Hkv, self.d, self.K = V, hidden, Hq, Hkv, d, K
        self.embed = rand(V, hidden, s=1.0)
        self.qkv = rand(hidden, (Hq + 2 * Hkv) * d, s=hidden ** -0.5)
        self.out = rand(Hq * d, hidden, s=0.2 * (Hq * d) ** -0.5)
        self.head = rand(V, hidden, s=4 * hidden ** -0.5)
        # one offset per drafted position; none for the first, which the drafter therefore often gets right
        self.draft = rand(K, hidden, s=0.5) * (torch.arange(K, device=device) > 0)[:, None]
        self.q_norm, self.k_norm = 1 + rand(d, s=0.1), 1 + rand(d, s=0.1)
        self.A, self.Bt, self.Wg = rand(V, rank, s=1 / 16), rand(V, rank, s=1 / 16), rand(rank, hidden, s=1 / 16)
        angle = torch.arange(max_pos, device=device).double()[:, None] * \
            1e4 ** (-torch.arange(0, d, 2, device=device).double() / d)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.head4 = None

    def hold_head_in_4_bits(self, group: int = 64):
        """The target's logits come from 4-bit weights from here on (the drafter's, whose fused head reads bf16, from the
        weights that they stand for, so both are held)."""
        self.head4 = d2.quant4(self.head, group=group)
        d2.dequant4(self.head4, out=self.head)

    def logits(self, states: torch.Tensor) -> torch.Tensor:
        return states @ self.head.T if self.head4 is None else d2.linear4(states, self.head4)


class Server:
    """B requests with a page table, their cache and what they have decoded so far."""

    def __init__(self, model: Model, B: int, budget: int, page: int = 32, recent: int = 32, sink: int = 4):
        m, dev = model, model.embed.device
        self.m, self.B, self.budget, self.recent, self.sink, self.T = m, B, budget, recent, sink, m.K + 1
        pages = -(-(budget + 4 * self.T) // page)              # room for a few blocks past the budget
        self.cache = d2.KVCache.empty(B * pages, m.Hkv, page, m.d, weights=True, positions=True, device=dev)
        self.table = torch.randperm(B * pages, device=dev).to(torch.int32).view(B, pages).contiguous()
        self.capacity = pages * page
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=dev)  # noqa: E731
        self.slots, self.length = i32(B), i32(B)               # slots in use, tokens in the sequence
        self.last = torch.randint(0, m.V, (B,), device=dev, dtype=torch.int32)
        self.step_ids = torch.arange(self.T, device=dev, dtype=torch.int32)
        self.ws_head = d2.Workspace.for_lmhead(B * m.K, m.V)
        self.ws_attn = d2.Workspace.for_paged_attn(B, self.T, m.Hq, m.Hkv, m.d, torch.bfloat16)
        self.ws_verify = d2.Workspace.for_verify(B, m.K)
        self.ws_evict = d2.Workspace.for_kv_evict(B, m.Hkv, self.capacity, budget)

    def first(self, tokens: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=20, top_p=0.95, min_p=0.0):
        """The token that every request starts from [B], drawn with the uniforms u [B] after the tokens of a prompt's end
        [B].  Returns the tokens' probabilities."""
        params = d2.sampling_params(temperature, top_k, top_p, n=self.B, device=u.device)
        logits = self.m.logits(self.m.embed[tokens.long()])
        self.last, prob = d2.sample(logits, u, params=params, min_p=torch.full_like(u, min_p))
        return prob

    def layer(self, tokens: torch.Tensor) -> torch.Tensor:
        """Hidden states [B, T, hidden] of a block of tokens [B, T] behind the cache; the block is in the cache
        afterwards."""
        m, (B, T) = self.m, tokens.shape
        x = m.embed[tokens.long()]
        qkv = (x.view(B * T, -1) @ m.qkv).view(B, T, m.Hq + 2 * m.Hkv, m.d)
        pos_ids = (self.length[:, None] + self.step_ids)[None].contiguous()
        q, used = d2.rope_append(qkv[:, :, :m.Hq], qkv[:, :, m.Hq:m.Hq + m.Hkv], qkv[:, :, m.Hq + m.Hkv:], m.cos_sin,
                                 pos_ids, self.cache, self.table, self.slots, q_norm=m.q_norm, k_norm=m.k_norm,
                                 seq_pos=self.length)
        o, _ = d2.paged_attn(q, self.cache, self.table, used, seq_pos=self.length, add_weights=True, ws=self.ws_attn)
        return x + (o.view(B * T, -1) @ m.out).view(B, T, -1)

    def step(self):
        """One draft, verify and cut.  Returns (accepted tokens per request, the block's output tokens, the block's
        tokens, its hidden states)."""
        m, B, K = self.m, self.B, self.m.K
        h = m.embed[self.last.long()][:, None] + m.draft       # [B, K, hidden]
        cand, U, _ = d2.lmhead_topk16(h.view(B * K, -1), m.head, ws=self.ws_head)
        gate = d2.ctx_gate(h.view(B * K, -1), m.Wg)
        cand, U = cand.view(B, K, 16), U.view(B, K, 16)
        path, slot, q_sel, _ = d2.pair_score_walk(cand, U, self.last, m.A, m.Bt, gate.view(B, K, -1))
        block = torch.cat([self.last[:, None], path], 1)
        states = self.layer(block)
        logits = m.logits(states.view(B * self.T, -1))
        accepted, out, _ = d2.verify(logits, path, cand, q_sel, slot, ws=self.ws_verify)
        keep = accepted + 1                                    # the block's first token and the accepted ones
        self.slots, self.length = self.slots + keep, self.length + keep
        self.last = out.gather(1, accepted.long()[:, None])[:, 0].contiguous()
        self.slots = d2.kv_evict(self.cache, self.table, self.slots, self.budget, recent=self.recent, sink=self.sink,
                                 seq_len=self.length, ws=self.ws_evict)
        return accepted, out, block, states


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--budget", type=int, default=256)
    ap.add_argument("--head4", action="store_true", help="hold the target's head in 4 bits")
    a = ap.parse_args()
    # positions: a warm-up step and a.steps more take up to K + 1 = 8 tokens each
    model = Model(max_pos=max(4096, 8 * (a.steps + 1)))
    if a.head4:
        model.hold_head_in_4_bits()
    server = Server(model, a.requests, a.budget)
    server.first(server.last, torch.rand(a.requests, device="cuda"))
    total = torch.zeros(a.requests, dtype=torch.int64, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    server.step()
    start.record()
    for _ in range(a.steps):
        total += server.step()[0] + 1
    end.record()
    torch.cuda.synchronize()
    print(f"{a.requests} requests, {a.steps} steps: {float(total.float().mean()) / a.steps:.2f} tokens per step and "
          f"request, {start.elapsed_time(end) / a.steps:.3f} ms per step, sequences of {server.length.tolist()} tokens "
          f"in {server.slots.tolist()} slots")
    assert d2.device_error() == 0


if __name__ == "__main__":
    main()
