"""The paged cache path in 64 bits: inputs and plain implementations from the definitions in the header, one request,
head and row at a time (no code of the library's)."""
import math

import numpy as np
import torch

NAN = float("nan")


class Case:
    """A paged cache and a block of queries.  Slots that are not in use, pages of nobody and the table's unused
    entries hold NaN or garbage."""

    def __init__(self, seed, lens, T, Hq, Hkv, d, page, dtype=torch.bfloat16, q_lens=None, held=False, nhd=False,
                 spare=2, sigma=1.0, far=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        per = max(1, max(-(-n // page) for n in lens)) + 1
        self.B, self.T, self.Hq, self.Hkv, self.d, self.page, self.dtype = B, T, Hq, Hkv, d, page, dtype
        self.lens, self.q_lens = list(lens), list(q_lens) if q_lens is not None else [T] * B
        pages = B * per + spare
        ids = rng.permutation(pages)[:B * per].reshape(B, per)
        self.k = torch.full((pages, Hkv, page, d), NAN).to(dtype)
        self.v = torch.full((pages, Hkv, page, d), NAN).to(dtype)
        self.weight = torch.full((pages, Hkv, page), NAN)
        self.pos = torch.full((pages, Hkv, page), -7, dtype=torch.int32)
        self.table = torch.tensor(ids, dtype=torch.int32)
        self.seq_pos = []
        for b, n in enumerate(self.lens):
            old = max(n - self.q_lens[b], 0)
            base = old + (old // 2 + 3 if held else 0) if held else n - self.q_lens[b]
            self.seq_pos.append(base)
            for h in range(Hkv):
                at = np.sort(rng.choice(base, old, replace=False)) if held else np.arange(old)
                if held:
                    rng.shuffle(at)
                at = np.concatenate([at, base + np.arange(n - old)])
                for s in range(n):
                    pg, off = ids[b, s // page], s % page
                    self.pos[pg, h, off] = int(at[s])
            for s0 in range(0, n, page):
                m = min(page, n - s0)
                pg = ids[b, s0 // page]
                self.k[pg, :, :m] = (torch.randn(Hkv, m, d, generator=g) * sigma).to(dtype)
                self.v[pg, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
                self.weight[pg, :, :m] = torch.rand(Hkv, m, generator=g)
            self.table[b, -(-n // page):] = int(rng.choice([-1, 2 ** 31 - 1, pages, pages + 5]))
        self.q = torch.randn(B, T, Hq, d, generator=g).to(dtype)
        self.held, self.nhd = held, nhd

    def slot(self, b, s):
        return int(self.table[b, s // self.page]), s % self.page

    def gather(self, x, b, h):
        n = self.lens[b]
        s = torch.arange(n)
        return x[self.table[b].long()[s // self.page], h, s % self.page]

    def on(self, dev):
        """The library's objects on `dev`."""
        import dflash_draft_selection_gb300 as d2
        if self.nhd:
            k, v = (x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) for x in (self.k, self.v))
        else:
            k, v = self.k.to(dev), self.v.to(dev)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        cache = d2.KVCache(k, v, weight=self.weight.to(dev), pos=self.pos.to(dev) if self.held else None)
        return dict(cache=cache, page_table=self.table.to(dev), kv_len=i32(self.lens), q_len=i32(self.q_lens),
                    seq_pos=i32(self.seq_pos))


def attn64(c, scale, causal, window, blind=()):
    """out, lse, added weights (by request [Hkv, n]), and per element the sum of p |v| and per row the largest
    |scale| sum |q k|, which the error bounds need.  `blind`: slots (b, s) that no row sees."""
    B, T, Hq, Hkv, d = c.B, c.T, c.Hq, c.Hkv, c.d
    G = Hq // Hkv
    out = np.zeros((B, T, Hq, d))
    pv = np.zeros((B, T, Hq, d))
    lse = np.full((B, T, Hq), -math.inf)
    big = np.zeros((B, T, Hq))
    added = [np.zeros((Hkv, n)) for n in c.lens]
    for b in range(B):
        n, nq = c.lens[b], min(max(c.q_lens[b], 0), T)
        if n == 0 or nq == 0:
            continue
        for h in range(Hkv):
            K, V = (c.gather(x, b, h).double().numpy() for x in (c.k, c.v))
            P = c.gather(c.pos, b, h).numpy().astype(np.int64) if c.held else np.arange(n)
            q = c.q[b, :nq, h * G:(h + 1) * G].double().numpy()
            mine = c.seq_pos[b] + np.arange(nq)
            see = np.ones((nq, n), dtype=bool)
            if causal:
                see &= P[None] <= mine[:, None]
            if window:
                see &= P[None] > mine[:, None] - window
            for bb, s in blind:
                if bb == b:
                    see[:, s] = False
            for t in range(nq):
                w = np.flatnonzero(see[t])
                if not w.size:
                    continue
                x = q[t] @ K[w].T * scale                                  # [G, seen]
                m = x.max(1, keepdims=True)
                if np.isneginf(m).any():
                    continue
                e = np.exp(x - m)
                z = e.sum(1, keepdims=True)
                p = e / z
                hs = slice(h * G, (h + 1) * G)
                out[b, t, hs], pv[b, t, hs] = p @ V[w], p @ np.abs(V[w])
                lse[b, t, hs] = (m + np.log(z))[:, 0]
                big[b, t, hs] = (np.abs(q[t]) @ np.abs(K[w]).T * abs(scale)).max(1)
                added[b][h, w] += p.sum(0)
    return out, lse, added, pv, big


def rope64(c, q, k, v, cos_sin, pos_ids, pair_axis, interleaved, q_norm, k_norm, eps, lens, q_lens):
    """Rotated q [B, T, Hq, d] and k, v of the stored tokens as lists of (b, t, slot, k [Hkv, d], v [Hkv, d]).
    A token that cannot be stored has NaN queries."""
    B, T = q.shape[:2]
    rot = cos_sin.shape[1]
    half = rot // 2
    cs, sn = cos_sin[:, :half].double().numpy(), cos_sin[:, half:].double().numpy()
    p = np.arange(half)
    i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
    ax = np.zeros(half, dtype=int) if pair_axis is None else np.minimum(pair_axis.numpy().astype(int), pos_ids.shape[0] - 1)

    def turn(x, w, ids):
        y = x.double().numpy().copy()
        if w is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w.double().numpy()
        ok = (ids >= 0) & (ids < cos_sin.shape[0])
        c1 = np.where(ok, cs[np.where(ok, ids, 0), p], np.nan)
        s1 = np.where(ok, sn[np.where(ok, ids, 0), p], np.nan)
        z = y.copy()
        z[..., i], z[..., j] = y[..., i] * c1 - y[..., j] * s1, y[..., j] * c1 + y[..., i] * s1
        return z

    out = np.zeros((B, T, c.Hq, c.d))
    stored = []
    pages = c.k.shape[0]
    for b in range(B):
        for t in range(min(max(q_lens[b], 0), T)):
            ids = pos_ids[ax, b, t].numpy()
            s = lens[b] + t
            pg = int(c.table[b, s // c.page]) if s // c.page < c.table.shape[1] else -1
            if not 0 <= pg < pages:
                out[b, t] = np.nan
                continue
            out[b, t] = turn(q[b, t], q_norm, ids)
            stored.append((b, t, s, pg, turn(k[b, t], k_norm, ids), v[b, t]))
    return out, stored


def evict64(c, budget, recent, sink, seq_len):
    """For each (b, h) with more than `budget` slots: where each of the first `budget` slots comes from."""
    src = {}
    for b, n in enumerate(c.lens):
        if n <= budget:
            continue
        for h in range(c.Hkv):
            w, P = c.gather(c.weight, b, h).double().numpy(), c.gather(c.pos, b, h).numpy()
            safe = (P >= seq_len[b] - recent) | (P < sink)
            w = np.where(np.isnan(w), -np.inf, w)
            nan = np.isnan(c.gather(c.weight, b, h).numpy()) & ~safe
            order = sorted(range(n), key=lambda s: (not safe[s], nan[s], -w[s] if not safe[s] else 0.0, s))
            kept = np.zeros(n, dtype=bool)
            kept[order[:budget]] = True
            f = np.arange(budget)
            f[np.flatnonzero(~kept[:budget])] = budget + np.flatnonzero(kept[budget:])
            src[b, h] = f
    return src
