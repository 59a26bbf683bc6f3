"""Definitions in 64 bits of the 4-bit weights, their products and the sampling (plain torch, any device)."""
import math

import torch

INF = math.inf


def unpack(w):
    """The codes of a Weight4 as whole numbers [N, K]."""
    b = w.codes.long()
    return torch.stack([b % 16, b // 16], 2).flatten(1)[:, :w.K]


def per_column(side, K, group):
    """[N, groups] -> [N, K]: every column's group entry."""
    return side.double().repeat_interleave(group, 1)[:, :K]


def values(w):
    """What a Weight4 stands for, [N, K]."""
    zero = 8.0 if w.zero is None else per_column(w.zero, w.K, w.group)
    return (unpack(w).double() - zero) * per_column(w.scale, w.K, w.group)


def quantised(W, group, zero, dtype):
    """(codes [N, K], scale, zero) by the definition, in f32 with every step rounded once."""
    N, K = W.shape
    f = torch.nn.functional.pad(W.float(), (0, -K % group)).view(N, -1, group)
    bad = ~torch.isfinite(f).all(2)
    f = torch.where(bad[..., None], 0.0, f)
    lo, hi = f.amin(2).clamp(max=0.0), f.amax(2).clamp(min=0.0)
    n = torch.full_like(hi, 15.0 if zero else 7.0)      # a tensor: a scalar would be multiplied by its reciprocal
    scale = (hi / n - lo / n if zero else torch.maximum(hi, -lo) / n).to(dtype)
    step = torch.where(scale == 0, 1.0, scale.float())
    z = (-lo / step).round().clamp(0, 15) if zero else torch.full_like(step, 8.0)
    code = ((f / step[..., None]).round() + z[..., None]).clamp(0, 15)
    code, z = torch.where(bad[..., None], 8.0, code), torch.where(bad, 8.0, z)
    scale = torch.where(bad, math.nan, scale.float()).to(dtype)
    return code.flatten(1)[:, :K].long(), scale, z.to(dtype) if zero else None


def ranked(z):
    """Values best first and their ids, ties by the lower id."""
    v, i = (z.double() + 0.0).sort(dim=-1, descending=True, stable=True)
    return v, i


def draw(z, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob, margin) of one row [V]: margin is how far u times the mass lies from the next border, and a cut of
    top_p from the next running mass, relative to the mass."""
    if torch.isnan(z).any() or (z == INF).any() or not (z > -INF).any() or math.isnan(u):
        return -1, math.nan, 1.0
    if not (0 <= T < INF) or top_k < 0 or not (0 < top_p <= 1) or not (0 <= min_p <= 1):
        return -1, math.nan, 1.0
    v, ids = ranked(z)
    if T == 0:
        return int(ids[0]), 1.0, 1.0
    w = torch.exp((v - v[0]) / T)
    V = z.shape[0]
    w = w[:top_k] if 0 < top_k < V else w
    margin = 1.0
    if top_p < 1:
        run = w.cumsum(0)
        goal = top_p * run[-1]
        margin = min(margin, float((run[:-1] - goal).abs().min() / run[-1])) if len(w) > 1 else margin
        w = w[:int((run < goal).sum()) + 1]
    n = max(1, int((w >= min_p).sum()))
    w = w[:n]
    run = w.cumsum(0)
    goal = u * run[-1]
    margin = min(margin, float(((run[:-1] - goal).abs() / run[-1]).min())) if n > 1 else margin
    at = min(int((run <= goal).sum()), int((w > 0).sum()) - 1)
    return int(ids[at]), float(w[at] / run[-1]), margin
