"""The cache-attention operators as a user's program calls them, with their plain forms.

Three operators that a speculative decoder runs around the draft selection and the verify of every block:

* ``append``  the new tokens' queries and keys are normalised (RMS per head, optional) and rotated (one or several
  position axes), keys and values go into the pages of their request;
* ``attn``    a block of new tokens attends to its request's paged cache (causally for a verify, both ways inside the
  block for a drafter, within a window for a ring cache), optionally adding the softmax weight that every cached
  key received to the cache's running weights;
* ``evict``   a cache over its budget keeps the newest, the first and the most attended keys of every head
  (requests within their budget stay as they are).

``listed`` and ``draw`` give cases, ``prepare`` makes what a program has in hand before the call, ``run`` is one call.
Widths are those of the repository's workloads: hidden 2560 and 5120 (20 and 40 heads of 128), blocks of 8 and 16
tokens, 16, 32 and 64 requests, a drafter's window of 2048 positions plus 64.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def _append(name, B, T, Hq, Hkv, d, rot, axes, norm, interleaved, page, dtype, ctx, ragged):
    return {"name": name, "op": "append", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "axes": axes,
            "norm": norm, "interleaved": interleaved, "page": page, "dtype": dtype, "ctx": ctx, "ragged": ragged}


def _attn(name, B, T, Hq, Hkv, d, page, dtype, lo, ctx, window, causal, weights, held, ragged):
    return {"name": name, "op": "attn", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype,
            "lo": lo, "ctx": ctx, "window": window, "causal": causal, "weights": weights, "held": held,
            "ragged": ragged}


def _evict(name, B, Hkv, d, page, dtype, budget, extra, recent, sink):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "d": d, "page": page, "dtype": dtype, "budget": budget,
            "extra": extra, "recent": recent, "sink": sink}


def listed():
    return [
        # one request decodes one token: the latency of a call
        _append("append_1token", 1, 1, 20, 4, 128, 128, 1, False, False, 16, "bf16", 777, False),
        # a verify step of 64 requests, blocks of up to 8 tokens, with normalised heads
        _append("append_verify64", 64, 8, 40, 8, 128, 128, 1, True, False, 32, "bf16", 1021, True),
        # two long prompts with images: three position axes, a quarter of wide heads rotated
        _append("append_prompt_axes3", 2, 8192, 24, 4, 256, 64, 3, True, False, 64, "bf16", 0, False),
        # one request, one token, a short context: the latency of a call
        _attn("attn_1token_short", 1, 1, 20, 4, 128, 16, "bf16", 777, 777, 0, True, False, False, False),
        # one request, one token, a very long context: the cache's length is split over the GPU
        _attn("attn_1token_long", 1, 1, 40, 8, 128, 64, "bf16", 131071, 131071, 0, True, False, False, False),
        # 64 drafters' blocks, seen both ways, over a window of 2048 positions
        _attn("attn_draft_window", 64, 8, 20, 4, 128, 64, "bf16", 9, 8192, 2048, False, False, False, False),
        # the verify of 32 requests of very different lengths
        _attn("attn_verify_ragged", 32, 8, 40, 8, 128, 32, "bf16", 1, 16384, 0, True, False, False, True),
        # blocks of 16 tokens with wide heads: 96 query rows share each cached key
        _attn("attn_verify_d256", 16, 16, 24, 4, 256, 128, "bf16", 500, 16384, 0, True, False, False, False),
        # a small float32 model
        _attn("attn_f32", 4, 8, 16, 4, 64, 16, "f32", 100, 4096, 0, True, False, False, False),
        # decoding on a cache under a budget: positions have gaps, attention weights are collected
        _attn("attn_weights", 16, 1, 32, 8, 128, 32, "bf16", 2048, 4160, 0, True, True, True, False),
        # a drafter's cache of 2048 positions, 64 over: the usual small eviction
        _evict("evict_2048_64", 16, 8, 128, 32, "bf16", 2048, 64, 64, 4),
        # prompts cut to a budget of 4096 keys at once
        _evict("evict_half", 32, 8, 128, 64, "bf16", 4096, 4096, 512, 4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        G = rng.randint(1, 8)
        rot = rng.choice([d, d, d // 2, d // 4])
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 2_000_000 // (T * (G + 2) * Hkv))))
        c = _append("", B, T, G * Hkv, Hkv, d, rot, rng.choice([1, 1, 3]), rng.random() < 0.5, rng.random() < 0.3, page,
                    dtype, rng.randint(0, 2000), rng.random() < 0.5)
    elif op == "attn":
        G = rng.randint(1, 8)
        T = rng.choice([1, 1, 2, 4, 8, 8, 16, 16, _log(rng, 1, 48)])
        ctx = _log(rng, T, 65536 if dtype == "bf16" else 8192)
        # at most about 2^31 multiply-adds per head dimension: a drawn case costs no more than the largest listed one
        room = (3_000_000 if dtype == "bf16" else 300_000) * 128 // (ctx * Hkv * d)
        room = min(room, 400_000_000 // (ctx * Hkv * G * T))
        B = _log(rng, 1, max(1, min(64, room)))
        held = rng.random() < 0.3
        window = 0 if rng.random() < 0.7 else _log(rng, 1, 4096)
        c = _attn("", B, T, G * Hkv, Hkv, d, page, dtype, rng.randint(T, ctx), ctx, window, rng.random() < 0.7,
                  rng.random() < 0.4, held, rng.random() < 0.4)
    else:
        budget = _log(rng, 80, 8192)
        extra = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(48, 1_500_000 * 128 // ((budget + extra) * Hkv * d))))
        sink = rng.choice([0, 1, 4])
        c = _evict("", B, Hkv, d, page, dtype, budget, extra, rng.randint(0, budget // 2), sink)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ----
def _spread(B, lo, hi):
    """B whole numbers spread evenly over lo .. hi in a scrambled order, the last one hi."""
    return [hi if b == B - 1 else lo + int((hi - lo) * (((b + 1) * 0.6180339887498949) % 1.0)) for b in range(B)]


def _q_lens(c):
    return _spread(c["B"], 1, c["T"]) if c["ragged"] else [c["T"]] * c["B"]


def _lens(c):
    """Slots in use per request before the call (append, evict) or with the new tokens (attn)."""
    if c["op"] == "append":
        return _spread(c["B"], c["ctx"] // 2, c["ctx"])
    if c["op"] == "evict":
        return _spread(c["B"], max(1, c["budget"] - c["extra"] // 4), c["budget"] + c["extra"])
    return [max(n, q) for n, q in zip(_spread(c["B"], c["lo"], c["ctx"]), _q_lens(c))]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    B, Hkv, d, page, dt = c["B"], c["Hkv"], c["d"], c["page"], _dt(c)
    lens = _lens(c)
    most = max(lens) + (c["T"] if c["op"] == "append" else 0)
    per = -(-most // page)
    s = {"case": c, "kv_len": _i32(lens), "most": most}
    # the pages of a request lie anywhere in the pool
    s["table"] = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
    rand = lambda *n: torch.randn(*n, generator=g, device=DEV, dtype=dt)  # noqa: E731
    s["k"], s["v"] = rand(B * per, Hkv, page, d), rand(B * per, Hkv, page, d)
    if c["op"] == "append":
        n_pos, rot, T = 32768, c["rot"], c["T"]
        s["qkv"] = rand(B, T, (c["Hq"] + 2 * Hkv) * d)
        # rotation tables, made once in 64 bits by whoever loads the model
        freq = 1e6 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        first = torch.randint(0, n_pos - 2 * T - 2048, (1, B, 1), generator=g, device=DEV)
        step = torch.arange(T, device=DEV)
        along = torch.stack([step // 1024, step % 1024 // 32, step % 32]) if c["axes"] == 3 else step[None]
        s["pos_ids"] = (first + along[:, None]).to(torch.int32).contiguous()
        pair = torch.arange(rot // 2, device=DEV)
        s["pair_axis"] = ((pair * 8 >= rot) + 0 + (pair * 16 >= 5 * rot)).to(torch.uint8) if c["axes"] == 3 else None
        s["q_norm"], s["k_norm"] = ((1 + 0.1 * rand(d)), (1 + 0.1 * rand(d))) if c["norm"] else (None, None)
        s["q_len"] = _i32(_q_lens(c))
        s["weight"] = torch.rand(B * per, Hkv, page, generator=g, device=DEV)
        s["pos"] = torch.zeros(B * per, Hkv, page, dtype=torch.int32, device=DEV)
    else:
        slot = torch.arange(per * page, device=DEV)
        if c["op"] == "attn":
            T = c["T"]
            s["q"] = rand(B, T, c["Hq"], d)
            s["k"] *= 1.5
            s["q_len"] = _i32(_q_lens(c))
            # positions with gaps that the evicted keys left, in no order; the new tokens come last
            start = s["kv_len"] - s["q_len"]
            s["seq_pos"] = start + start // 3 if c["held"] else start
            pos = slot + slot // 3 if c["held"] else slot
            where = torch.where(slot < start[:, None], pos, slot + (s["seq_pos"] - start)[:, None])[:, None]
            if c["held"]:
                mix = torch.rand(B, Hkv, per * page, generator=g, device=DEV)
                mix = torch.where(slot < start[:, None, None], mix, 2.0 + slot.float()).argsort(-1)
                where = where.expand(B, Hkv, -1).gather(2, mix)
        else:
            # positions of a cache that was evicted before: gaps, in no order; the last `extra` are newest, in order
            n = s["kv_len"][:, None, None]
            mix = torch.rand(B, Hkv, per * page, generator=g, device=DEV)
            mix = torch.where(slot < c["budget"], mix, 2.0 + slot.float()).argsort(-1)
            where = torch.where(mix < c["budget"], mix + mix // 2, mix + c["budget"] // 2)
            s["seq_len"] = (n[:, 0, 0] + c["budget"] // 2).to(torch.int32)
        where = where.expand(B, Hkv, -1).reshape(B, Hkv, per, page).transpose(1, 2).to(torch.int32)
        # what the call adds to or moves: kept beside it, so that every pass starts from the same state.  A heavy
        # tail, in steps, so that equal weights and zeros occur
        w = torch.rand(B, per, Hkv, page, generator=g, device=DEV)
        w = ((w ** -0.5 - 1.0) * 64).floor() / 64
        side = torch.stack([w.view(torch.int32), where.contiguous()])
        s["side0"] = torch.empty_like(side).view(2, B * per, Hkv, page)
        s["side0"][:, s["table"].view(-1).long()] = side.view(2, B * per, Hkv, page)
        s["side"] = s["side0"].clone()
        s["weight"], s["pos"] = s["side"][0].view(torch.float32), s["side"][1]
    if own:
        import dflash_draft_selection_gb300 as d2
        s["d2"] = d2
        with_pos = c["op"] != "attn" or c["held"]
        s["cache"] = d2.KVCache(s["k"], s["v"], weight=s["weight"], pos=s["pos"] if with_pos else None)
        if c["op"] == "attn":
            s["ws"] = d2.Workspace.for_paged_attn(B, c["T"], c["Hq"], Hkv, d, dt)
        if c["op"] == "evict":
            s["ws"] = d2.Workspace.for_kv_evict(B, Hkv, per * page, c["budget"])
    return s


# -------------------------------------------------------------- the calls ----
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _split(s):
    """The query, key and value heads of the fused projection."""
    c = s["case"]
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    x = s["qkv"].view(B, T, Hq + 2 * Hkv, d)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def _own_append(s):
    q, k, v = _split(s)
    q_rot, kv_len = s["d2"].rope_append(q, k, v, s["cos_sin"], s["pos_ids"], s["cache"], s["table"], s["kv_len"],
                                        pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"],
                                        q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, q_len=s["q_len"])
    return {"q": q_rot, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"], "kv_len": kv_len}


def _own_attn(s):
    c = s["case"]
    if c["weights"]:
        s["side"].copy_(s["side0"])
    out, lse = s["d2"].paged_attn(s["q"], s["cache"], s["table"], s["kv_len"], causal=c["causal"], window=c["window"],
                                  q_len=s["q_len"], seq_pos=s["seq_pos"], add_weights=c["weights"], ws=s["ws"])
    return {"out": out, "lse": lse, **({"weight": s["weight"]} if c["weights"] else {})}


def _own_evict(s):
    c = s["case"]
    s["side"].copy_(s["side0"])
    kv_len = s["d2"].kv_evict(s["cache"], s["table"], s["kv_len"], c["budget"], recent=c["recent"], sink=c["sink"],
                              seq_len=s["seq_len"], ws=s["ws"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"], "kv_len": kv_len}


# ------------------------------------------------------------ plain forms ----
def _rotate(x, cos, sin, interleaved):
    """x [B, T, H, d] float32, cos and sin [B, T, 1, rot / 2]: the first rot of the d entries turned pair by pair."""
    h = cos.shape[-1]
    r = x[..., :2 * h]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :h], r[..., h:])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([r, x[..., 2 * h:]], -1)


def _plain_append(s):
    c = s["case"]
    B, T, page, dt = c["B"], c["T"], c["page"], _dt(c)
    q, k, v = _split(s)
    q, k = q.float(), k.float()
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["q_norm"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["k_norm"].float()
    at = s["cos_sin"][s["pos_ids"].long()]                               # [axes, B, T, rot]
    if c["axes"] > 1:
        axis = s["pair_axis"].long().repeat(2).expand(1, B, T, -1)
        at = at.gather(0, axis)
    cos, sin = at[0, :, :, None].chunk(2, -1)
    q, k = _rotate(q, cos, sin, c["interleaved"]).to(dt), _rotate(k, cos, sin, c["interleaved"]).to(dt)
    step = torch.arange(T, device=DEV)
    new = step < s["q_len"][:, None]                                     # [B, T]: the others are not stored
    slot = s["kv_len"][:, None].long() + step
    pg, off = s["table"].long().gather(1, slot // page), slot % page
    keep = new[..., None, None]
    s["k"][pg, :, off] = torch.where(keep, k, s["k"][pg, :, off])
    s["v"][pg, :, off] = torch.where(keep, v, s["v"][pg, :, off])
    s["weight"][pg, :, off] = torch.where(new[..., None], 0.0, s["weight"][pg, :, off])
    s["pos"][pg, :, off] = torch.where(new[..., None], slot[..., None].to(torch.int32), s["pos"][pg, :, off])
    return {"q": q * keep, "k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"],
            "kv_len": s["kv_len"] + s["q_len"]}


def _paged(x, table, most):
    """[num_pages, Hkv, page, ...] -> [B, Hkv, most, ...] of every request."""
    x = x[table.long()].transpose(1, 2)                                  # [B, Hkv, pages, page, ...]
    return x.flatten(2, 3)[:, :, :most]


def _plain_attn(s):
    c = s["case"]
    if c["weights"]:
        s["side"].copy_(s["side0"])
    B, T, Hq, Hkv, d, L = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], s["most"]
    G = Hq // Hkv
    table = s["table"]
    k, v = _paged(s["k"], table, L).float(), _paged(s["v"], table, L).float()
    q = s["q"].float().view(B, T, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, d)
    slot, step = torch.arange(L, device=DEV), torch.arange(T, device=DEV)
    at = _paged(s["pos"], table, L)[:, :, None] if c["held"] else slot    # [B, Hkv, 1, L] or [L]
    mine = (s["seq_pos"][:, None] + step)[:, None, :, None]               # [B, 1, T, 1]
    see = (slot < s["kv_len"][:, None, None, None]) & (step[:, None] < s["q_len"][:, None, None, None])
    if c["causal"]:
        see = see & (at <= mine)
    if c["window"]:
        see = see & (at > mine - c["window"])
    see = see.expand(B, Hkv, T, L).repeat_interleave(G, 2)
    x = torch.where(see, (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d)), -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    heads = lambda y: y.view(B, Hkv, T, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, -1)  # noqa: E731
    got = {"out": heads(p @ v).to(_dt(c)), "lse": heads(top + torch.log(total))[..., 0]}
    if c["weights"]:
        page, per = c["page"], table.shape[1]
        more = torch.nn.functional.pad(p.sum(2), (0, per * page - L)).view(B, Hkv, per, page).transpose(1, 2)
        s["weight"][table.view(-1).long()] += more.reshape(B * per, Hkv, page)
        got["weight"] = s["weight"]
    return got


def _plain_evict(s):
    c = s["case"]
    s["side"].copy_(s["side0"])
    B, Hkv, page, L, budget = c["B"], c["Hkv"], c["page"], s["most"], c["budget"]
    table = s["table"].long()
    n = s["kv_len"].long()[:, None, None]
    slot = torch.arange(L, device=DEV)
    w, at = _paged(s["weight"], table, L), _paged(s["pos"], table, L)
    safe = (at >= s["seq_len"][:, None, None] - c["recent"]) | (at < c["sink"])
    w = torch.where(slot >= n, -math.inf, torch.where(safe, math.inf, w))
    order = w.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter(2, order[..., :budget], True) & (slot < n)
    holes = (~kept & (slot < n.clamp(max=budget))).sort(dim=-1, descending=True, stable=True)
    moved = (kept & (slot >= budget)).sort(dim=-1, descending=True, stable=True)
    E = min(c["extra"], budget)
    dst = holes.indices[..., :E]
    src = torch.where(holes.values[..., :E], moved.indices[..., :E], dst)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    to, of = (table[b, dst // page], h, dst % page), (table[b, src // page], h, src % page)
    for x in (s["k"], s["v"], s["weight"], s["pos"]):
        x[to] = x[of]
    return {"k": s["k"], "v": s["v"], "weight": s["weight"], "pos": s["pos"],
            "kv_len": s["kv_len"].clamp(max=budget)}


_run_own = {"append": _own_append, "attn": _own_attn, "evict": _own_evict}
_run_plain = {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "append":
        # every head of a new token read and written once; its row of the rotation table; weight and position
        n = sum(_q_lens(c))
        heads = (c["Hq"] + 2 * Hkv) * d
        return {"bytes": n * (2 * heads * e + c["rot"] * 4 + 4 * c["axes"] + 8 * Hkv),
                "flops": n * ((c["Hq"] + Hkv) * (3 * c["rot"] + (4 * d if c["norm"] else 0)))}
    if c["op"] == "evict":
        # weights and positions read; the kept keys past the budget move (weights come in no order)
        lens = _lens(c)
        moves = sum(max(0, n - c["budget"]) * c["budget"] / n for n in lens) * Hkv
        return {"bytes": sum(lens) * Hkv * 8 + moves * (4 * d * e + 16), "flops": sum(lens) * Hkv * 4}
    # the visible keys and values once, the weights of the cache read and written, queries and outputs
    q, lens = _q_lens(c), _lens(c)
    seen = [min(n, c["window"] + t - 1) if c["window"] and not c["held"] else n for n, t in zip(lens, q)]
    rows = sum(q) * c["Hq"]
    side = (8 * c["weights"] + 4 * c["held"]) * sum(lens) * Hkv
    return {"bytes": sum(seen) * Hkv * d * 2 * e + side + B * c["T"] * c["Hq"] * (2 * d * e + 4),
            "flops": sum(n * t for n, t in zip(seen, q)) * c["Hq"] * d * 4 + rows * d}


# ------------------------------------------------------------- in 64 bits ----
def _exact_evict(c, s):
    """Head by head: the slots in the order of (protected, weight, slot), the first `budget` of them kept."""
    table, page, budget = s["table"].long(), c["page"], c["budget"]
    weight, pos = s["side0"][0].view(torch.float32).double(), s["side0"][1]
    K, V, W = s["k"].double(), s["v"].double(), weight.clone()
    for b, n in enumerate(s["kv_len"].tolist()):
        slot = torch.arange(n, device=DEV)
        pg, off = table[b, slot // page], slot % page
        for h in range(c["Hkv"] if n > budget else 0):
            w, at = weight[pg, h, off], pos[pg, h, off]
            w = torch.where((at >= s["seq_len"][b] - c["recent"]) | (at < c["sink"]), math.inf, w)
            first = torch.argsort(-w, stable=True)[:budget]
            out = torch.ones_like(slot, dtype=torch.bool)
            out[first] = False
            to, of = slot[:budget][out[:budget]], slot[budget:][~out[budget:]]
            for x, y in ((K, s["k"]), (V, s["v"]), (W, weight)):
                x[pg[to], h, off[to]] = y[pg[of], h, off[of]].double()
    return {"k": K, "v": V, "weight": W, "pos": None, "kv_len": None}


def exact(case, seed):
    """What `run` returns, from the definitions, one request at a time in 64 bits; None where nothing is computed."""
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    B, T, Hq, Hkv, d, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    lens, news = s["kv_len"].tolist(), s["q_len"].tolist()
    table = s["table"].long()
    if c["op"] == "append":
        K, V = s["k"].double(), s["v"].double()
        out = torch.zeros(B, T, Hq, d, dtype=torch.float64, device=DEV)
        half = c["rot"] // 2
        pair = torch.arange(half, device=DEV)
        lo = 2 * pair if c["interleaved"] else pair
        hi = lo + 1 if c["interleaved"] else lo + half
        axis = s["pair_axis"].long() if c["axes"] > 1 else torch.zeros_like(pair)
        for b in range(B):
            n = news[b]
            x = s["qkv"][b, :n].double().view(n, Hq + 2 * Hkv, d)
            head = [x[:, :Hq], x[:, Hq:Hq + Hkv]]
            for i, w in enumerate((s["q_norm"], s["k_norm"])):
                if w is not None:
                    head[i] = head[i] / torch.sqrt(head[i].pow(2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
                where = s["pos_ids"][axis, b, :n].long().T               # [n, half]
                cs, sn = s["cos_sin"][where, pair].double(), s["cos_sin"][where, half + pair].double()
                y = head[i].clone()
                y[..., lo] = head[i][..., lo] * cs[:, None] - head[i][..., hi] * sn[:, None]
                y[..., hi] = head[i][..., lo] * sn[:, None] + head[i][..., hi] * cs[:, None]
                head[i] = y
            out[b, :n] = head[0]
            slot = torch.arange(lens[b], lens[b] + n, device=DEV)
            pg = table[b, slot // page]
            K[pg, :, slot % page] = head[1]
            V[pg, :, slot % page] = x[:, Hq + Hkv:]
        return {"q": out, "k": K, "v": V, "weight": None, "pos": None, "kv_len": None}
    out = torch.zeros(B, T, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    weight = s["side0"][0].view(torch.float32).double() if c["weights"] else None
    for b in range(B):
        n, t = lens[b], news[b]
        slot = torch.arange(n, device=DEV)
        pg, off = table[b, slot // page], slot % page
        mine = s["seq_pos"][b] + torch.arange(t, device=DEV)
        for h in range(Hkv):
            at = s["pos"][pg, h, off] if c["held"] else slot
            far = mine[:, None] - at[None]                                # [t, n]
            hide = torch.zeros_like(far, dtype=torch.bool)
            if c["causal"]:
                hide |= far < 0
            if c["window"]:
                hide |= far >= c["window"]
            x = torch.einsum("tgd,nd->tgn", s["q"][b, :t, h * G:(h + 1) * G].double(), s["k"][pg, h, off].double())
            x = (x / math.sqrt(d)).masked_fill(hide[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
            out[b, :t, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, s["v"][pg, h, off].double())
            lse[b, :t, h * G:(h + 1) * G] = z
            if c["weights"]:
                weight[pg, h, off] += p.sum((0, 1))
    return {"out": out, "lse": lse, **({"weight": weight} if c["weights"] else {})}
