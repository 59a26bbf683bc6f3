"""The last step of a decoded token as a user's program calls it, with its plain forms.

Operators that stand beside the fused LM head and the verify of a speculative decoder, for the tokens that are decoded
without a draft (the first one after a prompt, a request that runs without a drafter) and for a target whose head and
projections are held in 4 bits:

* ``quant``   weights [N, K] become 4-bit codes with a scale (and, if asked, a zero point) for every group of
  neighbours in a row, and are read back as the values that they stand for;
* ``linear``  y = x . W^T with such weights: one row for a decoded token, 8 for a verify block, 512 for the verify of
  64 requests;
* ``sample``  one token per row of logits from given uniforms: temperature, top-k, top-p, min-p, then the inverse of
  the cumulative distribution over the kept tokens, best first; greedy rows among them.  The token and its probability.

``listed`` and ``draw`` give cases, ``prepare`` makes what a program has in hand before the call, ``run`` is one call.
Widths are those of the repository's workloads: hidden 256, 2560 and 5120, vocabularies of 4096, 151936 and 262144
tokens, blocks of 8 tokens, 64 requests, top_k 20 with top_p 0.95.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def _quant(name, N, K, group, zero, dtype):
    return {"name": name, "op": "quant", "N": N, "K": K, "group": group, "zero": zero, "dtype": dtype}


def _linear(name, rows, N, K, group, zero, dtype, out, pad=0):
    return {"name": name, "op": "linear", "rows": rows, "N": N, "K": K, "group": group, "zero": zero, "dtype": dtype,
            "out": out, "pad": pad}


def _sample(name, rows, V, dtype, kind, temperature, top_k, top_p, min_p, masked=0.0, scale=1.0):
    return {"name": name, "op": "sample", "rows": rows, "V": V, "dtype": dtype, "kind": kind,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "masked": masked,
            "scale": scale}


def listed():
    return [
        # a drafter's projection brought to 4 bits when it is loaded
        _quant("quant_proj", 2560, 2560, 128, False, "bf16"),
        # an LM head brought to 4 bits, with zero points
        _quant("quant_head", 151936, 2560, 64, True, "bf16"),
        # one token through a small projection: the latency of a call
        _linear("linear_1row_proj", 1, 2560, 2560, 128, False, "bf16", "bf16"),
        # one token through a large LM head: the weights are read once
        _linear("linear_1row_head", 1, 151936, 5120, 128, False, "bf16", "bf16"),
        # a verify block of one request through a fused projection with zero points
        _linear("linear_8rows_zero", 8, 7168, 5120, 64, True, "bf16", "bf16"),
        # a small float32 model of odd width, small groups
        _linear("linear_f32_odd", 5, 4097, 264, 32, True, "f32", "f32", 4),
        # one token of 64 requests through an LM head, logits in float32
        _linear("linear_64rows_head", 64, 151936, 2560, 128, False, "bf16", "f32"),
        # the verify of 64 requests, 8 tokens each
        _linear("linear_512rows_head", 512, 151936, 5120, 128, False, "bf16", "bf16"),
        # one request's first token: the latency of a call
        _sample("sample_1row", 1, 151936, "bf16", "spike", 1.0, 20, 0.95, 0.0),
        # 64 requests, nucleus without top_k: thousands of tokens are kept
        _sample("sample_64_nucleus", 64, 151936, "bf16", "spike", 1.0, 0, 0.95, 0.0),
        # 64 requests with parameters of their own over float32 logits, some tokens forbidden
        _sample("sample_64_mixed", 64, 151936, "f32", "flat", -1.0, 0, 1.0, 0.0, 0.3, 2.0),
        # a large vocabulary and a large batch, top_k with min_p
        _sample("sample_512_wide", 512, 262144, "bf16", "flat", 0.8, 50, 1.0, 0.02, 0.0, 2.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear", "linear", "sample", "sample", "sample"])
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.4
    if op == "sample":
        V = _log(rng, 100, 262144)
        rows = _log(rng, 1, max(1, min(512, 512 * 151936 // V)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        mixed = rng.random() < 0.3
        c = _sample("", rows, V, dtype, rng.choice(["spike", "flat"]),
                    -1.0 if mixed else rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5]),
                    rng.choice([0, 0, 1, 20, 50, 100, _log(rng, 2, 5000)]), rng.choice([1.0, 0.95, 0.9, 0.5]),
                    rng.choice([0.0, 0.0, 0.02, 0.1]), rng.choice([0.0, 0.0, 0.3, 0.9]), rng.choice([0.5, 1.0, 2.0]))
    elif op == "linear":
        K = _log(rng, 32, 20480)
        K = K if rng.random() < 0.2 else -(-K // 64) * 64
        N = _log(rng, 16, max(16, min(151936, 777_912_320 // K)))
        rows = rng.choice([1, 1, 2, 8, 8, 16, _log(rng, 1, 512), _log(rng, 1, 512)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if dtype == "f32":
            rows = min(rows, 64)
        c = _linear("", rows, N, K, group, zero, dtype, dtype if rng.random() < 0.7 else "f32",
                    rng.choice([0, 0, 8, 24]))
    else:
        K = _log(rng, 64, 20480)
        K = K if rng.random() < 0.2 else -(-K // 64) * 64
        c = _quant("", _log(rng, 16, max(16, min(151936, 388_956_160 // K))), K, group, zero,
                   rng.choice(["bf16", "bf16", "f32"]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs ----
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": c}
    dt = _dt(c["dtype"])
    if own:
        import dflash_draft_selection_gb300 as d2
        s["d2"] = d2
    if c["op"] == "sample":
        rows, V = c["rows"], c["V"]
        step = 16 // (2 if dt is torch.bfloat16 else 4)
        ld = -(-V // step) * step                       # rows start on 16-byte boundaries
        z = torch.empty(rows, ld, device=DEV)
        if c["kind"] == "spike":                        # noise, and one token with 85 % of the mass
            z.exponential_(generator=g).log_().neg_()
            hot = torch.randint(0, V, (rows, 1), generator=g, device=DEV)
            z.scatter_(1, hot, torch.logsumexp(z[:, :V], 1, keepdim=True) + math.log(0.85 / 0.15))
        else:
            z.normal_(generator=g)
        z *= c["scale"]
        if c["masked"]:                                 # tokens that the request may not produce; one is always left
            away = torch.rand(rows, ld, generator=g, device=DEV) < c["masked"]
            away[torch.arange(rows, device=DEV), torch.randint(0, V, (rows,), generator=g, device=DEV)] = False
            z.masked_fill_(away, -math.inf)
        s["logits"] = z.to(dt)[:, :V]
        s["u"] = torch.rand(rows, generator=g, device=DEV)
        if c["temperature"] < 0:                        # every request has its own
            pick = lambda *v: torch.tensor(v)[torch.randint(0, len(v), (rows,), generator=h)]  # noqa: E731
            h = torch.Generator().manual_seed(int(seed))
            par = {"temperature": pick(0.0, 0.6, 1.0, 1.0, 1.3), "top_k": pick(0, 0, 1, 20, 400, 5000),
                   "top_p": pick(1.0, 1.0, 0.95, 0.8, 0.5), "min_p": pick(0.0, 0.0, 0.05, 0.3)}
        else:
            par = {k: torch.full((rows,), c[k]) for k in ("temperature", "top_p", "min_p")}
            par["top_k"] = torch.full((rows,), c["top_k"])
        s["par"] = {k: v.to(DEV) for k, v in par.items()}
        if own:
            s["params"] = d2.sampling_params(par["temperature"].numpy(), par["top_k"].numpy(), par["top_p"].numpy())
            s["min_p"] = s["par"]["min_p"].float()
        return s
    N, K, group = c["N"], c["K"], c["group"]
    if c["op"] == "quant":
        s["w"] = torch.empty(N, K, device=DEV, dtype=dt).normal_(std=K ** -0.5, generator=g)
        return s
    # what a checkpoint holds: two codes to a byte (the even neighbour in the low half), rows padded to 16 bytes
    bytes_, G = -(-K // 32) * 16, -(-K // group)
    s["codes"] = torch.randint(0, 256, (N, bytes_), generator=g, device=DEV, dtype=torch.uint8)
    s["scale"] = ((0.5 + torch.rand(N, G, generator=g, device=DEV)) * (K ** -0.5 / 4)).bfloat16()
    s["zero"] = torch.randint(5, 11, (N, G), generator=g, device=DEV).bfloat16() if c["zero"] else None
    s["x"] = torch.randn(c["rows"], K + c["pad"], generator=g, device=DEV, dtype=dt)[:, :K]
    if own:
        s["w4"] = d2.Weight4(s["codes"], s["scale"], s["zero"], K=K, group=group)
    return s


# -------------------------------------------------------------- the calls ----
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_quant(s):
    c, d2 = s["case"], s["d2"]
    w4 = d2.quant4(s["w"], group=c["group"], zero=c["zero"])
    return {"values": d2.dequant4(w4, dtype=_dt(c["dtype"])), "scale": w4.scale,
            **({"zero": w4.zero} if c["zero"] else {})}


def _own_linear(s):
    return s["d2"].linear4(s["x"], s["w4"], dtype=_dt(s["case"]["out"]))


def _own_sample(s):
    token, prob = s["d2"].sample(s["logits"], s["u"], params=s["params"], min_p=s["min_p"])
    return {"token": token, "prob": prob}


# ------------------------------------------------------------ plain forms ----
def _grouped(x, group, fill):
    """[N, K] -> [N, groups, group], the last group filled up."""
    K = x.shape[1]
    G = -(-K // group)
    return torch.nn.functional.pad(x, (0, G * group - K), value=fill).view(x.shape[0], G, group)


def _plain_quant(s):
    c = s["case"]
    w = _grouped(s["w"].float(), c["group"], 0.0)
    top = w.abs().amax(2)
    steps = torch.full_like(top, 15.0 if c["zero"] else 7.0)    # a tensor: a scalar is multiplied by its reciprocal
    if c["zero"]:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        scale = (hi / steps - lo / steps).bfloat16()
    else:
        scale = (top / steps).bfloat16()
    step = torch.where(scale == 0, 1.0, scale.float())
    zero = torch.round(-lo / step).clamp(0, 15) if c["zero"] else torch.full_like(step, 8.0)
    code = (torch.round(w / step[..., None]) + zero[..., None]).clamp(0, 15)
    value = ((code - zero[..., None]) * scale.float()[..., None]).flatten(1)[:, :c["K"]]
    return {"values": value.to(_dt(c["dtype"])).contiguous(), "scale": scale,
            **({"zero": zero.bfloat16()} if c["zero"] else {})}


def _values(codes, scale, zero, K, group):
    """The weights that codes stand for, float32 [N, K]."""
    code = torch.stack([codes & 15, codes >> 4], 2).flatten(1).float()
    code = _grouped(code, group, 8.0)
    G = scale.shape[1]
    code = code[:, :G] - (8.0 if zero is None else zero.float()[..., None])
    return (code * scale.float()[..., None]).flatten(1)[:, :K]


def _plain_linear(s):
    c = s["case"]
    w = _values(s["codes"], s["scale"], s["zero"], c["K"], c["group"])
    return (s["x"].float() @ w.T).to(_dt(c["out"]))


def _plain_sample(s):
    V, z, par = s["case"]["V"], s["logits"].float(), s["par"]
    cold = (par["temperature"] == 0)[:, None]
    T = torch.where(cold, 1.0, par["temperature"].double()[:, None])
    k = torch.where(cold, 1, par["top_k"][:, None])
    k = torch.where(k == 0, V, k)
    z, order = z.sort(dim=1, descending=True, stable=True)
    # masses in 64 bits: a draw is next to a border of two of 150000 tokens
    w = torch.exp((z.double() - z[:, :1].double()) / T)
    w = torch.where(torch.arange(V, device=DEV) < k, w, 0.0)
    before = w.cumsum(1) - w
    kept = (before < par["top_p"].double()[:, None] * w.sum(1, keepdim=True)) & (w >= par["min_p"].double()[:, None])
    kept[:, 0] = True
    w = torch.where(kept, w, 0.0)
    total = w.sum(1, keepdim=True)
    hit = (w.cumsum(1) > s["u"].double()[:, None] * total) & (w > 0)
    at = torch.where(hit.any(1), hit.to(torch.uint8).argmax(1), (w > 0).sum(1) - 1)[:, None]
    return {"token": order.gather(1, at)[:, 0].to(torch.int32), "prob": (w.gather(1, at) / total)[:, 0].float()}


_run_own = {"quant": _own_quant, "linear": _own_linear, "sample": _own_sample}
_run_plain = {"quant": _plain_quant, "linear": _plain_linear, "sample": _plain_sample}


# ------------------------------------------------------------------- work ----
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "sample":
        # every logit read once; a maximum, an exponential and a sum each
        n = c["rows"] * c["V"]
        return {"bytes": n * e + c["rows"] * 28, "flops": n * 6}
    side = c["N"] * -(-c["K"] // c["group"]) * (4 if c["zero"] else 2)
    n = c["N"] * c["K"]
    if c["op"] == "quant":
        # weights read; codes written, and read to write their values
        return {"bytes": n * (2 * e + 1) + 2 * side, "flops": n * 5}
    o = 2 if c["out"] == "bf16" else 4
    return {"bytes": n // 2 + side + c["rows"] * (c["K"] * e + c["N"] * o), "flops": 2 * c["rows"] * n}


# ------------------------------------------------------------- in 64 bits ----
def _exact_quant(c, s):
    """Group by group of columns, from the definition."""
    N, K, group = c["N"], c["K"], c["group"]
    values = torch.empty(N, K, dtype=torch.float64, device=DEV)
    scales, zeros = [], []
    for a in range(0, K, group):
        w = s["w"][:, a:a + group].double()
        if c["zero"]:
            low = torch.minimum(w.min(1).values, torch.zeros((), dtype=torch.float64, device=DEV))
            high = torch.maximum(w.max(1).values, torch.zeros((), dtype=torch.float64, device=DEV))
            scale = ((high - low) / 15).to(torch.bfloat16).double()
            zero = (-low / scale).nan_to_num().round().clamp(0, 15)
        else:
            scale = (w.abs().max(1).values / 7).to(torch.bfloat16).double()
            zero = torch.full_like(scale, 8.0)
        code = (w / scale[:, None]).nan_to_num().round().add_(zero[:, None]).clamp_(0, 15)
        values[:, a:a + group] = (code - zero[:, None]) * scale[:, None]
        scales.append(scale)
        zeros.append(zero)
    return {"values": values, "scale": torch.stack(scales, 1), **({"zero": torch.stack(zeros, 1)} if c["zero"] else {})}


def _exact_linear(c, s):
    """A few thousand outputs at a time: the sum of x times code, and of x times zero point, over every group."""
    rows, N, K, group = c["rows"], c["N"], c["K"], c["group"]
    out = torch.empty(rows, N, dtype=torch.float64, device=DEV)
    x = s["x"].double()
    at = torch.arange(K, device=DEV)
    for a in range(0, N, 4096):
        byte = s["codes"][a:a + 4096, at // 2].int()
        w = torch.where(at % 2 == 0, byte % 16, byte // 16).double()
        w -= 8.0 if s["zero"] is None else s["zero"][a:a + 4096, at // group].double()
        w *= s["scale"][a:a + 4096, at // group].double()
        out[:, a:a + 4096] = torch.einsum("rk,nk->rn", x, w)
    return out


def _exact_sample(c, s):
    """Row by row: the probability of the token that the definition draws."""
    par = {k: v.tolist() for k, v in s["par"].items()}
    u = s["u"].double().tolist()
    prob = torch.ones(c["rows"], dtype=torch.float64, device=DEV)
    for r in range(c["rows"]):
        z = s["logits"][r].double()
        if par["temperature"][r] == 0:
            continue
        p = torch.softmax(z / par["temperature"][r], 0).sort(descending=True).values
        if par["top_k"][r]:
            p = p[:par["top_k"][r]] / p[:par["top_k"][r]].sum()
        n = int((p.cumsum(0) < par["top_p"][r] * (1 if par["top_p"][r] < 1 else 2)).sum()) + 1
        floor = float(p[0]) * par["min_p"][r]
        p = p[:n]
        p = p[p >= floor]
        p = p / p.sum()
        i = min(int((p.cumsum(0) <= u[r]).sum()), int((p > 0).sum()) - 1)
        prob[r] = p[i]
    return {"token": None, "prob": prob}


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits; None where nothing is computed."""
    c = dict(case)
    return {"quant": _exact_quant, "linear": _exact_linear, "sample": _exact_sample}[c["op"]](c, prepare(c, seed))
