"""The scored router and the float8 (block-scaled) operators: their cases, their plain forms in
elementary torch operations, their values in 64 bits and the calls a user makes of them.

Four operators:
  route     logits -> scores, group-limited top-k with a balance bias, weights, and the grouping of
            the (token, slot) pairs by expert
  quantize  activations -> e4m3 values with one fp32 scale per row and 128 columns
  matmul    the product of such activations with e4m3 weights of one fp32 scale per 128 x 128 block
  experts   the experts' SwiGLU FFN on such weights for routed tokens, combined by routing weight
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BLOCK = 128
E4M3_MAX = 448.0


def listed():
    return [
        # one decoded token of a 256-expert model: softmax scores, weights renormalised
        dict(name="route 1 token", op="route", tokens=1, experts=256, top_k=8, score="softmax",
             groups=1, kept=1, group_top=1, bias=False, renorm=True, scale=1.0, skew=0.0),
        # a long prompt through a router with sigmoid scores, a balance bias and expert groups
        dict(name="route 8192 tokens", op="route", tokens=8192, experts=512, top_k=10,
             score="sigmoid", groups=8, kept=4, group_top=2, bias=True, renorm=True, scale=2.5,
             skew=0.5),
        # the hidden state of a three-token verify step
        dict(name="quantize 3 rows", op="quantize", tokens=3, width=2560, dtype="float32"),
        # the hidden state of a long prompt
        dict(name="quantize 8192 rows", op="quantize", tokens=8192, width=2560, dtype="bfloat16"),
        # one token through one expert-sized projection (gate and up stacked)
        dict(name="matmul 1 row", op="matmul", rows=1, cols=1280, inner=2560, dtype="float32"),
        # ragged in every direction
        dict(name="matmul ragged", op="matmul", rows=777, cols=1001, inner=1296, dtype="bfloat16"),
        # a prompt through one always-on expert's gate and up
        dict(name="matmul prompt", op="matmul", rows=4096, cols=1280, inner=2560, dtype="float32"),
        # a large dense projection
        dict(name="matmul large", op="matmul", rows=8192, cols=8192, inner=8192, dtype="bfloat16"),
        # one decoded token: 8 of 256 experts
        dict(name="experts 1 token", op="experts", tokens=1, hidden=2048, ffn=512, experts=256,
             top_k=8, shared=False, skew=0.0, dtype="bfloat16"),
        # the three tokens of a verify step: 10 of 512 experts and the always-on one
        dict(name="experts 3 tokens", op="experts", tokens=3, hidden=2560, ffn=640, experts=512,
             top_k=10, shared=True, skew=1.1, dtype="bfloat16"),
        # a batch of 64 sequences, one token each
        dict(name="experts 64 tokens", op="experts", tokens=64, hidden=2560, ffn=640, experts=512,
             top_k=10, shared=True, skew=0.0, dtype="bfloat16"),
        # a long prompt, some experts an order of magnitude more popular than others
        dict(name="experts 8192 tokens", op="experts", tokens=8192, hidden=2560, ffn=640,
             experts=512, top_k=10, shared=True, skew=0.5, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "matmul", "matmul", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log(rng, 8, 512 // groups)
        kept = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=groups * per,
                    top_k=rng.randint(1, min(kept * per, 12)),
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, kept=kept,
                    group_top=rng.choice([1, 2]), bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    skew=rng.choice([0.0, 0.5, 1.1]))
    if op == "quantize":
        return dict(op=op, tokens=_log(rng, 1, 8192), width=_log(rng, 16, 2560),
                    dtype=rng.choice(list(DTYPES)))
    if op == "matmul":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 8192),
                    inner=16 * _log(rng, 2, 512), dtype=rng.choice(list(DTYPES)))
    experts = _log(rng, 8, 512)
    return dict(op=op, tokens=_log(rng, 1, 8192), hidden=16 * _log(rng, 16, 160),
                ffn=16 * _log(rng, 4, 40), experts=experts, top_k=rng.randint(1, min(10, experts)),
                shared=rng.random() < 0.5, skew=rng.choice([0.0, 0.5]),
                dtype=rng.choice(["bfloat16", "float16"]))


def _blocks(n):
    return -(-n // BLOCK)


def _popularity(case):
    """The share of each expert rank: r^-skew, normalised."""
    p = np.arange(1, case["experts"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _distinct(case):
    """Expected number of experts that at least one of the tokens is routed to: a token's
    exponential race takes an expert of share p with probability 1 - exp(-c p), sum = top_k."""
    p, k = _popularity(case), case["top_k"]
    if k >= case["experts"]:
        return float(case["experts"])
    lo, hi = 0.0, 1e9
    for _ in range(100):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if (1 - np.exp(-mid * p)).sum() < k else (lo, mid)
    return float((1 - np.exp(-lo * p * case["tokens"])).sum())


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": 4 * (t * e + e * case["bias"] + 4 * t * k + 2 * e + 1), "flops": 4 * t * e}
    if case["op"] == "quantize":
        t, w = case["tokens"], case["width"]
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": t * w * (size + 1) + 4 * t * _blocks(w), "flops": 3 * t * w}
    if case["op"] == "matmul":
        m, n, k = case["rows"], case["cols"], case["inner"]
        size = DTYPES[case["dtype"]].itemsize
        scales = 4 * _blocks(k) * (m + _blocks(n))
        return {"bytes": m * k + n * k + scales + m * n * size, "flops": 2 * m * n * k}
    t, h, f, k = case["tokens"], case["hidden"], case["ffn"], case["top_k"]
    shared = int(case["shared"])
    size = DTYPES[case["dtype"]].itemsize
    weights = (_distinct(case) + shared) * 3 * (f * h + 4 * _blocks(f) * _blocks(h))
    return {"bytes": weights + 2 * t * h * size + t * k * 16 + 4 * t * shared,
            "flops": 6 * t * (k + shared) * f * h}


# ------------------------------------------------------------------ inputs


def _logits(case, gen):
    """Router logits: N(0, 2), or r^-skew popularity over shuffled experts with Gumbel noise, so
    that the top k are k picks without replacement."""
    t, e = case["tokens"], case["experts"]
    if not case["skew"]:
        return 2.0 * torch.randn(t, e, generator=gen, device="cuda")
    logp = torch.log(torch.from_numpy(_popularity(case))).to("cuda", torch.float32)
    logp = logp[torch.randperm(e, generator=gen, device="cuda")]
    u = torch.rand(t, e, generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    return logp - torch.log(-torch.log(u))


def _activations(t, width, dtype, gen):
    """N(0, 1) with one channel in a hundred twenty times larger, the same for every token."""
    x = torch.randn(t, width, generator=gen, device="cuda")
    out = torch.rand(width, generator=gen, device="cuda") < 0.01
    return torch.where(out, 20.0 * x, x).to(dtype)


def _values(shape, gen):
    """e4m3 values as a quantised matrix holds them: normal, the largest near 448."""
    v = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in v.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(130.0)
                   .clamp_(-E4M3_MAX, E4M3_MAX))
    return v


def _scales(shape, mean, gen):
    return mean * torch.exp(0.5 * torch.randn(shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = {"case": case}
    if case["op"] == "route":
        st["logits"] = _logits(case, gen)
        e = case["experts"]
        st["bias"] = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
    elif case["op"] == "quantize":
        st["x"] = _activations(case["tokens"], case["width"], DTYPES[case["dtype"]], gen)
    elif case["op"] == "matmul":
        m, n, k = case["rows"], case["cols"], case["inner"]
        st["a"] = _values((m, k), gen)
        st["a_scale"] = _scales((_blocks(k), m), 1e-2, gen)
        st["b"] = _values((n, k), gen)
        st["b_scale"] = _scales((_blocks(n), _blocks(k)), 1e-4, gen)
    else:
        t, h, f, k = case["tokens"], case["hidden"], case["ffn"], case["top_k"]
        e = case["experts"]
        n = e + int(case["shared"])
        st["x"] = _activations(t, h, DTYPES[case["dtype"]], gen)
        for name, rows, cols in (("gate", f, h), ("up", f, h), ("down", h, f)):
            st[name] = _values((n, rows, cols), gen)
            st[name + "_scale"] = _scales((n, _blocks(rows), _blocks(cols)),
                                          1.0 / (130.0 * math.sqrt(cols)), gen)
        top, ids = torch.topk(_logits(case, gen), k)
        st["w"] = torch.softmax(top, 1)
        st["ids"] = ids.to(torch.int32)
        st["gate_shared"] = torch.rand(t, generator=gen, device="cuda") if case["shared"] else None
        # the grouping, as the router leaves it
        flat = ids.reshape(-1)
        perm = torch.argsort(flat, stable=True)
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(t * k, device="cuda")
        counts = torch.bincount(flat, minlength=e)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["perm"], st["inv_perm"] = perm.to(torch.int32), inv.to(torch.int32)
        st["most"] = int(counts.max())       # tokens of the most popular expert (the plain form's)
    return st


# ------------------------------------------------------------------ plain forms


def _round_e4m3(v):
    """float64 values of magnitude <= 448 to the nearest e4m3 value, ties to even."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(ex - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _quantize(x):
    """x [..., n] -> (the e4m3 values [..., n] as float64, fp32 scales [..., ceil(n / 128)])."""
    n = x.shape[-1]
    pad = torch.nn.functional.pad(x.double(), (0, _blocks(n) * BLOCK - n))
    v = pad.unflatten(-1, (-1, BLOCK))
    s = (v.abs().amax(-1) / E4M3_MAX).float()
    d = torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1)
    q = torch.where(s.unsqueeze(-1) > 0, v / d, torch.zeros_like(v))
    return _round_e4m3(q.clamp(-E4M3_MAX, E4M3_MAX)).flatten(-2)[..., :n], s


def _wide(w, scale):
    """e4m3 weights [..., N, K] with scales per 128 x 128 block, as fp32."""
    n, k = w.shape[-2:]
    s = scale.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return w.float() * s


def _plain_route(st):
    c = st["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    l = st["logits"].double()
    if c["score"] == "softmax":
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    v = s if st["bias"] is None else s + st["bias"].double()
    order = l if st["bias"] is None else v       # both scores rise with the logit
    if c["groups"] > 1:
        per = e // c["groups"]
        best = torch.sort(v.view(t, c["groups"], per), dim=2, descending=True)[0]
        score = best[:, :, :c["group_top"]].sum(2)
        rank = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, rank, True)
        order = torch.where(keep.repeat_interleave(per, 1), order, order.new_full((), -math.inf))
    ids = torch.sort(order, dim=1, descending=True, stable=True)[1][:, :k]
    w = s.gather(1, ids)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    flat = ids.reshape(-1)
    perm = torch.sort(flat, stable=True)[1]
    inv = torch.empty_like(perm).scatter_(0, perm, torch.arange(t * k, device=l.device))
    counts = torch.zeros(e, dtype=torch.int64, device=l.device)
    counts = counts.scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"ids": ids.int(), "w": (w * c["scale"]).float(), "counts": counts.int(),
            "offsets": offsets.int(), "perm": perm.int(), "inv_perm": inv.int()}


def _plain_quantize(st):
    q, s = _quantize(st["x"])
    return {"q": q.float().to(torch.float8_e4m3fn), "s": s.t().contiguous()}


def _plain_matmul(st):
    c = st["case"]
    m, k = c["rows"], c["inner"]
    a = st["a"].float() * st["a_scale"].t().repeat_interleave(BLOCK, 1)[:, :k]
    return {"out": (a @ _wide(st["b"], st["b_scale"]).t()).to(DTYPES[c["dtype"]])}


def _ffn(x, st, pick):
    """x [n, c, H] (x^ in fp32) through the experts `pick` ([n], or a slice): y [n, c, H]."""
    wide = lambda name: _wide(st[name][pick], st[name + "_scale"][pick])  # noqa: E731
    g = torch.bmm(x, wide("gate").transpose(1, 2))
    u = torch.bmm(x, wide("up").transpose(1, 2))
    q, s = _quantize(g / (1.0 + torch.exp(-g)) * u)
    h = q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]
    return torch.bmm(h, wide("down").transpose(1, 2))


def _plain_experts(st):
    c = st["case"]
    t, e, k, h = c["tokens"], c["experts"], c["top_k"], c["hidden"]
    q, s = _quantize(st["x"])
    x = q.float() * s.repeat_interleave(BLOCK, -1)[..., :h]
    if t * k <= e:               # few pairs: each one's expert on its own
        y = _ffn(x.repeat_interleave(k, 0).unsqueeze(1), st, st["ids"].reshape(-1).long())
        y = y.view(t, k, h)
    else:                        # every expert's tokens, padded to the most popular one's
        slot = st["offsets"][:e, None].long() + torch.arange(st["most"], device=x.device)
        slot = slot.clamp(max=t * k - 1)
        y = _ffn(x[st["perm"].long()[slot] // k], st, slice(0, e))
        inv = st["inv_perm"].long()
        at = st["ids"].reshape(-1).long()
        y = y[at, inv - st["offsets"].long()[at]].view(t, k, h)
    out = (st["w"].unsqueeze(2) * y).sum(1)
    if c["shared"]:
        y = _ffn(x.unsqueeze(0), st, slice(e, e + 1))[0]
        out = out + st["gate_shared"].unsqueeze(1) * y
    return {"out": out.to(st["x"].dtype)}


# ------------------------------------------------------------------ the framework's calls


def _ints(n, like):
    return torch.empty(n, dtype=torch.int32, device=like.device)


def _bytes(n, like):
    return torch.empty(max(n, 1), dtype=torch.uint8, device=like.device)


def _own_route(st):
    from expert_ffn_token_b200 import moe
    c, l = st["case"], st["logits"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    if "plan" not in st:
        out = {"ids": _ints((t, k), l), "w": torch.empty(t, k, device=l.device),
               "counts": _ints(e, l), "offsets": _ints(e + 1, l), "perm": _ints(t * k, l),
               "inv_perm": _ints(t * k, l)}
        rule = moe.RouteRule(
            moe.SCORE_SIGMOID if c["score"] == "sigmoid" else moe.SCORE_SOFTMAX, c["groups"],
            c["kept"], c["group_top"], c["renorm"], c["scale"],
            None if st["bias"] is None else st["bias"].data_ptr())
        st["plan"] = out, rule, _bytes(moe.route_workspace_size(t, e, k), l)
    out, rule, ws = st["plan"]
    moe.route_scored(l.data_ptr(), t, e, k, rule, out["ids"].data_ptr(), out["w"].data_ptr(),
                     out["counts"].data_ptr(), out["offsets"].data_ptr(), out["perm"].data_ptr(),
                     out["inv_perm"].data_ptr(), None, ws.data_ptr(), ws.numel(),
                     torch.cuda.current_stream().cuda_stream)
    return out


def _own_quantize(st):
    from expert_ffn_token_b200 import moe
    x = st["x"]
    t, n = x.shape
    if "plan" not in st:
        st["plan"] = (torch.empty(t, -(-n // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device),
                      torch.empty(_blocks(n), t, device=x.device))
    q, s = st["plan"]
    moe.scaled_quantize(x.data_ptr(), moe.dtype_of(x), t, n, n, q.data_ptr(), q.shape[1],
                        s.data_ptr(), t, None, torch.cuda.current_stream().cuda_stream)
    return {"q": q[:, :n], "s": s}


def _own_matmul(st):
    from expert_ffn_token_b200 import moe
    c, a, b = st["case"], st["a"], st["b"]
    m, n, k = c["rows"], c["cols"], c["inner"]
    if "plan" not in st:
        st["plan"] = (torch.empty(m, n, dtype=DTYPES[c["dtype"]], device=a.device),
                      _bytes(moe.scaled_matmul_workspace_size(m, n, k), a))
    out, ws = st["plan"]
    moe.scaled_matmul(a.data_ptr(), k, st["a_scale"].data_ptr(), m, m, k, b.data_ptr(), k,
                      st["b_scale"].data_ptr(), n, out.data_ptr(), moe.dtype_of(out), n, None,
                      ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    return {"out": out}


def _own_experts(st):
    from expert_ffn_token_b200 import moe
    c, x = st["case"], st["x"]
    if "plan" not in st:
        st["plan"] = (moe.ScaledExperts(st["gate"], st["gate_scale"], st["up"], st["up_scale"],
                                        st["down"], st["down_scale"], c["tokens"], c["top_k"],
                                        shared=c["shared"]), torch.empty_like(x))
    layer, out = st["plan"]
    layer.forward(x, st["ids"], st["w"], st["offsets"], st["perm"], st["inv_perm"],
                  gate=st["gate_shared"], out=out)
    return {"out": out}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "quantize": _own_quantize, "matmul": _own_matmul,
                "experts": _own_experts}[op](state)
    return {"route": _plain_route, "quantize": _plain_quantize, "matmul": _plain_matmul,
            "experts": _plain_experts}[op](state)


# ------------------------------------------------------------------ values in 64 bits


def _e4m3_table():
    """The 127 non-negative finite e4m3 values in order of their codes."""
    codes = np.arange(127)
    ex, man = codes >> 3, codes & 7
    return np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))


def _exact_quantize(x):
    """x [rows, n] float64 -> (values, scales [rows, blocks]): by search among the values; a
    quotient halfway between two goes to the one with the even code."""
    rows, n = x.shape
    table = torch.from_numpy(_e4m3_table()).to(x.device)
    middle = (table[1:] + table[:-1]) / 2
    val = torch.zeros_like(x)
    scale = torch.zeros(rows, _blocks(n), dtype=torch.float64, device=x.device)
    for b in range(_blocks(n)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        s = (part.abs().max(1).values / E4M3_MAX).float().double()
        scale[:, b] = s
        r = part.abs() / torch.where(s > 0, s, torch.full_like(s, math.inf))[:, None]
        low = torch.searchsorted(middle, r.contiguous(), right=False)    # middles below r
        high = torch.searchsorted(middle, r.contiguous(), right=True)    # and those equal to it
        code = torch.where((low != high) & (low % 2 == 1), high, low)
        val[:, b * BLOCK:(b + 1) * BLOCK] = torch.sign(part) * table[code]
    return val, scale


def _exact_weight(w, scale):
    n, k = w.shape
    out = w.double()
    for b in range(_blocks(k)):
        rows = scale[:, b].double().repeat_interleave(BLOCK)[:n]
        out[:, b * BLOCK:(b + 1) * BLOCK] *= rows[:, None]
    return out


def _exact_route(st):
    c = st["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    l = st["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        z = np.exp(l - l.max(1)[:, None])
        s = z / z.sum(1)[:, None]
    else:
        s = 1 / (1 + np.exp(-l))
    bias = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    v = s if bias is None else s + bias
    by = l.copy() if bias is None else v.copy()
    if c["groups"] > 1:
        per = e // c["groups"]
        parts = [v[:, g * per:(g + 1) * per] for g in range(c["groups"])]
        take = min(c["group_top"], per)
        total = np.stack([np.partition(p, per - take, 1)[:, per - take:].sum(1) for p in parts], 1)
        drop = np.argsort(-total, 1, kind="stable")[:, c["kept"]:]
        out = np.zeros((t, c["groups"]), bool)
        np.put_along_axis(out, drop, True, 1)
        by[np.repeat(out, per, 1)] = -np.inf
    ids = np.argsort(-by, 1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    if c["renorm"]:
        w = w / np.maximum(w.sum(1)[:, None], 1e-300)
    flat = ids.ravel()
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(t * k)
    counts = np.bincount(flat, minlength=e)
    return {"ids": ids.astype(np.int32), "w": w * c["scale"], "counts": counts.astype(np.int32),
            "offsets": np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
            "perm": perm.astype(np.int32), "inv_perm": inv.astype(np.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st)
    if case["op"] == "quantize":
        val, scale = _exact_quantize(st["x"].double())
        return {"q": val, "s": scale.t().contiguous()}
    if case["op"] == "matmul":
        a = st["a"].double()
        for b in range(_blocks(case["inner"])):
            a[:, b * BLOCK:(b + 1) * BLOCK] *= st["a_scale"][b].double()[:, None]
        return {"out": a @ _exact_weight(st["b"], st["b_scale"]).t()}
    t, e, k, h = case["tokens"], case["experts"], case["top_k"], case["hidden"]
    val, scale = _exact_quantize(st["x"].double())
    x = val * scale.repeat_interleave(BLOCK, 1)[:, :h]
    out = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    jobs = [(i, None) for i in torch.unique(st["ids"]).tolist()]
    if case["shared"]:
        jobs.append((e, torch.arange(t, device="cuda")))
    for i, rows in jobs:
        if rows is None:
            rows, slot = torch.nonzero(st["ids"] == i, as_tuple=True)
            weight = st["w"][rows, slot].double()
        else:
            weight = st["gate_shared"].double()
        g = x[rows] @ _exact_weight(st["gate"][i], st["gate_scale"][i]).t()
        u = x[rows] @ _exact_weight(st["up"][i], st["up_scale"][i]).t()
        hv, hs = _exact_quantize(g / (1 + torch.exp(-g)) * u)
        hq = hv * hs.repeat_interleave(BLOCK, 1)[:, :hv.shape[1]]
        y = hq @ _exact_weight(st["down"][i], st["down_scale"][i]).t()
        out.index_add_(0, rows, weight[:, None] * y)
    return {"out": out}
