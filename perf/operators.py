"""The feed-forward operators around the FP8 block GEMM: cases, plain forms and 64-bit values.

Three operators of a transformer's feed-forward block with fine-grained FP8 weights (E4M3 codes,
one scale per 128x128 block; activations E4M3 in 1x128 groups along the input dimension):

epilogue  y = act(A . W^T + bias) + residual, the block-scaled GEMM with its epilogue
route     the router of a mixture of experts: top-k experts of every token and their weights
moe       a whole mixture-of-experts layer for a few tokens, from bf16 rows to bf16 rows:
          y[t] = residual[t] + sum_j weight[t, j] * W2[e] . Q(act(gate) * up),
          (gate, up) = W13[e] . Q(x[t]), e = ids[t, j], Q the 1x128-group E4M3 quantization

`run` computes them in elementary torch operations in 32 bits where `own` is false, and calls the
library where it is true.
"""
import math
import random

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
ZIPF = 1.1  # expert popularity p_e ~ (e + 1)^-1.1, as in the MoE workload of this repository


# ------------------------------------------------------------------------------------- cases
def _epilogue(name, m, n, k, ue8m0, bias, act, residual):
    return dict(name=name, op="epilogue", m=m, n=n, k=k, ue8m0=ue8m0, bias=bias, act=act, residual=residual)


def _route(name, tokens, experts, top_k, scoring, renorm, logits, masked):
    return dict(name=name, op="route", tokens=tokens, experts=experts, top_k=top_k, scoring=scoring, renorm=renorm,
                logits=logits, masked=masked)


def _moe(name, tokens, experts, top_k, hidden, inter, ue8m0, act, residual, absent):
    return dict(name=name, op="moe", tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter,
                ue8m0=ue8m0, act=act, residual=residual, absent=absent)


def listed():
    return [
        # one token through the attention output projection, added to the bf16 residual stream
        _epilogue("epilogue-1x4096x4096", 1, 4096, 4096, False, "none", "none", True),
        # the QKV projection with biases for the next token of 23 sequences
        _epilogue("epilogue-23x6144x4096", 23, 6144, 4096, True, "f32", "none", False),
        # a short prompt (ragged length) through a down projection, added to the residual stream
        _epilogue("epilogue-333x4096x14336", 333, 4096, 14336, False, "none", "none", True),
        # a chunk of a prompt: bias, activation and residual together (short rows, narrow layer)
        _epilogue("epilogue-1000x7168x2048", 1000, 7168, 2048, False, "bf16", "gelu_tanh", True),
        # a full prefill batch through an up projection with bias and activation: the largest product
        _epilogue("epilogue-4096x28672x4096", 4096, 28672, 4096, True, "bf16", "silu", False),
        # the router of one token: a call whose latency is everything
        _route("route-1x32", 1, 32, 8, "softmax", True, "f32", False),
        # 64 decoding sequences, many experts, sigmoid scores
        _route("route-64x256", 64, 256, 8, "sigmoid", True, "f32", False),
        # a prefill batch, bf16 logits (ties are common), some experts masked out
        _route("route-8191x256", 8191, 256, 8, "softmax", False, "bf16", True),
        # one token through the experts: reads top_k experts' weights and little else
        _moe("moe-1", 1, 32, 8, 7168, 2048, True, "silu", False, False),
        # a few sequences: most experts have one or two rows
        _moe("moe-7", 7, 32, 8, 7168, 2048, False, "silu", True, False),
        # a full decode batch: every expert is read, popular ones have dozens of rows
        _moe("moe-64", 64, 32, 8, 7168, 2048, True, "silu", True, False),
        # a rank of an expert-parallel group: a narrow layer, half the experts live elsewhere
        _moe("moe-19-absent", 19, 24, 4, 2048, 1408, False, "gelu_tanh", False, True),
    ]


def _log(rng, lo, hi):
    """An integer of lo .. hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("epilogue", "route", "moe"))
    if op == "epilogue":
        while True:
            m, n, k = _log(rng, 1, 4096), BLOCK * _log(rng, 1, 224), BLOCK * _log(rng, 1, 144)
            if n * k <= 28672 * 4096 and m * n * k <= 4096 * 28672 * 2048:
                break
        c = _epilogue("", m, n, k, rng.random() < 0.5, rng.choice(("none", "f32", "bf16")),
                      rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), rng.random() < 0.5)
    elif op == "route":
        while True:
            tokens, experts = _log(rng, 1, 8191), _log(rng, 2, 512)
            if tokens * experts <= 8191 * 256:
                break
        c = _route("", tokens, experts, rng.randint(1, min(experts, 12)), rng.choice(("softmax", "sigmoid")),
                   rng.random() < 0.5, rng.choice(("f32", "bf16")), rng.random() < 0.5)
    else:
        while True:
            experts, hidden, inter = _log(rng, 2, 64), BLOCK * _log(rng, 1, 56), BLOCK * _log(rng, 1, 56)
            if experts * hidden * inter <= 32 * 7168 * 2048:
                break
        c = _moe("", _log(rng, 1, 64), experts, rng.randint(1, min(experts, 8)), hidden, inter, rng.random() < 0.5,
                 rng.choice(("silu", "gelu", "gelu_tanh")), rng.random() < 0.5, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _heavy(shape, gen):
    """bf16 activations: N(0, 1) with 1% of the entries 20 times larger."""
    x = torch.randn(shape, generator=gen, device=gen.device)
    return torch.where(torch.rand(shape, generator=gen, device=gen.device) < 0.01, 20.0 * x, x).to(torch.bfloat16)


def _group_codes(x):
    """E4M3 codes [M, K] and float32 scales [M, K/128] of the 1x128-group quantization of x."""
    g = x.float().unflatten(-1, (-1, BLOCK))
    s = g.abs().amax(-1) / E4M3_MAX
    q = (g / torch.where(s == 0, 1.0, s).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.flatten(-2), s


def _block_codes(w, ue8m0):
    """E4M3 codes [N, K] (as bytes) and scales [N/128, K/128] of a weight in 128x128 blocks."""
    n, k = w.shape
    b = w.reshape(n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    s = b.abs().amax((1, 3)) / E4M3_MAX
    if ue8m0:  # the smallest power of two that is not below amax / 448, as its exponent's byte
        mant, e = torch.frexp(s)
        e = torch.where(mant == 0.5, e - 1, e).clamp(-127, 127)
        s, stored = torch.ldexp(torch.ones_like(s), e), (e + 127).to(torch.uint8)
    else:
        stored = s
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(n, k), stored


def _weight(n, k, ue8m0, gen):
    w = (0.02 * torch.randn((n, k), generator=gen, device=gen.device)).to(torch.bfloat16).float()
    return _block_codes(w, ue8m0)


def _prepare_epilogue(c, gen):
    m, n, k = c["m"], c["n"], c["k"]
    q, s = _group_codes(_heavy((m, k), gen))
    s_a = torch.zeros((k // BLOCK, (m + 3) // 4 * 4), device=gen.device)  # K-block-major, as the quantizer lays it out
    s_a[:, :m] = s.t()
    st = {"case": c, "a_q": q.view(torch.uint8), "s_a": s_a, "bias": None, "residual": None}
    st["w_q"], st["s_w"] = _weight(n, k, c["ue8m0"], gen)
    if c["bias"] != "none":
        bias = 0.5 * torch.randn(n, generator=gen, device=gen.device)
        st["bias"] = bias.to(torch.float32 if c["bias"] == "f32" else torch.bfloat16)
    if c["residual"]:
        st["residual"] = torch.randn((m, n), generator=gen, device=gen.device).to(torch.bfloat16)
    return st


def _prepare_route(c, gen):
    logits = 2.0 * torch.randn((c["tokens"], c["experts"]), generator=gen, device=gen.device)
    if c["masked"]:  # a third of the experts are closed to a token; every seventh token has none at all
        closed = torch.rand(logits.shape, generator=gen, device=gen.device) < 1 / 3
        closed[3::7] = True
        logits = logits.masked_fill(closed, -math.inf)
    return {"case": c, "logits": logits.to(torch.float32 if c["logits"] == "f32" else torch.bfloat16)}


def _prepare_moe(c, gen):
    dev, e, h, i = gen.device, c["experts"], c["hidden"], c["inter"]
    up = [_weight(2 * i, h, c["ue8m0"], gen) for _ in range(e)]
    down = [_weight(h, i, c["ue8m0"], gen) for _ in range(e)]
    st = {"case": c, "x": _heavy((c["tokens"], h), gen), "residual": None,
          "w13_q": torch.stack([w for w, _ in up]), "s_w13": torch.stack([s for _, s in up]),
          "w2_q": torch.stack([w for w, _ in down]), "s_w2": torch.stack([s for _, s in down])}
    p = torch.arange(1, e + 1, device=dev, dtype=torch.float32).pow(-ZIPF).expand(c["tokens"], e)
    ids = torch.multinomial(p, c["top_k"], replacement=False, generator=gen).to(torch.int32)
    st["weights"] = torch.softmax(torch.randn(ids.shape, generator=gen, device=dev), -1)
    if c["absent"]:  # experts that another rank holds
        ids = torch.where(torch.rand(ids.shape, generator=gen, device=dev) < 0.5, torch.full_like(ids, -1), ids)
    st["ids"] = ids
    if c["residual"]:
        st["residual"] = torch.randn((c["tokens"], h), generator=gen, device=dev).to(torch.bfloat16)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"epilogue": _prepare_epilogue, "route": _prepare_route, "moe": _prepare_moe}[case["op"]](case, gen)


# ---------------------------------------------------------------------------------- plain forms
def _activate(v, act):
    if act == "relu":
        return v.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_weight(q, s):
    """The float32 weight that codes [..., N, K] and block scales [..., N/128, K/128] stand for."""
    if s.dtype == torch.uint8:
        s = torch.exp2(s.float() - 127.0)
    w = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    return (w * s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)


def _plain_quantized(v):
    """The float32 values that the 1x128-group quantization of v stands for."""
    q, s = _group_codes(v)
    return (q.float().unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _plain_epilogue(st):
    c, m = st["case"], st["case"]["m"]
    a = st["a_q"].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, BLOCK)) * st["s_a"][:, :m].t().unsqueeze(-1)
    y = a.flatten(-2) @ _plain_weight(st["w_q"], st["s_w"]).t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _activate(y, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def _plain_route(st):
    c, logits = st["case"], st["logits"].float()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    top, ids = top[:, :c["top_k"]], ids[:, :c["top_k"]]
    none = torch.isinf(top)
    if c["scoring"] == "softmax":
        big = logits.amax(-1, keepdim=True)
        big = torch.where(torch.isinf(big), 0.0, big)
        w = torch.exp(top - big) / torch.exp(logits - big).sum(-1, keepdim=True)
    else:
        w = 1.0 / (1.0 + torch.exp(-top))
    w = torch.where(none, 0.0, w)
    if c["renorm"]:
        w = torch.where(none, 0.0, w / w.sum(-1, keepdim=True))
    return [torch.where(none, -1, ids).to(torch.int32), w]


def _plain_moe(st):
    """Every expert on every token, combined by the tokens' weights (zero where not routed)."""
    c, x = st["case"], st["x"]
    t, e = x.shape[0], c["experts"]
    there = st["ids"] >= 0
    share = torch.zeros((t, e), device=x.device)
    share.scatter_add_(1, st["ids"].clamp_min(0).long(), torch.where(there, st["weights"], 0.0))
    gate_up = torch.matmul(_plain_quantized(x), _plain_weight(st["w13_q"], st["s_w13"]).transpose(1, 2))  # [E, T, 2I]
    gate, up = gate_up.split(c["inter"], dim=-1)
    h = _plain_quantized(_activate(gate, c["act"]) * up)
    y = (torch.matmul(h, _plain_weight(st["w2_q"], st["s_w2"]).transpose(1, 2)) * share.t().unsqueeze(-1)).sum(0)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        return {"epilogue": _plain_epilogue, "route": _plain_route, "moe": _plain_moe}[c["op"]](state)
    import fine_grained_block_amd as fgb

    if c["op"] == "epilogue":
        return fgb.gemm_epilogue(state["a_q"], state["s_a"], state["w_q"], state["s_w"], bias=state["bias"],
                                 activation=c["act"], residual=state["residual"])
    if c["op"] == "route":
        return list(fgb.moe_route(state["logits"], c["top_k"], scoring=c["scoring"], renormalize=c["renorm"]))
    return fgb.moe_ffn(state["x"], state["ids"], state["weights"], state["w13_q"], state["s_w13"], state["w2_q"],
                       state["s_w2"], activation=c["act"], residual=state["residual"])


# -------------------------------------------------------------------------------------- work
def _reached(c, rng):
    """The distinct experts that one batch of the case's tokens is routed to."""
    # the top_k smallest of independent exponentials with rates p_e: a draw without replacement
    picks = (sorted((rng.expovariate(1.0) * (e + 1) ** ZIPF, e) for e in range(c["experts"]))[:c["top_k"]]
             for _ in range(c["tokens"]))
    return {e for row in picks for _, e in row if not c["absent"] or rng.random() < 0.5}


def work(case):
    c = case
    size = {"none": 0, "bf16": 2, "f32": 4}
    if c["op"] == "epilogue":
        m, n, k = c["m"], c["n"], c["k"]
        read = m * k + 4 * m * k // BLOCK + n * k + (1 if c["ue8m0"] else 4) * (n // BLOCK) * (k // BLOCK)
        return {"bytes": read + size[c["bias"]] * n + (2 + 2 * c["residual"]) * m * n,
                "flops": 2 * m * n * k}
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (size[c["logits"]] * c["experts"] + 8 * c["top_k"]),
                "flops": 2 * c["tokens"] * c["experts"]}
    t, h, i, pairs = c["tokens"], c["hidden"], c["inter"], c["tokens"] * c["top_k"] * (0.5 if c["absent"] else 1.0)
    weights = 3 * h * i * (1 + (1 if c["ue8m0"] else 4) / BLOCK ** 2)  # of one expert
    rng = random.Random(1)  # the mean number of experts that are read: the same few batches every time
    reached = sum(len(_reached(c, rng)) for _ in range(8)) / 8
    return {"bytes": reached * weights + t * h * (4 + 2 * c["residual"]) + 8 * t * c["top_k"],
            "flops": 6 * h * i * pairs}


# ------------------------------------------------------------------------------- 64-bit values
def _exact_weight(q, s):
    s = torch.pow(2.0, s.double() - 127.0) if s.dtype == torch.uint8 else s.double()
    return q.view(torch.float8_e4m3fn).double() * s.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


def _exact_e4m3(v):
    """Round to the nearest E4M3 value (ties to even, at most 448 in magnitude)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.pow(2.0, e - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantized(v):
    """Group quantization by definition.  Of bf16 rows the scale and the quotient are float32
    roundings by definition; of computed values they are taken in 64 bits."""
    part = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    part = part.float() if v.dtype == torch.bfloat16 else part
    s = part.abs().max(-1, keepdim=True).values / E4M3_MAX
    q = part / torch.where(s == 0, torch.ones_like(s), s)
    return (_exact_e4m3(q.double()) * s.double()).reshape(v.shape)


def _exact_act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
        return v * torch.sigmoid(2.0 * u)
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "epilogue":
        m, k = c["m"], c["k"]
        a = st["a_q"].view(torch.float8_e4m3fn).double()
        a = a * st["s_a"][:, :m].double().t().repeat_interleave(BLOCK, 1)
        y = torch.mm(a, _exact_weight(st["w_q"], st["s_w"]).t().contiguous())
        if st["bias"] is not None:
            y += st["bias"].double()
        y = _exact_act(y, c["act"])
        if st["residual"] is not None:
            y += st["residual"].double()
        return y
    if c["op"] == "route":
        x = st["logits"].double().cpu()
        ids = torch.full((c["tokens"], c["top_k"]), -1, dtype=torch.int32)
        w = torch.zeros((c["tokens"], c["top_k"]), dtype=torch.float64)
        left = x.clone()
        for j in range(c["top_k"]):
            best, at = left.max(-1)
            at = torch.where(left == best[:, None], torch.arange(c["experts"]), c["experts"]).min(-1).values
            open_ = torch.isfinite(best)
            ids[:, j] = torch.where(open_, at, -1).to(torch.int32)
            if c["scoring"] == "softmax":
                p = torch.exp(best - torch.logsumexp(x, -1))
            else:
                p = torch.sigmoid(best)
            w[:, j] = torch.where(open_, p, torch.zeros_like(p))
            left.scatter_(1, at[:, None].clamp_max(c["experts"] - 1), -math.inf)
        if c["renorm"]:
            w = torch.where(ids >= 0, w / w.sum(-1, keepdim=True), torch.zeros_like(w))
        return [ids, w]
    x = _exact_quantized(st["x"])
    y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device=x.device)
    for e in range(c["experts"]):
        at, slot = torch.nonzero(st["ids"] == e, as_tuple=True)
        if at.numel():
            gate_up = x[at] @ _exact_weight(st["w13_q"][e], st["s_w13"][e]).t().contiguous()
            h = _exact_act(gate_up[:, :c["inter"]], c["act"]) * gate_up[:, c["inter"]:]
            o = _exact_quantized(h) @ _exact_weight(st["w2_q"][e], st["s_w2"][e]).t().contiguous()
            y.index_add_(0, at, o * st["weights"][at, slot].double()[:, None])
    if st["residual"] is not None:
        y += st["residual"].double()
    return y
