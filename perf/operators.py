"""Timed cases of the scored router and of the dense layer, with their plain forms.

``own`` false: elementary torch operations in 32 bits (the selection keys in 64, since two keys that
lie closer than a 32-bit rounding would otherwise change places), rounded once at the end.
``own`` true: the library's entry points ``moe_route_scored``, ``moe_linear`` and ``moe_linear_w8a8``.

A case is a dict of plain values; ``op`` is "route", "linear" or "linear8".

route   logits [T, E] fp32 (the router product, as moe_route takes it in logits_in) -> experts [T, k] and
        weights [T, k].  score 0: softmax over the experts, 1: sigmoid of each.  bias: a per-expert
        selection bias.  groups > 1: only the experts of the topk_group best groups can be selected, a
        group's value being its largest key (top2 false) or the sum of its two largest.
        pad: rows at the end of the batch that hold no token (every logit -inf).
linear  y = act(x W^T + bias) + residual on bf16 x [M, K] and W [N, K]; act "swiglu" is
        silu(x W^T + bias) * (x W_up^T + bias_up).
linear8 the same layer with e4m3 weights and one fp32 scale per weight row; each row of x is rounded to e4m3
        with the scale amax / 448 first.
"""
import math

import torch

own = False


def listed():
    return [
        # one token being decoded, 256 experts in 8 groups: all latency
        dict(name="route one token", op="route", T=1, E=256, k=8, groups=8, topk_group=4, top2=True, score=1, bias=True,
             renorm=True, scale=2.5, pad=0),
        # a decode batch of 256 sequences, 40 of its slots empty
        dict(name="route decode batch", op="route", T=256, E=256, k=8, groups=8, topk_group=4, top2=True, score=1,
             bias=True, renorm=True, scale=2.5, pad=40),
        # a prefill chunk of the same router
        dict(name="route prefill 256 experts", op="route", T=32768, E=256, k=8, groups=8, topk_group=4, top2=True,
             score=1, bias=True, renorm=True, scale=2.5, pad=0),
        # prefill with 128 ungrouped experts, softmax scores
        dict(name="route prefill 128 experts", op="route", T=16384, E=128, k=8, groups=1, topk_group=1, top2=False,
             score=0, bias=False, renorm=True, scale=1.0, pad=0),
        # an odd number of tokens, groups of 20 experts by their best one, weights as the softmax gives them
        dict(name="route odd groups", op="route", T=4099, E=160, k=6, groups=8, topk_group=3, top2=False, score=0,
             bias=True, renorm=False, scale=16.0, pad=3),
        # one token through a square projection with its residual: the weights' stream
        dict(name="linear one token", op="linear", M=1, N=4096, K=4096, act="none", bias=True, residual=True),
        # a decode batch through a wide down projection
        dict(name="linear decode batch", op="linear", M=256, N=7168, K=2048, act="none", bias=False, residual=True),
        # odd sizes throughout: ragged tiles on every side, an output row that is not a multiple of 16 bytes
        dict(name="linear ragged", op="linear", M=777, N=1001, K=1384, act="gelu", bias=True, residual=True),
        # a prefill chunk through a square projection with its residual
        dict(name="linear prefill", op="linear", M=16384, N=4096, K=4096, act="none", bias=True, residual=True),
        # the first half of a gated dense feed-forward block: the largest
        dict(name="linear prefill gated", op="linear", M=4096, N=14336, K=4096, act="swiglu", bias=False,
             residual=False),
        # a few drafted tokens through a gated layer with fp8 weights
        dict(name="linear8 few tokens", op="linear8", M=24, N=2048, K=7168, act="swiglu", bias=False, residual=False),
        # a prefill chunk through the first half of a dense feed-forward block with fp8 weights
        dict(name="linear8 prefill", op="linear8", M=4096, N=14336, K=4096, act="gelu_tanh", bias=True,
             residual=False),
    ]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        T = _log_int(rng, 1, 32768)
        groups = rng.choice((1, 1, 2, 4, 5, 8, 16))
        each = max(2, _log_int(rng, 8, 512) // groups)
        if rng.random() < 0.5:
            each = max(4, each // 4 * 4)
        E = groups * each
        topk_group = rng.randint(1, groups)
        k = rng.randint(1, min(16, topk_group * each))
        while T * E > 32768 * 256:
            T //= 2
        return dict(op="route", T=T, E=E, k=k, groups=groups, topk_group=topk_group, top2=rng.random() < 0.5,
                    score=rng.randint(0, 1), bias=rng.random() < 0.7, renorm=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5, 16.0)), pad=rng.choice((0, 0, T // 8, T // 3)))
    while True:
        act, op = rng.choice(ACTS), rng.choice(("linear", "linear", "linear8"))
        M, N = _log_int(rng, 1, 16384), _log_int(rng, 64, 14336)
        K = 8 * _log_int(rng, 8, 1792) if op == "linear" else 16 * _log_int(rng, 8, 896)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        case = dict(op=op, M=M, N=N, K=K, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        if work(case)["flops"] <= 4 * 4096 * 14336 * 4096:
            return case


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * 4 + (E * 4 if case["bias"] else 0) + T * k * 8, "flops": T * E * 4}
    M, N, K = case["M"], case["N"], case["K"]
    two = 2 if case["act"] == "swiglu" else 1
    weights = two * N * (K + 4) if case["op"] == "linear8" else 2 * two * N * K
    data = weights + 2 * (M * K + M * N + (M * N if case["residual"] else 0))
    return {"bytes": data + (4 * two * N if case["bias"] else 0), "flops": 2 * M * N * K * two}


def _rows_to_e4m3(x):
    """(codes as bytes, one fp32 scale per row): e4m3(x / scale) with scale = amax / 448, 1 for a row of zeros."""
    x = x.float()
    most = x.abs().amax(dim=1)
    scale = most / torch.full_like(most, 448)       # by a tensor: torch multiplies by a number's rounded reciprocal
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = dict(case)
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # router scores: unit variance over tokens and a popularity that differs from expert to expert
        s["logits"] = normal(T, E) + 0.3 * normal(E)
        if case["pad"]:
            s["logits"][T - case["pad"]:] = -math.inf
        s["sel_bias"] = None
        if case["bias"]:
            spread = 0.1 if case["score"] == 1 else 1.0 / E     # of the order of the scores it balances
            s["sel_bias"] = (torch.rand(E, generator=g, device="cuda") * 2 - 1) * spread
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
        return s
    M, N, K = case["M"], case["N"], case["K"]
    gated = case["act"] == "swiglu"
    s["x"] = normal(M, K).bfloat16()
    s["W"] = normal(N, K, std=K ** -0.5).bfloat16()
    s["W_up"] = normal(N, K, std=K ** -0.5).bfloat16() if gated else None
    if case["op"] == "linear8":
        s["W"], s["sw"] = _rows_to_e4m3(s["W"])
        s["W_up"], s["sw_up"] = _rows_to_e4m3(s["W_up"]) if gated else (None, None)
        s["ws"] = torch.empty(M * K + 4 * M + 512, dtype=torch.uint8, device="cuda")
    s["b"] = normal(N, std=0.5) if case["bias"] else None
    s["b_up"] = normal(N, std=0.5) if case["bias"] and gated else None
    s["r"] = normal(M, N).bfloat16() if case["residual"] else None
    s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    return s


def run(state):
    if state["op"] == "route":
        return _route_own(state) if own else _route_plain(state)
    return _linear_own(state) if own else _linear_plain(state)


def _route_own(s):
    import moe_layer_router_b200 as moe

    params = moe.moe_route_params(
        score=moe.MOE_SCORE_SIGMOID if s["score"] else moe.MOE_SCORE_SOFTMAX, n_group=s["groups"],
        topk_group=s["topk_group"], group_score=moe.MOE_GROUP_TOP2 if s["top2"] else moe.MOE_GROUP_MAX,
        renormalise=int(s["renorm"]), scale=s["scale"])
    moe.moe_route_scored(None, None, s["sel_bias"], s["logits"], params, s["T"], 64, s["E"], s["k"], None, s["idx"],
                         s["w"], None)
    return {"idx": s["idx"], "w": s["w"]}


def _linear_own(s):
    import moe_layer_router_b200 as moe

    kind = getattr(moe, "MOE_ACT_" + s["act"].upper())
    if s["op"] == "linear8":
        moe.moe_linear_w8a8(s["x"], s["W"], s["sw"], s["W_up"], s["sw_up"], s["b"], s["b_up"], s["r"], s["M"], s["N"],
                            s["K"], kind, s["y"], s["ws"])
        return {"y": s["y"]}
    moe.moe_linear(s["x"], s["W"], s["W_up"], s["b"], s["b_up"], s["r"], s["M"], s["N"], s["K"], kind, s["y"])
    return {"y": s["y"]}


def _scores(logits, score):
    if score == 1:
        return 1 / (1 + torch.exp(-logits))
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _route_plain(s):
    T, E, k, groups = s["T"], s["E"], s["k"], s["groups"]
    none = -math.inf
    wide = s["logits"].double()
    key = _scores(wide, s["score"])
    if s["sel_bias"] is not None:
        key = key + s["sel_bias"].double()
    key = torch.where(wide == none, torch.full_like(key, none), key)
    if groups > 1:
        inside = key.view(T, groups, E // groups).sort(dim=2, descending=True).values
        value = inside[:, :, 0]
        if s["top2"]:
            value = value + torch.where(inside[:, :, 1] == none, torch.zeros_like(value), inside[:, :, 1])
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
        out = torch.ones(T, groups, dtype=torch.bool, device=key.device)
        out.scatter_(1, kept, False)
        key = key.masked_fill(out.repeat_interleave(E // groups, dim=1), none)
    key, place = key.sort(dim=1, descending=True, stable=True)
    empty = key[:, :k] == none
    place = place[:, :k]
    w = _scores(s["logits"], s["score"]).gather(1, place).masked_fill(empty, 0.0)
    if s["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return {"idx": place.masked_fill(empty, -1).int(), "w": w * s["scale"]}


def _product(s, weight, scale):
    if s["op"] == "linear":
        return s["x"].float() @ s[weight].float().t()
    codes, rows = _rows_to_e4m3(s["x"])
    return (_e4m3(codes).float() @ _e4m3(s[weight]).float().t()) * rows[:, None] * s[scale]


def _linear_plain(s):
    y = _product(s, "W", "sw")
    if s["b"] is not None:
        y = y + s["b"]
    act = s["act"]
    if act == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif act == "swiglu":
        up = _product(s, "W_up", "sw_up")
        if s["b_up"] is not None:
            up = up + s["b_up"]
        y = y / (1 + torch.exp(-y)) * up
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.bfloat16()}


def exact(case, seed):
    """The definitions in 64 bits: y of the dense layer, the weights of the router (its experts are whole
    numbers, which are compared as they are)."""
    s = prepare(case, seed)
    if case["op"] != "route":
        rows = []
        eight = case["op"] == "linear8"
        W, W_up = s["W"], s["W_up"]
        if eight:       # the rounding to e4m3 is taken in 32 bits by definition; all else in 64
            W = _e4m3(W).double() * s["sw"].double()[:, None]
            W_up = None if W_up is None else _e4m3(W_up).double() * s["sw_up"].double()[:, None]
        for x in s["x"].split(1024):            # a block of rows at a time: 64-bit copies are large
            if eight:
                codes, size = _rows_to_e4m3(x)
                x = _e4m3(codes).double() * size.double()[:, None]
            z = torch.mm(x.double(), W.double().T)
            z = z if s["b"] is None else z.add(s["b"].double())
            if case["act"] == "relu":
                z = z.clamp(min=0)
            elif case["act"] == "silu":
                z = z * z.sigmoid()
            elif case["act"] == "gelu":         # x times the normal distribution function at x
                z = z * torch.special.ndtr(z)
            elif case["act"] == "gelu_tanh":    # (1 + tanh u) / 2 = sigmoid(2 u)
                z = z * torch.sigmoid((8 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
            elif case["act"] == "swiglu":
                u = torch.mm(x.double(), W_up.double().T)
                u = u if s["b_up"] is None else u.add(s["b_up"].double())
                z = z * z.sigmoid() * u
            rows.append(z)
        y = torch.cat(rows)
        return {"y": y if s["r"] is None else y.add_(s["r"].double())}
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    lg = s["logits"].double()
    p = lg.sigmoid() if case["score"] else torch.nan_to_num(lg.softmax(1), nan=0.0)
    dead = torch.isneginf(lg)
    q = p.clone() if s["sel_bias"] is None else p + s["sel_bias"].double()
    q[dead] = -1e300
    if G > 1:
        n = 2 if case["top2"] else 1
        best = q.view(T, G, -1).topk(n, dim=2).values
        best = torch.where(best == -1e300, torch.zeros_like(best), best).sum(2)
        floor = best.topk(case["topk_group"], dim=1).values[:, -1:]
        q[(best < floor).repeat_interleave(E // G, 1)] = -1e300
    at = q.topk(k, dim=1)
    w = p.gather(1, at.indices) * (at.values > -1e300)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return {"idx": None, "w": w * case["scale"]}
