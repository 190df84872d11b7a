"""moe_route_scored and the layers routed by it: refusals on the CPU, values on the GPU against the
definition in 64 bits.

Weights: the kernel's fp32 steps are a difference of logits (relative error of the exponential
2^-24 |l - m|), exponentials and divides of at most 2 ulp each, and sums of at most E <= 1024 positive
terms taken 32 ways (at most E / 32 + 5 <= 37 roundings): relative error below
(range of the row's logits + 64) 2^-24.  Experts have to be equal.
"""
import ctypes

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import moe_layer_router_b200 as m
    return m


# ----------------------------------------------------------------------------- definition in 64 bits

def define(logits, bias, k, n_group=1, topk_group=1, top2=True, sigmoid=True, renorm=True, scale=1.0):
    """(experts, weights in 64 bits) of one batch, a token at a time."""
    T, E = logits.shape
    idx = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = np.isfinite(l)
        if not live.any():
            continue
        s = np.zeros(E)
        with np.errstate(over="ignore"):
            if sigmoid:
                s[live] = 1 / (1 + np.exp(-l[live]))
            else:
                e = np.exp(l[live] - l[live].max())
                s[live] = e / e.sum()
        plain_order = bias is None and (n_group == 1 or not top2)
        key = np.where(live & np.isfinite(b), l if plain_order else s + b, -np.inf)
        per = E // n_group
        if n_group > 1:
            value = np.empty(n_group)
            for g in range(n_group):
                a = np.sort(key[g * per:(g + 1) * per])[::-1]
                value[g] = a[0] + (a[1] if top2 and per > 1 and np.isfinite(a[1]) else 0.0)
            keep = np.argsort(-value, kind="stable")[:topk_group]
            for g in set(range(n_group)) - set(keep.tolist()):
                key[g * per:(g + 1) * per] = -np.inf
        order = np.argsort(-key, kind="stable")[:k]
        order = order[np.isfinite(key[order])]
        n = len(order)
        idx[t, :n] = order
        if n == 0:
            continue
        if not renorm:
            w[t, :n] = s[order]
        elif sigmoid:                      # ratios, relative to the largest logit: no underflow
            lo = l[order]
            m = min(lo.max(), 0.0)
            r = np.where(lo >= 0, 1 / (1 + np.exp(-np.maximum(lo, 0))),
                         np.exp(np.minimum(lo, 0) - m) / (1 + np.exp(np.minimum(lo, 0))))
            w[t, :n] = r / r.sum()
        else:
            r = np.exp(l[order] - l[order].max())
            w[t, :n] = r / r.sum()
    return idx, w * scale


def call(moe, logits, bias, k, n_group=1, topk_group=1, top2=True, sigmoid=True, renorm=True, scale=1.0, stream=None):
    T, E = logits.shape
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    lg = torch.from_numpy(logits).cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    p = moe.moe_route_params(score=moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX, n_group=n_group,
                             topk_group=topk_group, group_score=moe.MOE_GROUP_TOP2 if top2 else moe.MOE_GROUP_MAX,
                             renormalise=int(renorm), scale=scale)
    moe.moe_route_scored(None, None, b, lg, p, T, 64, E, k, None, idx, w, None, stream=stream)
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7.0).all()          # nothing written behind the last token
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def check(moe, logits, bias, k, **kw):
    idx, w = call(moe, logits, bias, k, **kw)
    ri, rw = define(logits, bias, k, **kw)
    assert np.array_equal(idx, ri)
    live = np.isfinite(logits)
    span = np.where(live, logits, -3e38).max(1).astype(np.float64) - np.where(live, logits, 3e38).min(1)
    tol = (np.clip(span, 0, 1e3) + 64) * 2.0 ** -24
    assert (np.abs(w - rw) <= tol[:, None] * np.abs(rw) + 1e-37).all()
    return idx, w


def draw(T, E, seed, spread=1.0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, E)) * spread + 0.3 * r.standard_normal(E)).astype(np.float32)


def draw_bias(E, seed, size=0.1):
    return np.random.default_rng(seed + 1000).uniform(-size, size, E).astype(np.float32)


# ----------------------------------------------------------------------------- refusals (CPU)

def _raw(moe, T=8, E=64, k=4, params=None, idx=16, w=16, logits=16, bias=None, x=None, Wg=None, d=64, ws=None, nws=0):
    p = moe.moe_route_params(n_group=8, topk_group=4) if params is None else params
    return moe.lib().moe_route_scored(x, Wg, bias, logits, ctypes.byref(p) if p is not False else None, T, d, E, k, None, idx, w, ws,
                                      nws, None)


def test_refusals(moe):
    P = moe.moe_route_params
    shape, arg, align, small = -2, -1, -3, -4
    for kw in [dict(T=0), dict(k=0), dict(k=33, E=64), dict(E=1025), dict(E=3, k=4), dict(T=1 << 30, k=4)]:
        assert _raw(moe, params=P(), **kw) == shape, kw
    assert _raw(moe, params=P(n_group=0)) == shape
    assert _raw(moe, params=P(n_group=33, topk_group=33), E=66) == shape
    assert _raw(moe, params=P(n_group=7)) == shape                       # 64 % 7
    assert _raw(moe, params=P(n_group=8, topk_group=0)) == shape
    assert _raw(moe, params=P(n_group=8, topk_group=9)) == shape
    assert _raw(moe, params=P(n_group=32, topk_group=1)) == shape        # 2 experts left for k = 4
    assert _raw(moe, params=False) == arg
    for p in [P(score=2), P(score=-1), P(group_score=2), P(renormalise=2), P(scale=float("nan")),
              P(scale=float("inf"))]:
        assert _raw(moe, params=p) == arg
    assert _raw(moe, idx=None) == arg and _raw(moe, w=None) == arg
    assert _raw(moe, idx=20) == align and _raw(moe, logits=8) == align and _raw(moe, bias=4) == align
    assert _raw(moe, logits=None) == arg                                  # neither logits nor x
    assert _raw(moe, logits=None, x=16, Wg=16, d=100) == shape
    assert _raw(moe, logits=None, x=16, Wg=24, d=64) == align
    assert _raw(moe, logits=None, x=16, Wg=16, d=64, ws=16, nws=100) == small
    with pytest.raises(ValueError, match="cpu"):          # host tensors are refused before they reach a kernel
        moe.moe_route_scored(None, None, None, torch.zeros(8, 64), P(), 8, 64, 64, 2, None, 16, 16, None, stream=0)


def test_layer_refusals(moe):
    P = moe.moe_route_params
    lib = moe.lib()
    ok = (16,) * 3
    def fwd(p, cap=0, T=8):
        return lib.moe_layer_forward_scored(16, 16, None, ctypes.byref(p) if p else None, *ok, None, None, None, 0, T,
                                            128, 64, 2, 64, 1.0, cap, 16, 16, 1 << 10, None)
    assert fwd(None) == -1 and fwd(P(), cap=9) == -1 and fwd(P(n_group=5)) == -2 and fwd(P(), T=0) == -2
    assert fwd(P()) == -4                                                 # workspace too small
    assert lib.moe_layer_route_count_scored(16, 16, None, None, 0, 8, 128, 64, 2, 64, 16, 1 << 10, None) == -1
    q = moe.moe_w8_experts(*([16] * 6))
    def w8(p, a8, d=128, routed=q):
        return lib.moe_layer_forward_scored_w8(16, 16, None, ctypes.byref(p) if p else None,
                                               ctypes.byref(routed) if routed else None, None, 0, a8, 8, d, 64, 2, 64,
                                               1.0, 0, 16, 16, 1 << 10, None)
    assert w8(None, 0) == -1 and w8(P(), 2) == -1 and w8(P(), 0, routed=None) == -1
    assert w8(P(), 1, d=192) == -2 and w8(P(), 0) == -4


def test_params_struct_matches_the_header():
    import moe_layer_router_b200 as moe
    from test_abi import header_struct_fields
    assert [n for n, _ in moe.moe_route_params._fields_] == header_struct_fields("moe_route_params")


def test_definition_on_a_worked_example():
    # two groups of three; keys 0.9 0.1 0.1 | 0.6 0.55 0.5 as softmax-free sigmoids
    s = np.array([[0.9, 0.1, 0.1, 0.6, 0.55, 0.5]])
    l = np.log(s / (1 - s)).astype(np.float32)
    idx, w = define(l, None, 2, n_group=2, topk_group=1, top2=True, scale=2.0)
    assert idx.tolist() == [[3, 4]]                                       # 1.15 > 1.0
    np.testing.assert_allclose(w[0], 2 * np.array([0.6, 0.55]) / 1.15, rtol=1e-6)
    idx, _ = define(l, None, 2, n_group=2, topk_group=1, top2=False)
    assert idx.tolist() == [[0, 1]]                                       # by the best expert; the tie goes low
    idx, w = define(l, np.array([-1, 0, 0, 0, 0, 0], np.float32), 2, renorm=False)
    assert idx.tolist() == [[3, 4]]
    np.testing.assert_allclose(w[0], [0.6, 0.55], rtol=1e-6)              # weights without the bias


# ----------------------------------------------------------------------------- values (GPU)

SHAPES = [(1, 256, 8, 8, 4), (64, 256, 8, 8, 4), (1000, 8, 2, 1, 1), (777, 128, 8, 1, 1), (333, 160, 6, 8, 3),
          (100, 1024, 32, 1, 1), (100, 1024, 32, 32, 1), (50, 5, 5, 1, 1), (33, 39, 3, 13, 2), (65, 60, 4, 20, 9),
          (40, 1020, 7, 17, 5), (129, 64, 1, 4, 1), (31, 32, 32, 32, 32), (7, 1, 1, 1, 1), (50, 24, 3, 24, 3),
          (70, 512, 16, 16, 16), (90, 72, 5, 2, 1)]


@gpu
@pytest.mark.parametrize("T,E,k,n_group,topk_group", SHAPES)
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_values(moe, T, E, k, n_group, topk_group, sigmoid, with_bias):
    bias = draw_bias(E, 3, 0.1 if sigmoid else 1.0 / E) if with_bias else None
    for top2, renorm, scale in [(True, True, 2.5), (False, False, 1.0)]:
        check(moe, draw(T, E, E + T), bias, k, n_group=n_group, topk_group=topk_group, top2=top2, sigmoid=sigmoid,
              renorm=renorm, scale=scale)
    assert moe.moe_get_error() == 0


@gpu
def test_many_tokens(moe):
    check(moe, draw(20011, 96, 5), draw_bias(96, 5), 6, n_group=6, topk_group=3, scale=2.5)
    check(moe, draw(9001, 256, 6), draw_bias(256, 6), 8, n_group=8, topk_group=4, scale=2.5)
    assert moe.moe_get_error() == 0


@gpu
@pytest.mark.parametrize("E,k,n_group,topk_group", [(8, 2, 1, 1), (16, 15, 1, 1), (60, 6, 1, 1), (72, 5, 12, 4),
                                                    (128, 8, 1, 1), (130, 9, 1, 1), (187, 1, 1, 1), (256, 15, 16, 7),
                                                    (240, 8, 15, 2), (64, 16, 8, 4)])
def test_many_tokens_of_every_kind(moe, E, k, n_group, topk_group):
    # enough tokens for two per warp where that is done; an odd number, a masked tail, near and exact ties
    T = 4999
    logits = draw(T, E, E)
    logits[::7] = np.round(logits[::7] * 2) / 2
    r = np.random.default_rng(E)
    near = np.stack([r.permutation(E) for _ in range(len(logits[3::11]))]).astype(np.int32)
    logits[3::11] = (logits[3::11, :1].view(np.int32) + near).view(np.float32)
    logits[5::13][r.random(logits[5::13].shape) < 0.7] = -np.inf
    logits[-31:] = -np.inf
    kw = dict(n_group=n_group, topk_group=topk_group)
    check(moe, logits, draw_bias(E, 8), k, top2=True, sigmoid=True, scale=2.5, **kw)
    check(moe, logits, draw_bias(E, 8, 1.0 / E), k, top2=False, sigmoid=False, renorm=False, **kw)
    check(moe, logits, None, k, top2=False, sigmoid=False, **kw)
    check(moe, logits, np.zeros(E, np.float32), k, top2=True, sigmoid=True, renorm=False, **kw)
    assert moe.moe_get_error() == 0


@gpu
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("n_group,topk_group,top2", [(1, 1, True), (8, 3, False), (8, 3, True)])
def test_ties_go_to_the_lower_expert(moe, sigmoid, n_group, topk_group, top2):
    logits = np.round(draw(400, 64, 7) * 1.5).astype(np.float32)
    logits[0] = 0.0
    logits[1, 1::2] = -np.inf
    kw = dict(n_group=n_group, topk_group=topk_group, top2=top2, sigmoid=sigmoid)
    check(moe, logits, None, 8, **kw)
    idx, _ = check(moe, logits, np.zeros(64, np.float32), 8, **kw)
    assert idx[0].tolist() == list(range(8))
    check(moe, logits, (np.arange(64) % 3 - 1).astype(np.float32) / 4, 8, **kw)


@gpu
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (8, 3)])
def test_keys_closer_than_a_32_bit_rounding(moe, sigmoid, n_group, topk_group):
    # logits a few steps of fp32 apart in random order: fp32 scores of many of them are equal
    r = np.random.default_rng(11)
    T, E = 300, 64
    base = r.uniform(-3, 3, (T, 1)).astype(np.float32)
    steps = np.stack([r.permutation(E) for _ in range(T)])
    logits = (base.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    check(moe, logits, np.zeros(E, np.float32), 8, n_group=n_group, topk_group=topk_group, sigmoid=sigmoid)
    # and keys that a bias brings together: bias = -score + a few 2^-30
    l = draw(1, E, 12).repeat(T, 0)
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    if not sigmoid:
        e = np.exp(l[0].astype(np.float64) - l[0].max())
        s = e / e.sum()
    bias = (0.5 - s).astype(np.float32)
    check(moe, l[:3], bias, 8, n_group=n_group, topk_group=topk_group, sigmoid=sigmoid)


@gpu
@pytest.mark.parametrize("E,n_group,topk_group", [(1020, 17, 5), (1023, 31, 31), (1024, 1, 1), (992, 31, 9), (240, 15, 15)])
@pytest.mark.parametrize("top2", [True, False])
def test_near_keys_with_many_experts_per_lane(moe, E, n_group, topk_group, top2):
    # softmax sums of up to 60 terms per lane, and a bias that brings all keys of a row within some 2^-26 of each other (in
    # every other row: the rows between have other logits)
    T = 64
    l = draw(1, E, 51, spread=2.0)
    e = np.exp(l[0].astype(np.float64) - l[0].max())
    bias = (0.25 - e / e.sum()).astype(np.float32)
    logits = l.repeat(T, 0)
    logits[1::2] += draw(T // 2, E, 52)
    check(moe, logits, bias, 9, n_group=n_group, topk_group=topk_group, top2=top2, sigmoid=False, renorm=False)


@gpu
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("n_group,topk_group,top2", [(1, 1, True), (8, 2, True), (8, 2, False), (16, 9, True)])
@pytest.mark.parametrize("renorm", [True, False])
def test_masks(moe, sigmoid, n_group, topk_group, top2, renorm):
    T, E, k = 200, 64, 8
    r = np.random.default_rng(13)
    logits = draw(T, E, 14)
    logits[r.random((T, E)) < np.linspace(0, 1, T)[:, None]] = -np.inf   # from few to all masked
    logits[-5:] = -np.inf
    logits[20] = -np.inf
    logits[20, 37] = -2.0
    kw = dict(n_group=n_group, topk_group=topk_group, top2=top2, sigmoid=sigmoid, renorm=renorm, scale=2.5)
    bias = draw_bias(E, 14)
    for b in (None, bias, np.where(np.arange(E) % 5 == 0, -np.inf, bias).astype(np.float32),
              np.full(E, -np.inf, np.float32)):
        idx, w = check(moe, logits, b, k, **kw)
        assert (idx[-1] == -1).all() and (w[-1] == 0).all()
    assert moe.moe_get_error() == 0                                       # masks are no errors


@gpu
@pytest.mark.parametrize("sigmoid", [True, False])
def test_far_logits(moe, sigmoid):
    # scores that saturate or underflow: lowest and largest finite values, hundreds either way
    logits = draw(64, 40, 15, spread=60.0)
    logits[0] = np.finfo(np.float32).min
    logits[1] = np.finfo(np.float32).max
    logits[2, ::2] = np.finfo(np.float32).min
    logits[3] = np.linspace(-600, -100, 40)
    logits[4] = np.linspace(100, 600, 40)
    for bias in (None, draw_bias(40, 15)):
        for renorm in (True, False):
            idx, w = check(moe, logits, bias, 4, sigmoid=sigmoid, renorm=renorm)
            assert np.isfinite(w).all()
    assert moe.moe_get_error() == 0


@gpu
@pytest.mark.parametrize("T", [12, 9000])
@pytest.mark.parametrize("with_bias", [True, False])
def test_selected_scores_far_apart(moe, T, with_bias):
    # renormalised sigmoid weights whose smaller scores underflow in 32 bits while their ratio to the largest does not
    rows = np.stack([np.linspace(hi, lo, 8) for hi, lo in [(-59, -95), (-50, -88), (-59.99, -87.5), (-30, -110), (0, -87.4),
                                                           (3, -85), (40, -44), (-60.01, -140), (-86, -104), (-59, -59),
                                                           (88, -0.5), (-20, -103)]]).astype(np.float32)
    logits = np.tile(rows, (T // 12, 1))
    bias = np.zeros(8, np.float32) if with_bias else None
    for k in (8, 5):
        idx, w = check(moe, logits, bias, k)
        assert (w > 0).all()


def device_us(moe, logits, bias, k, kw, n=20):      # the least of n calls
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    lg, b = torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda()
    p = moe.moe_route_params(**kw)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(n + 1)]
    for _ in range(3):
        moe.moe_route_scored(None, None, b, lg, p, T, 64, E, k, None, idx, w, None)
    for e in ev:
        e.record()
        moe.moe_route_scored(None, None, b, lg, p, T, 64, E, k, None, idx, w, None)
    torch.cuda.synchronize()
    return min(x.elapsed_time(y) * 1e3 for x, y in zip(ev, ev[1:]))


@gpu
@pytest.mark.parametrize("low", [-1e4, -1e9, float(np.finfo(np.float32).min), 1e4])
@pytest.mark.parametrize("score,group_score,n_group", [(0, 0, 1), (0, 1, 8), (1, 0, 8), (1, 1, 8)])
def test_one_large_finite_bias_costs_no_second_pass(moe, low, score, group_score, n_group):
    # an expert that is switched off (or always on) by a large finite bias, as programs do that have no -inf
    T, E, k = 16384, 256, 8
    logits, bias = draw(T, E, 41), draw_bias(E, 41, 0.1 if score else 1.0 / E)
    kw = dict(score=score, group_score=group_score, n_group=n_group, topk_group=max(1, n_group // 2))
    plain = device_us(moe, logits, bias, k, kw)
    bias[77] = low
    off = device_us(moe, logits, bias, k, kw)
    assert off < 1.7 * plain, f"{plain:.1f} -> {off:.1f} us"      # a second pass for every token: 2.4 to 3.1 times
    check(moe, logits[:2000], bias, k, n_group=n_group, topk_group=max(1, n_group // 2), top2=bool(group_score),
          sigmoid=bool(score))


@gpu
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_nan_and_inf_are_reported_and_masked(moe, bad, sigmoid):
    logits = draw(32, 64, 16)
    clean = logits.copy()
    logits[3, 5] = bad
    clean[3, 5] = -np.inf
    ri, rw = define(clean, None, 4, sigmoid=sigmoid)
    idx, w = call(moe, logits, None, 4, sigmoid=sigmoid)
    assert moe.moe_get_error() == moe.MOE_ERR_CHECK and moe.moe_get_error() == 0
    assert np.array_equal(idx, ri)
    np.testing.assert_allclose(w, rw, rtol=128 * 2.0 ** -24)
    bias = draw_bias(64, 16)
    bias[7] = bad
    idx, _ = call(moe, clean, bias, 4, n_group=4, topk_group=2, sigmoid=sigmoid)
    assert moe.moe_get_error() == moe.MOE_ERR_CHECK
    assert not (idx == 7).any()


@gpu
@pytest.mark.parametrize("T,d,E,k", [(3, 512, 64, 4), (130, 4096, 256, 8), (200, 256, 300, 6)])
def test_from_hidden_states(moe, T, d, E, k):
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    Wg = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    bias = torch.from_numpy(draw_bias(E, 17)).cuda()
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    ws = torch.empty(moe.moe_workspace_bytes(T, d, E, k, 64), dtype=torch.uint8, device="cuda")
    lg, lg0 = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    i0 = torch.empty(T, k, dtype=torch.int32, device="cuda")
    idx, w, w0 = torch.empty_like(i0), torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route(x, Wg, None, None, T, d, E, k, lg0, i0, w0, ws)
    moe.moe_route_scored(x, Wg, bias, None, p, T, d, E, k, lg, idx, w, ws)
    assert torch.equal(lg, lg0)                                            # the same product, the same sums
    ri, _ = define(lg.cpu().numpy(), bias.cpu().numpy(), k, n_group=4, topk_group=2, scale=2.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)                    # without logits_out
    moe.moe_route_scored(x, Wg, bias, None, p, T, d, E, k, None, i2, w2, ws)
    assert torch.equal(i2, idx) and torch.equal(w2, w)
    lg3 = torch.empty_like(lg)                                             # from logits, copied out
    moe.moe_route_scored(None, None, bias, lg, p, T, d, E, k, lg3, i2, w2, None)
    assert torch.equal(i2, idx) and torch.equal(w2, w) and torch.equal(lg3, lg)
    assert moe.moe_get_error() == 0


def layer_inputs(T, d, E, f, fs, seed=19):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, n: (torch.randn(*s, generator=g, device="cuda") * n ** -0.5).bfloat16()
    return dict(x=r(T, d, n=1), Wg=r(E, d, n=d), W=(r(E, f, d, n=d), r(E, f, d, n=d), r(E, d, f, n=f)),
                Ws=(r(fs, d, n=d), r(fs, d, n=d), r(d, fs, n=fs)) if fs else (None, None, None))


@gpu
@pytest.mark.parametrize("T,fs,cap", [(1, 0, 0), (77, 128, 0), (300, 0, 2), (2000, 128, 0)])
def test_layer_is_its_stages(moe, T, fs, cap):
    d, E, k, f = 256, 16, 4, 192
    a = layer_inputs(T, d, E, f, fs)
    bias = torch.from_numpy(draw_bias(E, 20)).cuda()
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    ws = torch.empty(moe.moe_workspace_bytes(T, d, E, k, f, fs), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_forward_scored(a["x"], a["Wg"], bias, p, *a["W"], *a["Ws"], fs, T, d, E, k, f, 1.0, cap, out, ws)
    two = torch.empty_like(out)
    ws2 = torch.empty_like(ws)
    moe.moe_layer_route_count_scored(a["x"], a["Wg"], bias, p, fs, T, d, E, k, f, ws2)
    L = moe.moe_workspace_layout(T, d, E, k, f, fs)
    counts = moe.workspace_view(ws2, L, "counts_raw", (E,), torch.int32).clone()
    C = moe.moe_capacity(T, E, k, 1.0, cap)
    moe.moe_layer_finish(a["x"], *a["W"], *a["Ws"], fs, T, d, E, k, f, C, None, two, ws2)
    assert torch.equal(out, two)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_scored(a["x"], a["Wg"], bias, None, p, T, d, E, k, None, idx, w, ws2)
    assert torch.equal(counts.long(), torch.bincount(idx.flatten().long(), minlength=E))
    assert torch.equal(moe.workspace_view(ws, L, "idx", (T, k), torch.int32), idx)
    assert torch.equal(moe.workspace_view(ws, L, "w", (T, k), torch.float32), w)
    # softmax over all experts, no bias: the layer's own routing
    q = moe.moe_route_params(score=moe.MOE_SCORE_SOFTMAX)
    moe.moe_layer_forward_scored(a["x"], a["Wg"], None, q, *a["W"], *a["Ws"], fs, T, d, E, k, f, 1.0, cap, out, ws)
    moe.moe_layer_forward(a["x"], a["Wg"], None, *a["W"], *a["Ws"], fs, T, d, E, k, f, 1.0, cap, two, ws2)
    assert torch.equal(out, two)
    assert moe.moe_get_error() == 0


@gpu
@pytest.mark.parametrize("a8", [0, 1])
def test_fp8_layer(moe, a8):
    T, d, E, k, f, fs = 150, 256, 16, 4, 256, 128
    a = layer_inputs(T, d, E, f, fs)
    def q8(w):
        s = w.float().abs().amax(-1) / 448
        return (w.float() / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s.contiguous()
    def experts(W):
        (q1, s1), (q3, s3), (q2, s2) = (q8(w) for w in W)
        return dict(W1q=q1, s1=s1, W3q=q3, s3=s3, W2q=q2, s2=s2)
    R, S = experts(a["W"]), experts(a["Ws"])
    bytes_ = moe.moe_workspace_bytes_a8(T, d, E, k, f, fs) if a8 else moe.moe_workspace_bytes(T, d, E, k, f, fs)
    ws = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    out, two = (torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = moe.moe_route_params(score=moe.MOE_SCORE_SOFTMAX)
    moe.moe_layer_forward_scored_w8(a["x"], a["Wg"], None, q, R, S, fs, a8, T, d, E, k, f, 1.0, 0, out, ws)
    ref = moe.moe_layer_forward_w8a8 if a8 else moe.moe_layer_forward_w8
    order = ("W1q", "s1", "W3q", "s3", "W2q", "s2")
    ref(a["x"], a["Wg"], None, *[R[n] for n in order], *[S[n] for n in order], fs, T, d, E, k, f, 1.0, 0, two, ws)
    assert torch.equal(out, two)
    bias = torch.from_numpy(draw_bias(E, 21)).cuda()
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    moe.moe_layer_forward_scored_w8(a["x"], a["Wg"], bias, p, R, S, fs, a8, T, d, E, k, f, 1.0, 0, out, ws)
    L = moe.moe_workspace_layout(T, d, E, k, f, fs)
    lg = moe.workspace_view(ws, L, "logits", (T, E), torch.float32).cpu().numpy()
    ri, _ = define(lg, bias.cpu().numpy(), k, n_group=4, topk_group=2, scale=2.5)
    assert np.array_equal(moe.workspace_view(ws, L, "idx", (T, k), torch.int32).cpu().numpy(), ri)
    assert moe.moe_get_error() == 0


@gpu
@pytest.mark.parametrize("exchange", ["put", "fused", "a2a"])
@pytest.mark.parametrize("cap_mode", [0, 1])
@pytest.mark.parametrize("masked", [False, True])
def test_scored_routing_goes_on_into_the_sharded_and_the_expert_parallel_layer(moe, exchange, cap_mode, masked):
    # from moe_layer_route_count_scored on as from moe_layer_route_count, against the whole batch in one call, bit for bit;
    # masked: most experts switched off, so that every token has slots that no expert is left for
    from moe_layer_router_b200.ep import EmulatedEP
    R, T, d, E, k, f, fs = 2, 96, 256, 16, 4, 192, 128
    a = layer_inputs(R * T, d, E, f, fs, seed=23)
    bias = draw_bias(E, 24)
    if masked:
        bias[[0, 1, 2, 5, 6, 7, 8, 9, 10, 12, 14]] = -np.inf
    bias = torch.from_numpy(bias).cuda()
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    C = moe.moe_capacity(R * T, E, k, 1.25, cap_mode)
    whole = torch.empty(R * T, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_workspace_bytes(R * T, d, E, k, f, fs), dtype=torch.uint8, device="cuda")
    moe.moe_layer_forward_scored(a["x"], a["Wg"], bias, p, *a["W"], *a["Ws"], fs, R * T, d, E, k, f, 1.25, cap_mode, whole,
                                 ws)
    LW = moe.moe_workspace_layout(R * T, d, E, k, f, fs)
    idx = moe.workspace_view(ws, LW, "idx", (R * T, k), torch.int32)
    dest = moe.workspace_view(ws, LW, "dest", (R * T, k), torch.int32)
    assert bool((idx == -1).any(1).all()) == masked and (dest[idx == -1] == -1).all()
    if cap_mode:
        assert bool((dest[idx != -1] == -1).any())                        # capacity drops slots too
    x = [a["x"][r * T:(r + 1) * T].contiguous() for r in range(R)]
    # token-sharded
    L = moe.moe_workspace_layout(T, d, E, k, f, fs)
    parts = [torch.empty(moe.moe_workspace_bytes(T, d, E, k, f, fs), dtype=torch.uint8, device="cuda") for _ in range(R)]
    for r in range(R):
        moe.moe_layer_route_count_scored(x[r], a["Wg"], bias, p, fs, T, d, E, k, f, parts[r])
    counts = torch.stack([moe.workspace_view(w, L, "counts_raw", (E,), torch.int32) for w in parts])
    out = [torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(R)]
    for r in range(R):
        base = torch.empty(E, dtype=torch.int32, device="cuda")
        moe.moe_fill_base(counts, R, r, E, base)
        moe.moe_layer_finish(x[r], *a["W"], *a["Ws"], fs, T, d, E, k, f, C, base, out[r], parts[r])
    assert torch.equal(torch.cat(out), whole)

    # expert-parallel, its routing step replaced
    class Scored:
        def __getattr__(self, name):
            return getattr(moe, name)

        def moe_layer_route_count(self, x, Wg, bias, *rest):
            moe.moe_layer_route_count_scored(x, Wg, bias, p, *rest)

    ep = EmulatedEP(R, T, d, E, k, f, fs, exchange=exchange)
    ep.moe = Scored()
    for o in out:
        o.zero_()
    ep.forward(x, a["Wg"], bias, *a["W"], *a["Ws"], 1.25, cap_mode, out)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(out), whole)
    assert moe.moe_get_error() == 0


@gpu
def test_padded_tokens_drop_out_of_the_layer(moe):
    # logits of -inf from a masked batch: the permutation drops the rows, the combine leaves them zero
    T, d, E, k, f, live = 96, 256, 16, 4, 128, 61
    a = layer_inputs(T, d, E, f, 0)
    logits = draw(T, E, 22)
    logits[live:] = -np.inf
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    idx, w = i32(T, k), torch.empty(T, k, device="cuda")
    moe.moe_route_scored(None, None, None, torch.from_numpy(logits).cuda(), p, T, d, E, k, None, idx, w, None)
    ws = torch.empty(moe.moe_workspace_bytes(T, d, E, k, f), dtype=torch.uint8, device="cuda")
    raw, cnt, off, dest, src = i32(E), i32(E), i32(E + 1), i32(T, k), i32(T * k)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    xp, h, yp, out = bf(T * k, d), bf(T * k, f), bf(T * k, d), bf(T, d)
    moe.moe_permute(a["x"], idx, T, d, E, k, -1, raw, cnt, off, dest, src, xp, ws)
    assert int(off[E]) == live * k and (dest[live:] == -1).all()
    moe.moe_expert_ffn(xp, off, T * k, E, d, f, *a["W"], h, yp, ws)
    moe.moe_combine(yp, dest, w, None, T, d, k, out)
    assert (out[live:] == 0).all() and (out[:live].float().abs().sum(1) > 0).all()
    assert moe.moe_get_error() == 0


@gpu
def test_other_stream_and_graph_replay(moe):
    T, E, k = 130, 64, 6
    logits, bias = draw(T, E, 23), draw_bias(E, 23)
    kw = dict(n_group=8, topk_group=3, scale=2.5)
    ri, _ = define(logits, bias, k, **kw)
    s = torch.cuda.Stream()
    lg = torch.from_numpy(logits).cuda()
    b = torch.from_numpy(bias).cuda()
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    p = moe.moe_route_params(n_group=8, topk_group=3, scale=2.5)
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_route_scored(None, None, b, lg, p, T, 64, E, k, None, idx, w, None, stream=s)
    s.synchronize()
    assert np.array_equal(idx.cpu().numpy(), ri)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_scored(None, None, b, lg, p, T, 64, E, k, None, idx, w, None)
    other = draw(T, E, 24)
    lg.copy_(torch.from_numpy(other))
    p.scale = 100.0                                     # the parameters were read at the call
    graph.replay()
    torch.cuda.synchronize()
    ri, rw = define(other, bias, k, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5)


@gpu
def test_offsets_past_32_bits(moe):
    # more than 2^31 logits, all masked but the first and last rows
    E, k, T = 1024, 2, (1 << 21) + 37
    kw = dict(n_group=8, topk_group=4, scale=2.5)
    logits, bias = draw(80, E, 31), draw_bias(E, 31)
    lg = torch.full((T, E), -np.inf, device="cuda")
    lg[:40] = torch.from_numpy(logits[:40]).cuda()
    lg[-40:] = torch.from_numpy(logits[40:]).cuda()
    idx, w = torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.full((T, k), -7.0, device="cuda")
    p = moe.moe_route_params(n_group=8, topk_group=4, scale=2.5)
    moe.moe_route_scored(None, None, torch.from_numpy(bias).cuda(), lg, p, T, 64, E, k, None, idx, w, None)
    torch.cuda.synchronize()
    assert moe.moe_get_error() == 0
    ri, rw = define(logits, bias, k, **kw)
    assert np.array_equal(torch.cat([idx[:40], idx[-40:]]).cpu().numpy(), ri)
    np.testing.assert_allclose(torch.cat([w[:40], w[-40:]]).cpu().numpy(), rw, rtol=1e-5)
    assert (idx[40:-40] == -1).all() and (w[40:-40] == 0).all()
