"""moe_linear and moe_linear_w8a8: refusals on the CPU, values on the GPU against products in 64 bits.

Tolerance per output, by arithmetic.  Each tensor-core instruction adds 16 (bf16) or 32 (e4m3) exact
products into the fp32 accumulator; an addition that truncates loses at most 2^-23 of the running sum,
which S = sum |x_i w_i| bounds, and the joining of at most 8 partial sums and the two fp32 additions after
it are 10 more: the pre-activation is off by at most (K / 16 + 12) 2^-23 (S + |bias|).  The
activations have slopes below 1.13 (gelu) and are evaluated to a few ulp: 2^-20 of their value; the
gated product carries both factors' errors.  Then one rounding to bf16, at most 2^-8 of the value.
"""
import math
import pathlib
import re

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


@pytest.fixture(scope="module")
def moe():
    import moe_layer_router_b200 as m
    return m


# ----------------------------------------------------------------------------- definition in 64 bits

def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def define(act, x, W, W_up=None, bias=None, bias_up=None, residual=None):
    """(y, tolerance) in 64 bits from 64-bit operands."""
    K = x.shape[1]
    unit = (K / 16 + 12) * 2.0 ** -23

    def pre(w, b):
        z, s = x @ w.T, x.abs() @ w.abs().T
        if b is not None:
            z, s = z + b, s + b.abs()
        return z, unit * s

    z, dz = pre(W, bias)
    if act == "swiglu":
        u, du = pre(W_up, bias_up)
        g = act64("silu", z)
        y = g * u
        dy = 1.1 * dz * (u.abs() + du) + g.abs() * du + 2.0 ** -20 * y.abs()
    else:
        y = act64(act, z)
        dy = 1.13 * dz + 2.0 ** -20 * y.abs()
    if residual is not None:
        y = y + residual
    return y, dy + 2.0 ** -8 * (y.abs() + dy) + 1e-30


def close(got, want, tol):
    d = (got.double() - want).abs()
    assert bool((d <= tol).all()), f"{int((d > tol).sum())} of {d.numel()} outside, worst {float((d / tol).max()):.2f} tol"


def inputs(M, N, K, act, bias, residual, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + 31 * N + 977 * K)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    gated = act == "swiglu"
    return dict(x=r(M, K).bfloat16(), W=r(N, K, std=K ** -0.5).bfloat16(),
                W_up=r(N, K, std=K ** -0.5).bfloat16() if gated else None, bias=r(N) if bias else None,
                bias_up=r(N) if bias and gated else None, residual=r(M, N).bfloat16() if residual else None)


def wide(a):
    return {n: None if t is None else t.double() for n, t in a.items()}


def call(moe, a, act, stream=None, y=None):
    M, K = a["x"].shape
    N = a["W"].shape[0]
    room = torch.full((M * N + 64,), 123.0, dtype=torch.bfloat16, device="cuda")
    out = room[:M * N].view(M, N) if y is None else y
    moe.moe_linear(a["x"], a["W"], a["W_up"], a["bias"], a["bias_up"], a["residual"], M, N, K,
                   getattr(moe, "MOE_ACT_" + act.upper()), out, stream=stream)
    torch.cuda.synchronize()
    assert moe.moe_get_error() == 0
    assert (room[M * N:] == 123.0).all()                 # nothing written behind the last row
    return out


def check(moe, M, N, K, act="none", bias=False, residual=False):
    a = inputs(M, N, K, act, bias, residual)
    y, tol = define(act, **wide(a))
    close(call(moe, a, act), y, tol)


# ----------------------------------------------------------------------------- refusals (CPU)

def test_refusals(moe):
    L = moe.lib()
    def lin(M=8, N=64, K=64, act=0, x=16, W=32, up=None, b=None, bu=None, r=None, y=64):
        return L.moe_linear(x, W, up, b, bu, r, M, N, K, act, y, None)
    for kw in [dict(M=0), dict(N=0), dict(K=0), dict(M=-3), dict(K=60), dict(K=4), dict(M=(1 << 24) + 1),
               dict(N=(1 << 24) + 1), dict(K=1 << 25)]:
        assert lin(**kw) == -2, kw
    for kw in [dict(act=-1), dict(act=6), dict(x=None), dict(W=None), dict(y=None), dict(act=5), dict(up=48),
               dict(bu=48), dict(x=64), dict(W=64), dict(act=5, up=64)]:
        assert lin(**kw) == -1, kw
    for kw in [dict(x=8), dict(W=24), dict(y=72), dict(b=4), dict(r=2), dict(act=5, up=40), dict(act=5, up=48, bu=4)]:
        assert lin(**kw) == -3, kw
    def lin8(M=8, N=64, K=64, act=0, x=16, W=32, s=32, up=None, su=None, ws=128, nws=1 << 20):
        return L.moe_linear_w8a8(x, W, s, up, su, None, None, None, M, N, K, act, 64, ws, nws, None)
    assert lin8(K=8) == -2 and lin8(M=0) == -2
    assert lin8(s=None) == -1 and lin8(ws=None) == -1 and lin8(su=32) == -1 and lin8(act=5, up=48) == -1
    assert lin8(s=20) == -3 and lin8(ws=100) == -3
    assert lin8(nws=8 * 64) == -4
    assert moe.moe_linear_workspace_bytes(8, 64) == 512 + 32 and moe.moe_linear_workspace_bytes(3, 48) == 256 + 12
    for M, K in [(0, 64), (8, 40), (8, 0)]:
        with pytest.raises(moe.MoeError):
            moe.moe_linear_workspace_bytes(M, K)
    host = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cpu"):          # host tensors are refused before they reach a kernel
        moe.moe_linear(host, 16, None, None, None, None, 8, 64, 64, 0, 64, stream=0)
    with pytest.raises(ValueError, match="cpu"):
        moe.moe_linear_w8a8(16, host, 32, None, None, None, None, None, 8, 64, 64, 0, 64, 128, stream=0)


def test_overlapping_arrays_are_refused(moe):
    L = moe.lib()
    def lin(x, W, y, act=0, up=None, b=None, bu=None, r=None):
        return L.moe_linear(x, W, up, b, bu, r, 8, 64, 64, act, y, None)
    # 8 x 64 outputs are 1024 bytes at y, x as many, the weights 8192 (fp8: 4096), a bias or scales 256
    far = dict(x=1 << 20, W=2 << 20, y=3 << 20)
    top = far["y"] + 1024
    for kw in [dict(x=top - 16), dict(x=far["y"] - 1008), dict(W=top - 16), dict(W=far["y"] - 8176), dict(r=far["y"] + 128),
               dict(r=far["y"] - 128), dict(b=far["y"] - 240), dict(b=top - 16),
               dict(act=5, up=far["y"] - 16), dict(act=5, up=4 << 20, bu=far["y"])]:
        assert lin(**{**far, **kw}) == -1, kw
    def lin8_at(ws=5 << 20, x=1 << 20, W=2 << 20, s=6 << 20, y=3 << 20, r=None, b=None):
        return L.moe_linear_w8a8(x, W, s, None, None, b, None, r, 8, 64, 64, 0, y, ws, 1 << 20, None)
    for kw in [dict(ws=(1 << 20) + 512), dict(ws=(2 << 20) + 4080), dict(ws=6 << 20), dict(ws=(3 << 20) - 528),
               dict(ws=3 << 20), dict(r=5 << 20), dict(b=(5 << 20) + 512), dict(s=(3 << 20) + 1008), dict(r=(3 << 20) + 16)]:
        assert lin8_at(**kw) == -1, kw


def test_definition_gelu_forms_agree_with_their_formulas():
    z = torch.linspace(-9, 9, 101, dtype=torch.float64)
    ref = torch.tensor([v * 0.5 * (1 + math.erf(v / math.sqrt(2))) for v in z.tolist()], dtype=torch.float64)
    assert torch.allclose(act64("gelu", z), ref, atol=1e-13)
    tanh = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    assert torch.allclose(act64("gelu_tanh", z), tanh, atol=1e-13)


def test_warps_arrive_whole_at_aligned_barriers():
    # an .aligned barrier takes the lanes of a warp together, and a spinning wait lets them go one by one: the
    # statement in front of each such barrier brings them together, and no wait is taken lane by lane in front of it
    src = pathlib.Path(__file__).parent.parent / "moe_layer_router_b200" / "csrc" / "linear.cuh"
    code = [re.sub(r"//.*", "", line).strip() for line in src.read_text().splitlines()]
    code = [line for line in code if line]
    at = [i for i, line in enumerate(code) if re.search(r"\bnamed_barrier(_all)?\(", line)]
    assert len(at) == 2
    for i in at:
        assert code[i - 1] == "__syncwarp();", code[i - 1:i + 1]
    for line in code:       # an answer that is used is the warp's
        assert not re.search(r"(=|if \(|return) *!?mbar_wait\(", line), line


# ----------------------------------------------------------------------------- values (GPU)

@gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 128, 64), (2, 130, 72), (3, 7, 4096), (16, 128, 512), (17, 256, 136),
                                   (64, 4096, 2048), (100, 1001, 1384), (129, 640, 64), (255, 72, 1000),
                                   (256, 257, 256), (257, 512, 320), (300, 100, 8), (777, 1001, 1384)])
def test_sizes(moe, M, N, K):
    check(moe, M, N, K)
    check(moe, M, N, K, "swiglu", bias=True, residual=True)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_epilogues(moe, act, bias, residual):
    check(moe, 70, 200, 192, act, bias, residual)
    check(moe, 5, 33, 640, act, bias, residual)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (24, 2048, 7168), (512, 1536, 1024), (2048, 1000, 520),
                                   (4099, 2304, 256), (1500, 4104, 328)])
def test_larger(moe, M, N, K, act):
    check(moe, M, N, K, act, bias=True, residual=True)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_far_pre_activations(moe, act):
    # pre-activations out to +-60 and exactly 0: tails, saturation
    M, N, K = 64, 128, 64
    a = inputs(M, N, K, act, False, False)
    a["x"].zero_()
    a["x"][:, 0] = torch.linspace(-60, 60, M, device="cuda").bfloat16()
    a["W"].zero_()
    a["W"][:, 0] = 1
    a["bias"] = torch.linspace(-8, 8, N, device="cuda")
    y, tol = define(act, **wide(a))
    close(call(moe, a, act), y, tol)


@gpu
@pytest.mark.parametrize("act,lo,hi", [("silu", -90.0, -60.0), ("swiglu", -90.0, -60.0), ("gelu", -13.0, -8.0),
                                       ("gelu_tanh", -10.05, -7.0)])
@pytest.mark.parametrize("M,N,K", [(1, 400, 64), (40, 400, 64), (2100, 1000, 64), (2100, 1001, 64), (2100, 1000, 1032)])
def test_far_tails_keep_their_values(moe, M, N, K, act, lo, hi):
    # values down to 1e-38, all of them normal bf16.  The pre-activation is the bias, exact; an exponential of an argument
    # a is off by at most (2 + 1.2 |a|) 2^-23, forming the argument (two roundings, or three in the cubic) adds 3 |a|
    # 2^-23, |a| <= 90: (4 + 4.2 * 90) 2^-23 < 2^-14 with the divide; then one rounding to bf16
    a = inputs(M, N, K, act, True, False)
    a["x"].zero_()
    a["bias"] = torch.linspace(lo, hi, N, device="cuda")
    if act == "swiglu":
        a["bias_up"].fill_(1.0)
    want, _ = define(act, **wide({n: t[:1] if n == "x" else t for n, t in a.items()}))
    assert (want.abs() > 1.2e-38).all()
    y = call(moe, a, act)
    assert torch.equal(y, y[:1].expand_as(y))
    off = ((y[:1].double() - want) / want).abs()
    assert float(off.max()) <= 2.0 ** -8 + 2.0 ** -13


@gpu
@pytest.mark.parametrize("M,N,K", [(40, 200, 256), (2100, 1000, 256)])
def test_nan_and_infinity_stay_in_their_row(moe, M, N, K):
    a = inputs(M, N, K, "none", True, True)
    clean = call(moe, a, "relu").clone()
    a["x"][7, 3] = math.nan
    a["x"][M - 1, 5] = math.inf
    y = call(moe, a, "relu")
    same = torch.ones(M, dtype=torch.bool, device="cuda")
    same[7] = same[M - 1] = False
    assert torch.equal(y[same], clean[same])
    assert y[7].isnan().all()
    hit = a["W"][:, 5] > 0
    assert (y[M - 1][hit] == math.inf).all() and torch.equal(y[M - 1][~hit], a["residual"][M - 1][~hit])


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (2, 130, 72), (40, 200, 256), (2100, 1000, 256), (2100, 1001, 1032)])
def test_infinite_pre_activations(moe, M, N, K, act):
    # an infinity in x makes a whole row of them, of W's signs: what the definition gives for each
    a = inputs(M, N, K, act, True, True)
    a["x"][M - 1, 5] = math.inf
    want, _ = define(act, **wide({n: t[-1:] if n in ("x", "residual") and t is not None else t for n, t in a.items()}))
    assert not want.isfinite().any() or act == "relu"
    y = call(moe, a, act)
    torch.testing.assert_close(y[-1:].double(), want, rtol=2.0 ** -8, atol=0, equal_nan=True)
    if M > 1:
        assert y[:-1].isfinite().all()


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (40, 200, 256), (2100, 1000, 256), (2100, 1001, 1032)])
def test_sums_past_the_largest_fp32(moe, M, N, K, act):
    # 2e38 from the product and 3e38 from the bias: an infinity on its way to the activation; without the product, 3e38
    a = inputs(M, N, K, act, True, False)
    for n in ("x", "W", "W_up"):
        if a[n] is not None:
            a[n].zero_()
    a["x"][::3, 4] = 2e38
    a["W"][:, 4] = 1
    a["bias"].fill_(3e38)
    if act == "swiglu":
        a["bias_up"].fill_(0.5)
    y = call(moe, a, act)
    over = torch.zeros(M, dtype=torch.bool, device="cuda")
    over[::3] = True
    assert (y[over] == math.inf).all()
    want = torch.tensor(1.5e38 if act == "swiglu" else 3e38, device="cuda").bfloat16()
    assert (y[~over] == want).all()


@gpu
@pytest.mark.parametrize("N", [32768, 32771])
def test_offsets_past_32_bits(moe, N):
    # more than 2^31 outputs; a residual that repeats every 1000 rows, so the rows checked stand for all
    M, K = 66001, 64
    a = inputs(1000, N, K, "silu", True, True)
    rows = torch.arange(M, device="cuda") % 1000
    a["x"], a["residual"] = a["x"][rows], a["residual"][rows]
    y = call(moe, a, "silu")
    for m0 in (0, 65000, M - 300):
        part = dict(a, x=a["x"][m0:m0 + 300], residual=a["residual"][m0:m0 + 300])
        want, tol = define("silu", **wide(part))
        close(y[m0:m0 + 300], want, tol)
    for m0 in range(1000, M - 1000, 1000):
        assert torch.equal(y[m0:m0 + 1000], y[:1000])


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (33, 100, 512), (2048, 1024, 256), (2050, 1001, 256)])
def test_residual_in_place_and_repeatable(moe, M, N, K):
    a = inputs(M, N, K, "none", True, True)
    y = call(moe, a, "none")
    again = call(moe, a, "none")
    assert torch.equal(y, again)
    inplace = a["residual"].clone()
    moe.moe_linear(a["x"], a["W"], None, a["bias"], None, inplace, M, N, K, 0, inplace)
    assert torch.equal(inplace, y)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (40, 200, 256), (2100, 1000, 256)])
def test_arrays_side_by_side(moe, M, N, K):
    # y between its inputs, without a gap
    a = inputs(M, N, K, "silu", True, True)
    want = call(moe, a, "silu")
    parts = [a["x"], a["W"], torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), a["residual"]]
    arena = torch.cat([p.flatten() for p in parts])
    x, W, y, r = (v.view(p.shape) for v, p in zip(arena.split([p.numel() for p in parts]), parts))
    moe.moe_linear(x, W, None, a["bias"], None, r, M, N, K, moe.MOE_ACT_SILU, y)
    assert torch.equal(y, want)
    assert torch.equal(x, a["x"]) and torch.equal(W, a["W"]) and torch.equal(r, a["residual"])


@gpu
def test_transposed_tensors_are_refused(moe):
    a = inputs(16, 64, 64, "none", False, False)
    y = torch.zeros(64, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_linear(a["x"], a["W"], None, None, None, None, 16, 64, 64, 0, y.t())


@gpu
def test_other_stream_graph_and_two_calls_at_once(moe):
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    sets = [inputs(9, 1024, 2048, "silu", True, True, seed=i) for i in range(2)]
    want = [call(moe, a, "silu") for a in sets]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, o, s in zip(sets, outs, (s1, s2)):
            moe.moe_linear(a["x"], a["W"], None, a["bias"], None, a["residual"], 9, 1024, 2048, moe.MOE_ACT_SILU, o,
                           stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graph = torch.cuda.CUDAGraph()
    a = sets[0]
    with torch.cuda.graph(graph):
        moe.moe_linear(a["x"], a["W"], None, a["bias"], None, a["residual"], 9, 1024, 2048, moe.MOE_ACT_SILU, outs[0])
    for n in ("x", "W", "bias", "residual"):
        a[n].copy_(sets[1][n])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


@gpu
def test_captured_fork_and_join(moe):
    # two branches of a captured graph, each a chain of dependent calls, joined by a third
    M, d, f = 24, 512, 1024
    a, b = inputs(M, f, d, "silu", True, False), inputs(M, f, d, "swiglu", False, False, seed=1)
    c = inputs(M, d, f, "none", False, True)
    h, g, y = (torch.empty(M, n, dtype=torch.bfloat16, device="cuda") for n in (f, f, d))

    def first(stream=None):
        moe.moe_linear(a["x"], a["W"], None, a["bias"], None, None, M, f, d, moe.MOE_ACT_SILU, h, stream=stream)
        moe.moe_linear(h, c["W"], None, None, None, None, M, d, f, moe.MOE_ACT_NONE, y, stream=stream)

    def second(stream=None):
        moe.moe_linear(b["x"], b["W"], b["W_up"], None, None, None, M, f, d, moe.MOE_ACT_SWIGLU, g, stream=stream)

    def last():
        moe.moe_linear(g, c["W"], None, None, None, y, M, d, f, moe.MOE_ACT_NONE, y)

    first(), second(), last()
    torch.cuda.synchronize()
    want = y.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        second(side)
        first()
        main.wait_stream(side)
        last()
    for t in (h, g, y):
        t.zero_()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert moe.moe_get_error() == 0


# ----------------------------------------------------------------------------- fp8

def rows_to_e4m3(x):
    x = x.float()
    s = x.abs().amax(1)
    s = s / torch.full_like(s, 448)       # a true division: by a number, torch multiplies by its reciprocal
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def check8(moe, M, N, K, act="none", bias=False, residual=False, zero_row=False):
    a = inputs(M, N, K, act, bias, residual)
    if zero_row:
        a["x"][M // 2] = 0
    q = {"W_up": None}
    sc = {"W_up": None}
    for n in ("W", "W_up"):
        if a[n] is not None:
            q[n], sc[n] = rows_to_e4m3(a[n])
    xq, xs = rows_to_e4m3(a["x"])
    b = wide(a)
    b["x"] = xq.double() * xs.double()[:, None]
    for n in ("W", "W_up"):
        if a[n] is not None:
            b[n] = q[n].double() * sc[n].double()[:, None]
    y, tol = define(act, **b)
    room = torch.full((M * N + 64,), 123.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    u8 = lambda t: None if t is None else t.view(torch.uint8)
    moe.moe_linear_w8a8(a["x"], u8(q["W"]), sc["W"], u8(q["W_up"]), sc["W_up"], a["bias"], a["bias_up"], a["residual"],
                        M, N, K, getattr(moe, "MOE_ACT_" + act.upper()), room[:M * N], ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error() == 0
    assert (room[M * N:] == 123.0).all()
    assert torch.equal(ws[:M * K].view(M, K), xq.view(torch.uint8))       # the codes, bit for bit
    close(room[:M * N].view(M, N), y, tol)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 512, 2048), (2, 130, 144), (24, 2048, 7168), (100, 1001, 1392),
                                   (257, 512, 320), (777, 1001, 1392), (2048, 1000, 528), (1500, 4104, 336)])
def test_fp8_sizes(moe, M, N, K):
    check8(moe, M, N, K)
    check8(moe, M, N, K, "swiglu", bias=True, residual=True, zero_row=True)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_fp8_epilogues(moe, act):
    check8(moe, 70, 200, 192, act, True, True)
    check8(moe, 2048, 264, 256, act, False, True)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 200, 64), (40, 200, 64), (2100, 1000, 64), (2100, 1001, 1392)])
def test_fp8_sums_past_the_largest_fp32(moe, M, N, K, act):
    # as test_sums_past_the_largest_fp32; the row's code 448 times its scale is 2e38 within a rounding
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[::3, 4] = 2e38
    W = torch.zeros(N, K, device="cuda")
    W[:, 4] = 1
    Wq, one = W.to(torch.float8_e4m3fn).view(torch.uint8), torch.ones(N, device="cuda")
    gated = act == "swiglu"
    b, bu = torch.full((N,), 3e38, device="cuda"), torch.full((N,), 0.5, device="cuda") if gated else None
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    moe.moe_linear_w8a8(x, Wq, one, torch.zeros_like(Wq) if gated else None, one if gated else None, b, bu, None, M, N, K,
                        getattr(moe, "MOE_ACT_" + act.upper()), y, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error() == 0
    over = torch.zeros(M, dtype=torch.bool, device="cuda")
    over[::3] = True
    assert (y[over] == math.inf).all()
    assert (y[~over] == torch.tensor(1.5e38 if gated else 3e38, device="cuda").bfloat16()).all()


# ----------------------------------------------------------------------------- the kernel that a size runs on

def plan(M, N, K, f8, gated, residual=True, sms=148):
    """(kernel, tokens per tile, K slices, waves): plan_linear() of moe_api.cu again, so that what the sizes below reach
    is known."""
    if M <= 2 and not f8:
        return "rows", M, 1, 1
    nk = -(-K // (128 if f8 else 64))
    dram = ((2 if gated else 1) * N * K * (1 if f8 else 2) + M * K * (1 if f8 else 2) + M * N * (4 if residual else 2)) / 6.4e6
    found = []
    nt, bn = -(-N // (128 if gated else 256)), 256
    while bn >= 32:
        step = 16 if bn > 128 else 32
        if bn - step < M:
            waves, kb = -(-nt * -(-M // bn) // (sms // 2)), (128 * 128 + bn // 2 * 128) / 90e3
            us = 3.9 + max(waves * nk * kb, dram) + 0.2 * waves
            if N % 8:
                us = 3.9 + max(waves * max(nk * kb, 0.037 * bn), dram) + waves + 0.02 * bn
            found.append((us, "16 warps" if nk <= 10 else "8 warps", bn, 1, waves))
        bn -= step
    nt = -(-N // (64 if gated else 128))
    for want in (128, 64):
        mt = -(-M // want)
        bn = (-(-M // mt) + 15) // 16 * 16
        tiles = nt * -(-M // bn)
        for split in (1, 2, 4, 8):
            per = -(-tiles * split // sms)
            if split > nk or per > 2:
                break
            us = 3.9 + max(per * -(-nk // split) * (128 * 128 + 128 * bn) / 90e3, dram)
            us += 0.5 + 0.1 * split + 0.026 * bn if split > 1 else 0
            us += 0.1 * bn * per / split if N % 4 else 0
            found.append((us, "split", bn, split, 1))
    return min(found, key=lambda c: c[0])[1:]


LARGE = [(4099, 4104, 2064), (4099, 4101, 2064)]      # persistent pairs over several tiles, K long
LARGE_SHORT = [(4099, 4104, 528), (4099, 4101, 528)]  # and K short
SPLIT = [(3, 4096, 7168), (8, 7168, 4096), (128, 2048, 4096), (128, 4096, 4096), (256, 1000, 4096), (256, 2048, 7168),
         (256, 4096, 7168), (256, 1000, 2048), (40, 2050, 7168), (130, 2049, 4112), (33, 2052, 2064), (5, 100, 4096),
         (3, 2048, 4096), (3, 1000, 4096), (200, 300, 7168), (128, 2048, 7168),
         (256, 200, 7168)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("f8", [False, True])
def test_sizes_reach_every_kernel(f8, gated):
    for (M, N, K), warps in [(s, "8 warps") for s in LARGE] + [(s, "16 warps") for s in LARGE_SHORT]:
        kernel, bn, _, waves = plan(M, N, K, f8, gated)
        assert kernel == warps and bn > 96 and waves >= 3, (M, N, K, kernel, bn, waves)
        # whatever the estimate: more than two split CTAs per SM are not weighed, and K alone decides the warps
        assert -(-N // 128) * -(-M // 128) > 2 * 148 and (-(-K // (128 if f8 else 64)) > 10) == (warps == "8 warps")
    plans = [plan(*s, f8, gated) for s in SPLIT]
    for split in (2, 4, 8):       # up to 32 tokens per tile the partial sums have memory of their own
        for few in (True, False):
            assert any(p[0] == "split" and p[2] == split and (p[1] <= 32) == few for p in plans), (split, few, plans)


@gpu
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", LARGE + LARGE_SHORT)
def test_pairs_over_several_tiles(moe, M, N, K, act):
    check(moe, M, N, K, act, bias=True, residual=True)
    check8(moe, M, N, K, act, bias=True, residual=True, zero_row=True)


@gpu
@pytest.mark.parametrize("act", ["silu", "swiglu"])
@pytest.mark.parametrize("M,N,K", SPLIT)
def test_sums_cut_over_a_cluster(moe, M, N, K, act):
    check(moe, M, N, K, act, bias=True, residual=True)
    check8(moe, M, N, K, act, bias=True, residual=True, zero_row=True)


# ----------------------------------------------------------------------------- a block

@gpu
@pytest.mark.parametrize("T", [1, 40, 600])
def test_block_of_projection_routed_layer_and_dense_layer(moe, T):
    # as a block uses them: attention output -> projection into the residual stream -> scored router and
    # experts -> gated dense layer back into the residual stream, on one stream, captured and replayed
    d, E, k, f, da, fd = 256, 16, 4, 192, 320, 384
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s, n=1: (torch.randn(*s, generator=g, device="cuda") * n ** -0.5).bfloat16()
    attn, x0 = r(T, da), r(T, d)
    Wo, bo = r(d, da, n=da), torch.randn(d, generator=g, device="cuda") * 0.1
    Wg, W1, W3, W2 = r(E, d, n=d), r(E, f, d, n=d), r(E, f, d, n=d), r(E, d, f, n=f)
    G, U, D = r(fd, d, n=d), r(fd, d, n=d), r(d, fd, n=fd)
    bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2
    p = moe.moe_route_params(n_group=4, topk_group=2, scale=2.5)
    ws = torch.empty(moe.moe_workspace_bytes(T, d, E, k, f), dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    x1, m, h, y = bf(T, d), bf(T, d), bf(T, fd), bf(T, d)

    def block():
        moe.moe_linear(attn, Wo, None, bo, None, x0, T, d, da, moe.MOE_ACT_NONE, x1)
        moe.moe_layer_forward_scored(x1, Wg, bias, p, W1, W3, W2, None, None, None, 0, T, d, E, k, f, 1.0, 0, m, ws)
        moe.moe_linear(m, G, U, None, None, None, T, fd, d, moe.MOE_ACT_SWIGLU, h)
        moe.moe_linear(h, D, None, None, None, x1, T, d, fd, moe.MOE_ACT_NONE, y)

    block()
    torch.cuda.synchronize()
    first = y.clone()
    # each stage against 64 bits, from the stage's own inputs
    want, tol = define("none", attn.double(), Wo.double(), bias=bo.double(), residual=x0.double())
    close(x1, want, tol)
    L = moe.moe_workspace_layout(T, d, E, k, f, 0)
    idx = moe.workspace_view(ws, L, "idx", (T, k), torch.int32).long()
    w = moe.workspace_view(ws, L, "w", (T, k), torch.float32).double()
    s = torch.sigmoid(x1.double() @ Wg.double().T)
    np.testing.assert_allclose((2.5 * s.gather(1, idx) / s.gather(1, idx).sum(1, keepdim=True)).cpu().numpy(),
                               w.cpu().numpy(), rtol=1e-4)
    # the layer rounds h, each expert's y and the sum to bf16 (2^-8 of the value each); h's error reaches y
    # through |W2|, y's reaches the sum times its weight (the weights sum to 2.5, so a fixed bar would not do)
    ref, bar = (torch.zeros(T, d, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        he, dh = define("swiglu", x1[t].double(), W1[e].double(), W3[e].double())
        ye = he @ W2[e].double().T
        dy = (dh + (f / 16 + 12) * 2.0 ** -23 * he.abs()) @ W2[e].double().abs().T
        dy = dy + 2.0 ** -8 * (ye.abs() + dy)
        ref.index_add_(0, t, w[t, j][:, None] * ye)
        bar.index_add_(0, t, w[t, j][:, None] * (dy + k * 2.0 ** -23 * ye.abs()))
    close(m, ref, bar + 2.0 ** -8 * (ref.abs() + bar))
    want, tol = define("swiglu", m.double(), G.double(), U.double())
    close(h, want, tol)
    want, tol = define("none", h.double(), D.double(), residual=x1.double())
    close(y, want, tol)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first) and moe.moe_get_error() == 0
