"""The operators of a selective layer on the GPU against their fp64 oracle on
the same inputs, element by element.

Tolerances, derived from the arithmetic:
  a rounding to bf16 is off by at most 2^-8 of the value, to e4m3 by 2^-4 of it or
    by 2^-10 of the scale where it is below the smallest normal value;
  a fp32 sum of n products whose magnitudes add up to A is off by at most (n + 1)
    2^-24 A; on random signs by about sqrt(n) of that.  Convolution: n <= 9, 6e-7 A
    allowed.  Matrix product: groups of 128, whose accumulator on the tensor cores
    may cut off (2^-23 of a partial sum each time): sqrt(128 + groups) 2^-23 A =
    1.5e-6 A for K <= 4096, 4e-6 A allowed.  Norm: squares have one sign: at most 64
    per thread and 10 levels of joins, 75 2^-24 = 4.5e-6 of the sum, half of that
    for its root, and four roundings: 3e-6 of the value allowed;
  activations: fp32 by the formulas (1e-6 of the result, GELU 3e-7 of z), bf16 within 4e-4
    of the value before its rounding; their slope is at most 1.13.
"""
import numpy as np
import pytest

from oracle import layer

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _host(t):
    import torch
    return None if t is None else t.to(torch.float32).double().cpu().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def _offset(t, on=True):
    """The same values at an address that is a multiple of the element size only."""
    import torch
    if not on or t is None:
        return t
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    flat.copy_(t.reshape(-1))
    return flat.view(t.shape)


def _near(got, want, tol, what=""):
    """|got - want| <= tol, element by element."""
    got = _host(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    worst = np.abs(got - want) / np.maximum(tol, 1e-300)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values off, worst {np.nanmax(worst):.3g} of the tolerance"


def _act_tol(y, z_tol, act, dtype):
    """Tolerance of act(z) rounded to dtype, z off by z_tol."""
    if act == "none":
        return z_tol + HALF[dtype] * np.abs(y) + 1e-30
    own = 4e-4 * np.abs(y) if dtype == "bf16" else 1e-6 * np.abs(y) + 1e-6 * z_tol + 1e-30
    return 1.13 * z_tol + own + 3e-7 * (act == "gelu") * (np.abs(y) + 1) + HALF[dtype] * np.abs(y) + 1e-30


# ------------------------------------------------------------------ convolution
def _conv_case(B, T, C, K, dtype, extra=0, bias=True, cache=True, ragged=False, unaligned=False, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = _offset(n(B, T, C + extra).to(_dt(dtype)).cuda(), unaligned)[..., :C]
    t = dict(x=x, w=n(C, K).cuda() / K ** 0.5)
    if bias:
        t["bias"] = n(C).cuda()
    if cache:
        t["cache"] = n(B, K - 1, C).to(_dt(dtype)).cuda()
    if ragged:
        t["lens"] = torch.tensor([min(T, b) if b < 4 else (T * b) // max(1, B - 1) for b in range(B)], dtype=torch.int32).cuda()
    return t


def _conv_check(t, out, act, dtype):
    x, w, b, c = (_host(t.get(n)) for n in ("x", "w", "bias", "cache"))
    lens = None if t.get("lens") is None else t["lens"].cpu().numpy()
    y, keep = layer.short_conv(x, w, b, c, lens, act)
    mag, _ = layer.short_conv(np.abs(x), np.abs(w), None if b is None else np.abs(b), None if c is None else np.abs(c), lens)
    _near(out["y"], y, _act_tol(y, 6e-7 * mag, act, dtype), "y")
    np.testing.assert_array_equal(_host(out["cache"]), keep)


CONV = [(1, 1, 8, 4), (3, 1, 24, 4), (2, 2, 40, 4), (3, 3, 7, 4), (2, 16, 64, 3), (2, 17, 64, 8), (5, 40, 33, 2), (1, 300, 16, 5),
        (2, 70, 520, 1), (2, 70, 264, 6), (1, 129, 96, 7)]


@pytest.mark.parametrize("case", CONV, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_conv_parity(gpu_lib, case, dtype, act):
    from test_learned_neural_gb300.runner import ShortConv
    B, T, C, K = case
    t = _conv_case(B, T, C, K, dtype, bias=T % 2 == 0, cache=T % 3 != 0)
    _conv_check(t, ShortConv(C, K, act, dtype).forward(t), act, dtype)


@pytest.mark.parametrize("T", [1, 2, 5, 33, 100])
@pytest.mark.parametrize("dtype,C,extra,unaligned", [("bf16", 32, 0, False), ("bf16", 32, 8, False), ("bf16", 32, 3, False),
                                                     ("bf16", 31, 1, False), ("f32", 12, 4, False), ("f32", 12, 0, True),
                                                     ("bf16", 32, 0, True)])
def test_conv_ragged_strided_in_place(gpu_lib, T, dtype, C, extra, unaligned):
    """Lengths 0, 1, 2, 3, .. T; rows inside wider ones; the cache continued in
    place; what lies past a length or between the rows is never used."""
    from test_learned_neural_gb300.runner import ShortConv
    t = _conv_case(7, T, C, 4, dtype, extra, ragged=True, unaligned=unaligned)
    live = t["lens"].cpu().numpy()
    for b in range(7):
        t["x"][b, int(live[b]):] = float("nan")
    if extra:
        t["x"].as_strided((7, T, extra), t["x"].stride(), t["x"].storage_offset() + C).fill_(float("nan"))
    ref = {n: a.clone() for n, a in t.items()}
    op = ShortConv(C, 4, "silu", dtype)
    out = op.alloc_outputs(7, T, "cuda")
    out["y"].fill_(7)
    out["cache"].copy_(t["cache"])
    t["cache"] = out["cache"]
    op.forward(t, out=out)
    _conv_check(ref, out, "silu", dtype)


@pytest.mark.parametrize("cuts", [(1,) * 7, (3, 1, 2, 1), (2, 5), (6, 1)])
def test_conv_calls_continue_one_another(gpu_lib, cuts):
    """A sequence cut anywhere gives the same bits."""
    import torch
    from test_learned_neural_gb300.runner import ShortConv
    t = _conv_case(2, 7, 40, 4, "bf16")
    op = ShortConv(40, 4)
    whole = op.forward(t)
    at, cache, ys = 0, t["cache"].clone(), []
    for n in cuts:
        out = op.forward({**t, "x": t["x"][:, at:at + n].contiguous(), "cache": cache})
        cache, at = out["cache"], at + n
        ys.append(out["y"])
    assert torch.equal(torch.cat(ys, 1), whole["y"]) and torch.equal(cache, whole["cache"])


def test_conv_non_finite_values_reach_their_own_outputs(gpu_lib):
    import torch
    from test_learned_neural_gb300.runner import ShortConv
    t = _conv_case(2, 50, 16, 3, "bf16", cache=False)
    clean = ShortConv(16, 3).forward(t)["y"].clone()
    t["x"][1, 20, 5] = float("inf")
    t["x"][0, 49, 2] = float("nan")
    y = ShortConv(16, 3).forward(t)["y"]
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 20:23, 5] = True
    hit[0, 49, 2] = True
    assert torch.equal(y[~hit], clean[~hit]) and not torch.equal(y[hit], clean[hit])
    assert torch.isnan(y[0, 49, 2])


# ---------------------------------------------------------------------- norm
def _rms_case(M, C, x="bf16", r="bf16", affine=True, unaligned=False, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    t = dict(x=_offset(torch.randn(M, C, generator=g).to(_dt(x)).cuda(), unaligned))
    if r:
        t["residual"] = _offset((3 * torch.randn(M, C, generator=g)).to(_dt(r)).cuda(), unaligned)
    if affine:
        t["weight"] = _offset(1 + 0.3 * torch.randn(C, generator=g).cuda(), unaligned)
    return t


def _rms_check(t, out, x, r, y, block, eps=1e-6):
    want, h = layer.rms_norm(_host(t["x"]), _host(t.get("residual")), _host(t.get("weight")), eps)
    if r:
        _near(out["h"], h, (HALF[r] + 2.0 ** -24) * np.abs(h) + 1e-30, "h")
    else:
        assert "h" not in out
    if y != "e4m3":
        _near(out["y"], want, (3e-6 + HALF[y]) * np.abs(want) + 1e-30, "y")
        return
    scale = layer.e4m3_scales(want, block)
    _near(out["scale"], scale, 4e-6 * scale, "scale")
    wide = np.repeat(_host(out["scale"]), block or want.shape[1], axis=1)[:, :want.shape[1]]
    got = out["y"].float().double().cpu().numpy() * wide
    assert (np.abs(got - want) <= (2.0 ** -4 + 1e-5) * np.abs(want) + (2.0 ** -10 + 1e-5) * wide).all()


@pytest.mark.parametrize("M,C", [(1, 8), (5, 64), (3, 1), (9, 77), (4, 256), (7, 504), (2, 1024), (6, 2048), (3, 2056), (2, 4096),
                                 (3, 5000), (2, 8192), (1, 16384), (2, 32768), (1, 32767), (2, 13001)], ids=str)
@pytest.mark.parametrize("y,block", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 128)])
def test_rms_parity(gpu_lib, M, C, y, block):
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(M, C)
    out = RmsNorm(C, x_dtype="bf16", y_dtype=y, block=block).forward(t)
    _rms_check(t, out, "bf16", "bf16", y, block)


@pytest.mark.parametrize("x,r,y", [("bf16", "f32", "bf16"), ("f32", "bf16", "e4m3"), ("f32", "f32", "f32"), ("f32", None, "bf16"),
                                   ("bf16", None, "e4m3")])
@pytest.mark.parametrize("C,unaligned", [(512, False), (512, True), (70, False), (3000, False)])
def test_rms_types_and_alignment(gpu_lib, x, r, y, C, unaligned):
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(11, C, x, r, affine=C != 70, unaligned=unaligned)
    block = 128 if y == "e4m3" else 0
    out = RmsNorm(C, x_dtype=x, y_dtype=y, residual_dtype=r, block=block, eps=1e-3).forward(t)
    _rms_check(t, out, x, r, y, block, eps=1e-3)


@pytest.mark.parametrize("C", [96, 2048, 4096, 333])
def test_rms_in_place(gpu_lib, C):
    """h over the residual and y over x: the same bits."""
    import torch
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(9, C)
    op = RmsNorm(C)
    ref = op.forward(t)
    op.forward(t, out=dict(y=t["x"], h=t["residual"]))
    assert torch.equal(t["x"], ref["y"]) and torch.equal(t["residual"], ref["h"])


@pytest.mark.parametrize("C", [512, 515, 2560])
@pytest.mark.parametrize("block", [0, 128])
def test_rms_extreme_rows(gpu_lib, C, block):
    """Zeros, the smallest values, very large ones, a NaN, an infinity: their own rows only."""
    import torch
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(7, C, x="f32", r=None)
    x = t["x"]
    x[1] = 0.0
    x[2] *= 1e-38
    x[3] *= 1e17
    x[4, 5] = float("nan")
    x[5, 7] = float("inf")
    out = RmsNorm(C, x_dtype="f32", y_dtype="e4m3", block=block).forward(t)
    y, s = out["y"].float(), out["scale"]
    sub = {n: a[[0, 1, 2, 3, 6]] if n != "weight" else a for n, a in t.items()}
    keep = dict(y=out["y"].view(torch.uint8)[[0, 1, 2, 3, 6]].view(torch.float8_e4m3fn), scale=s[[0, 1, 2, 3, 6]])
    _rms_check(sub, keep, "f32", None, "e4m3", block)
    assert not y[1].any() and (s[1] > 0).all()
    assert torch.isnan(y[4]).all() and torch.isnan(s[4]).all()
    assert torch.isnan(y[5, 7]) and (torch.isnan(y[5]).all() if block == 0 else not y[5, 200:].any())


# ------------------------------------------------------------ 4-bit product
def _q4_case(M, K, N, group=128, zeros=False, x="bf16", x_block=0, bias=True, residual=None, unaligned=False, seed=0):
    """Codes, scales and zero points of the whole range, not those of a quantisation."""
    import torch
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    w = dict(q=torch.randint(0, 256, ((K + 1) // 2, N), generator=g, dtype=torch.uint8).cuda(),
             scales=(0.1 * torch.exp(torch.randn(G, N, generator=g)) / K ** 0.5).bfloat16().cuda(),
             zeros=torch.randint(0, 16, (G, N), generator=g, dtype=torch.uint8).cuda() if zeros else None)
    v = torch.randn(M, K, generator=g)
    t = {}
    if x == "e4m3":
        b = x_block or K
        t["x_scale"] = torch.exp(torch.randn(M, -(-K // b), generator=g)).cuda()
        v = 100 * v
    t["x"] = _offset(v.to(_dt(x)).cuda(), unaligned)
    if bias:
        t["bias"] = torch.randn(N, generator=g).cuda()
    if residual:
        t["residual"] = torch.randn(M, N, generator=g).to(_dt(residual)).cuda()
    return w, t


def _q4_check(w, t, y, K, group, act, x_block, out):
    W = layer.quant_weights(w["q"].cpu().numpy(), _host(w["scales"]), None if w["zeros"] is None else w["zeros"].cpu().numpy(),
                            K, group)
    x, xs, b, r = _host(t["x"]), _host(t.get("x_scale")), _host(t.get("bias")), _host(t.get("residual"))
    z = layer.quant_linear(x, W, xs, x_block, b)
    mag = layer.quant_linear(np.abs(x), np.abs(W), xs, x_block, None if b is None else np.abs(b))
    a = layer._act(z, act)
    tol = _act_tol(a, 4e-6 * mag, act, "f32" if out == "f32" else "bf16")
    want = a if r is None else a + r
    if r is not None:
        tol = tol + HALF[out] * (np.abs(want) + tol)
    _near(y, want, tol, "y")


Q4 = [(1, 64, 16), (1, 128, 64), (3, 200, 40), (8, 512, 96), (9, 96, 16), (16, 1024, 128), (17, 320, 33), (32, 256, 48), (33, 64, 64),
      (64, 640, 32), (65, 192, 40), (130, 256, 24), (1, 1, 1), (2, 33, 7), (5, 4096, 17), (1, 2048, 520)]


@pytest.mark.parametrize("case", Q4, ids=str)
@pytest.mark.parametrize("x,x_block,out", [("bf16", 0, "bf16"), ("bf16", 0, "f32"), ("f32", 0, "f32"), ("e4m3", 128, "bf16"),
                                           ("e4m3", 0, "f32")])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_parity(gpu_lib, case, x, x_block, out, group):
    from test_learned_neural_gb300.runner import QuantLinear
    M, K, N = case
    zeros = (K // group) % 2 == 1
    w, t = _q4_case(M, K, N, group, zeros, x, x_block)
    op = QuantLinear(K, N, group, zeros, "none", x, x_block, out)
    t["W"] = op.pack(**w)
    _q4_check(w, t, op.forward(t)["y"], K, group, "none", x_block, out)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 20])
def test_q4_epilogue(gpu_lib, act, out, M):
    """Activation, then the residual, in place of y too."""
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    w, t = _q4_case(M, 320, 72, residual=out)
    op = QuantLinear(320, 72, act=act, out_dtype=out)
    t["W"] = op.pack(w["q"], w["scales"])
    y = op.forward(t)["y"]
    _q4_check(w, t, y, 320, 128, act, 0, out)
    op.forward(t, out=dict(y=t["residual"]))
    assert torch.equal(t["residual"], y)


@pytest.mark.parametrize("x,K", [("bf16", 328), ("bf16", 331), ("e4m3", 328), ("e4m3", 331), ("f32", 331)])
@pytest.mark.parametrize("M", [2, 40])
def test_q4_unaligned_rows(gpu_lib, x, K, M):
    from test_learned_neural_gb300.runner import QuantLinear
    w, t = _q4_case(M, K, 50, 64, True, x, 0, unaligned=True)
    op = QuantLinear(K, 50, 64, True, "none", x, 0, "f32")
    t["W"] = op.pack(**w)
    _q4_check(w, t, op.forward(t)["y"], K, 64, "none", 0, "f32")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,group", [(256, 128), (100, 32), (33, 64), (1, 32)])
def test_q4_quantize(gpu_lib, zeros, dtype, K, group):
    """Every weight within half a step of its own (the scale's rounding to bf16
    moves the ends of the range by 2^-8 of 15 steps); a group of zeros is exact."""
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    g = torch.Generator().manual_seed(3)
    W = torch.randn(K, 20, generator=g)
    W[:, 3] = 0.0
    W[:, 4] = W[:, 4].abs() + 1
    W = W.to(_dt(dtype)).cuda()
    op = QuantLinear(K, 20, group, zeros)
    w = op.quantize(W)
    assert (w["zeros"] is not None) == zeros
    got = layer.quant_weights(w["q"].cpu().numpy(), _host(w["scales"]), w["zeros"].cpu().numpy() if zeros else None, K, group)
    want, step = _host(W), np.repeat(_host(w["scales"]), group, axis=0)[:K]
    # with zero points the rounded one shifts the range by up to half a step as well
    assert (np.abs(got - want) <= ((1.0 if zeros else 0.5) + 15 * 2.0 ** -8) * step + 1e-7).all()
    inner = np.abs(want) <= 6.4 * step
    if not zeros:
        assert (np.abs(got - want)[inner] <= 0.5001 * step[inner]).all()
    assert not got[:, 3].any()


def test_q4_non_finite_values_stay_in_their_row_and_column(gpu_lib):
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    for x in ("bf16", "f32"):
        w, t = _q4_case(20, 300, 40, x=x)
        op = QuantLinear(300, 40, x_dtype=x)
        t["W"] = op.pack(w["q"], w["scales"])
        clean = op.forward(t)["y"].clone()
        t["x"][3, 70], t["x"][11, 299] = float("nan"), float("inf")
        w["scales"][1, 9] = float("nan")
        t["W"] = op.pack(w["q"], w["scales"])
        y = op.forward(t)["y"]
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[3], hit[11], hit[:, 9] = True, True, True
        assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()


# ------------------------------------------------------------------- together
def _rows_ops():
    import torch
    from test_learned_neural_gb300.runner import QuantLinear, RmsNorm, ShortConv
    w, t = _q4_case(6, 200, 64, x="f32", bias=False)
    lin = QuantLinear(200, 64, x_dtype="f32")
    t["W"] = lin.pack(w["q"], w["scales"])
    return [(lin, t, (6,)), (RmsNorm(256, y_dtype="e4m3", block=128), _rms_case(6, 256), (6,)),
            (ShortConv(48, 4), _conv_case(3, 20, 48, 4, "bf16"), (3, 20))], torch


def test_repeated_streamed_and_captured_calls_give_the_same_bits(gpu_lib):
    ops, torch = _rows_ops()
    bits = lambda o: {n: a.view(torch.uint8).clone() for n, a in o.items()}  # noqa: E731
    for op, t, size in ops:
        ref = bits(op.forward(t))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = op.forward(t)
        side.synchronize()
        out = op.alloc_outputs(*size, "cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.forward(t, out=out)
        for a in out.values():
            a.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, a in ref.items():
            assert torch.equal(a, bits(other)[n]) and torch.equal(a, bits(out)[n]), n


def test_graph_behind_a_larger_call(gpu_lib):
    """A captured call's copy of x survives a later call that needs a larger one."""
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    w, t = _q4_case(2, 200, 64, x="f32")
    op = QuantLinear(200, 64, x_dtype="f32")
    W = op.pack(w["q"], w["scales"])
    t["W"] = W
    out, graph = op.alloc_outputs(2, "cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(t, out=out)
    graph.replay()
    torch.cuda.synchronize()
    ref = out["y"].clone()
    _, big = _q4_case(60, 200, 64, x="f32")
    op.forward({**big, "W": W})
    out["y"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["y"], ref)
    _q4_check(w, t, out["y"], 200, 128, "none", 0, "f32")


@pytest.mark.parametrize("C", [512, 515, 2560, 16384])
@pytest.mark.parametrize("y", ["f32", "e4m3"])
def test_rms_rows_whose_squares_leave_the_range(gpu_lib, C, y):
    """Values to the largest of fp32, beside ordinary rows: the sum of squares does not overflow."""
    import torch
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(6, C, x="f32", r=None)
    x = t["x"]
    x[1] *= 1e18
    x[2] *= 3e30
    x[3, 3] = 3e38
    x[4, C - 1] = -2e19
    block = 128 if y == "e4m3" else 0
    _rms_check(t, RmsNorm(C, x_dtype="f32", y_dtype=y, block=block).forward(t), "f32", None, y, block)


@pytest.mark.parametrize("C", [96, 2048, 333])
def test_rms_sum_in_place_of_x(gpu_lib, C):
    """h written over x, the residual left alone."""
    import torch
    from test_learned_neural_gb300.runner import RmsNorm
    t = _rms_case(7, C, x="bf16", r="bf16")
    op = RmsNorm(C)
    ref = {n: a.clone() for n, a in op.forward(t).items()}
    kept = t["residual"].clone()
    out = op.forward(t, out=dict(y=torch.empty_like(ref["y"]), h=t["x"]))
    assert torch.equal(out["y"], ref["y"]) and torch.equal(t["x"], ref["h"]) and torch.equal(t["residual"], kept)


def test_products_of_two_handles_on_two_streams_at_once(gpu_lib):
    """Each with its own fragments of x in its own workspace."""
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    calls = []
    for K, N, M in ((1024, 512, 40), (768, 1024, 33)):
        op = QuantLinear(K, N, 64)
        g = torch.Generator().manual_seed(K)
        W = op.quantize((torch.randn(K, N, generator=g) / K ** 0.5).cuda())
        t = dict(x=torch.randn(M, K, generator=g).bfloat16().cuda(), W=op.pack(**W))
        calls.append((op, t, op.forward(t)["y"].clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (op, t, _, st) in enumerate(calls):
            with torch.cuda.stream(st):
                outs[i].append(op.forward(t)["y"])
    torch.cuda.synchronize()
    for (op, _, ref, _), many in zip(calls, outs):
        op.status()
        assert all(torch.equal(y, ref) for y in many)


@pytest.mark.parametrize("B,T,C,K,dtype,extra", [(2, 1501, 2048, 4, "bf16", 8), (3, 777, 2560, 4, "f32", 4), (5, 2000, 1024, 8, "bf16", 0),
                                                 (4, 1200, 2048, 2, "bf16", 0), (7, 900, 1024, 7, "f32", 0), (2, 3001, 2048, 1, "bf16", 0)])
def test_conv_long_runs(gpu_lib, B, T, C, K, dtype, extra):
    """Sizes whose rows go through the ring of copies: runs that end inside a group, ragged lengths (0, 1, 2, .. T), the cache
    continued in place, NaN behind a length."""
    import torch
    from test_learned_neural_gb300.runner import ShortConv
    t = _conv_case(B, T, C, K, dtype, extra, ragged=True)
    for b, n in enumerate(t["lens"].tolist()):
        t["x"][b, n:] = float("nan")
    t["lens"][-1] = T - 5
    t["x"][-1] = 0.5
    ref = {n: a.clone() for n, a in t.items()}
    op = ShortConv(C, K, "silu", dtype)
    out = op.alloc_outputs(B, T, "cuda")
    out["cache"].copy_(t["cache"])
    t["cache"] = out["cache"]
    op.forward(t, out=out)
    _conv_check(ref, out, "silu", dtype)
