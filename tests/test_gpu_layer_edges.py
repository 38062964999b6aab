"""Cases of the layer operators where they can go wrong: results against the
fp64 oracle at sizes that take each kernel variant, element by element where a
bound on the largest value would hide an error, and the handles' workspaces."""
import numpy as np
import pytest

from oracle import layer
from tests.gpu_common import maxrel
from tests.test_gpu_layer import TOL, TOL_DECAY, _decay_inputs, _decay_ref, _dt, _host

pytestmark = pytest.mark.gpu


def _rms(a):
    return float(np.sqrt(np.mean(np.square(np.asarray(a, np.float64)))))


def _bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16).double().numpy()


# --------------------------------------------------------- decay attention
@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (48, 40), (96, 128)], ids=str)
@pytest.mark.parametrize("B,T", [(2, 600), (160, 140)])
def test_decay_bf16_readouts_carry_only_their_own_rounding(gpu_lib, dims, B, T):
    """Scores and states enter the read-outs' products with 16 bits or more: 2^-16
    of a term, 1/256 of the read-out's rounding of 2^-8.  The two add as squares
    (1 + 2^-16, and a few results rounded to the other side), so the distance
    from the exact read-outs is that of the rounded exact ones to 2 %."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    (dk, dv), H = dims, 2
    t = _decay_inputs(B, H, T, dk, dv, "bf16", 1, "heads", False, True, seed=21, gammas=[0.999, 0.97])
    op = DecayAttention(H, dk, dv)
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    assert op.last_path() == 2
    rows = min(B, 4)
    y, _ = _decay_ref({n: v if n == "decay" else v[:rows] for n, v in t.items()}, "heads", "heads")
    ours, rounding = _rms(_host(out["y"][:rows]) - y), _rms(_bf16(y) - y)
    print(f"{ours:.3e} rounding {rounding:.3e}")
    assert ours <= 1.02 * rounding


# ------------------------------------------------------------- activations
def _check_tails(y, z, act):
    """bf16 results of act(z), element by element, so that the tail counts: the
    formulas are within 4e-4 of the value (GELU to z = -12; SiLU's exponent,
    rounded to 2^-24 of 115 at z = -80, within 6e-6), and rounding is monotone, so
    a result lies between the rounded ends of that interval."""
    import math
    z = z.double().numpy()
    want = z * 0.5 * np.vectorize(math.erfc)(-z / math.sqrt(2.0)) if act == "gelu" else z / (1.0 + np.exp(-z))
    lo, hi = _bf16(want - 4e-4 * np.abs(want)), _bf16(want + 4e-4 * np.abs(want))
    bad = (y < lo) | (y > hi)
    at = np.argwhere(bad)
    assert not bad.any(), [(z[i[-1]], y[tuple(i)], want[i[-1]]) for i in at[:3]]


@pytest.mark.parametrize("act,lo", [("gelu", -12.0), ("silu", -80.0)])
@pytest.mark.parametrize("M", [1, 3, 40])
def test_linear_activation_tails(gpu_lib, act, lo, M):
    """z is the bias itself (x is zero)."""
    import torch
    from test_learned_neural_gb300.runner import Linear
    N = 4096
    z = torch.linspace(lo, 6.0, N)
    op = Linear(16, N, act)
    y = op.forward(dict(x=torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda"),
                        W=torch.ones(16, N, dtype=torch.bfloat16, device="cuda"), bias=z.cuda()))["y"]
    torch.cuda.synchronize()
    op.status()
    _check_tails(_host(y), z, act)


@pytest.mark.parametrize("act,lo", [("gelu", -12.0), ("silu", -80.0)])
@pytest.mark.parametrize("S", [1, 200])
def test_norm_activation_tails(gpu_lib, act, lo, S):
    """The same behind the norm: x is zero, so z is the bias."""
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    C = 4096
    z = torch.linspace(lo, 6.0, C)
    op = GroupNorm(C, C // 64, act, x_dtype="f32", y_dtype="bf16")
    y = op.forward(dict(x=torch.zeros(2, S, C, device="cuda"), bias=z.cuda()))["y"]
    torch.cuda.synchronize()
    _check_tails(_host(y).reshape(-1, C), z, act)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M", [2, 40])
def test_linear_activation_of_non_finite_values(gpu_lib, act, M):
    """act(inf) = inf; NaN stays NaN; -inf gives NaN as the formulas do (-inf * 0)."""
    import torch
    from test_learned_neural_gb300.runner import Linear
    z = torch.tensor([float("inf"), float("nan"), float("-inf"), 3e38, -3e38, 0.0, 1.0, -1.0])
    op = Linear(16, 8, act)
    y = _host(op.forward(dict(x=torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda"),
                              W=torch.ones(16, 8, dtype=torch.bfloat16, device="cuda"), bias=z.cuda()))["y"])
    op.status()
    assert np.isposinf(y[:, 0]).all() and np.isnan(y[:, 1:3]).all()
    assert (y[:, 3] > 2.9e38).all() and np.isfinite(y[:, 3]).all() and (y[:, 4] == 0).all() and (y[:, 5] == 0).all()


# ---------------------------------------------------------- matrix product
def _linear_check(M, K, N, act, in_dtype, out_dtype, bias, residual, inplace=False):
    import torch
    from test_learned_neural_gb300.runner import Linear
    g = torch.Generator().manual_seed(31)
    x = torch.randn(M, K, generator=g).to(_dt(in_dtype)).cuda()
    W = (torch.randn(K, N, generator=g) / K ** 0.5).to(_dt(in_dtype)).cuda()
    b = torch.randn(N, generator=g).cuda() if bias else None
    r = torch.randn(M, N, generator=g).to(_dt(out_dtype)).cuda() if residual else None
    ref = layer.linear(_host(x), _host(W), _host(b), _host(r), act)
    op = Linear(K, N, act, in_dtype, out_dtype)
    y = op.forward(dict(x=x, W=W, bias=b, residual=r), out=dict(y=r) if inplace else None)["y"]
    torch.cuda.synchronize()
    op.status()
    err = maxrel(_host(y), ref)
    print(f"path {op.last_path()} {err:.2e}")
    assert err <= TOL[out_dtype], err


# few rows; one pass of 256 of K, exactly two, three and a rest; a row length off 16 bytes; one tile per pair and
# several, narrow and wide; K split over the idle blocks
F32_TO_BF16 = [
    (3, 517, 264), (40, 100, 72), (40, 256, 136), (300, 512, 768), (300, 700, 1031), (1999, 517, 1031), (700, 2100, 1160),
    (4200, 520, 1300), (4200, 600, 2048), (40, 8192, 136), (128, 4096, 256),
]


@pytest.mark.parametrize("case", F32_TO_BF16, ids=str)
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True)])
def test_linear_fp32_to_bf16(gpu_lib, case, act, bias, residual):
    _linear_check(*case, act, "f32", "bf16", bias, residual)


@pytest.mark.parametrize("T", [1, 7, 300, 2000])
@pytest.mark.parametrize("dims", [(64, 64), (200, 65)], ids=str)
def test_decay_fp32_to_bf16(gpu_lib, T, dims):
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    dk, dv = dims
    t = _decay_inputs(2, 2, T, dk, dv, "f32", 1, "heads", False, True, seed=22)
    op = DecayAttention(2, dk, dv, qkv_dtype="f32", y_dtype="bf16")
    out = op.forward(t)
    torch.cuda.synchronize()
    y, S = _decay_ref(t, "heads", "heads")
    assert maxrel(_host(out["y"]), y) <= TOL["bf16"] and maxrel(_host(out["S"]), S) <= TOL_DECAY["f32"]


# -------------------------------------------------------------- group norm
def _norm_check(N, S, C, G, x_dtype, act="none", y_dtype=None, rows=None):
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    y_dtype = y_dtype or x_dtype
    g = torch.Generator().manual_seed(41)
    x = (torch.randn(N, S, C, generator=g) * 1.5 + 0.3).to(_dt(x_dtype)).cuda()
    w, b = (1 + 0.2 * torch.randn(C, generator=g)).cuda(), (0.2 * torch.randn(C, generator=g)).cuda()
    y = GroupNorm(C, G, act, x_dtype=x_dtype, y_dtype=y_dtype).forward(dict(x=x, weight=w, bias=b))["y"]
    torch.cuda.synchronize()
    pick = slice(None) if rows is None else rows
    err = maxrel(_host(y[pick]), layer.group_norm(_host(x[pick]), G, _host(w), _host(b), act))
    print(f"{err:.2e}")
    assert err <= TOL[y_dtype], err


# the one-read tile kernel around 48 KB of shared memory in all, and at its own limit of 48 KB of samples (then two passes)
@pytest.mark.parametrize("x_dtype,S", [("f32", S) for S in (42, 43, 44, 45, 48, 49)] +
                         [("bf16", S) for S in (86, 87, 90, 96, 97)])
def test_norm_tiles_at_the_shared_memory_limits(gpu_lib, x_dtype, S):
    _norm_check(200, S, 255, 3, x_dtype, rows=slice(0, 200, 40))


# ------------------------------------------------------ graphs and workspaces
def _ops():
    """(name, handle, a call of a size on fixed tensors): each call needs a workspace."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention, GroupNorm, Linear

    def decay(op, size, seed):
        t = _decay_inputs(1, 2, 300 * size, 64, 64, "bf16", 1, "heads", False, True, seed=seed)
        out = op.alloc_outputs(1, 300 * size, "cuda")
        return lambda: op.forward(t, out=out), [out["y"], out["S"]]

    def norm(op, size, seed):
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(1, 700 * size, 66, generator=g).cuda()
        out = op.alloc_outputs(1, 700 * size, "cuda")
        return lambda: op.forward(dict(x=x), out=out), [out["y"]]

    def linear(op, size, seed):
        g = torch.Generator().manual_seed(seed)
        x, W = torch.randn(50 * size, 600, generator=g).cuda(), torch.randn(600, 200, generator=g).cuda()
        out = op.alloc_outputs(50 * size, "cuda")
        return lambda: op.forward(dict(x=x, W=W), out=out), [out["y"]]

    return {"decay": (lambda: DecayAttention(2, 64, 64), decay), "norm": (lambda: GroupNorm(66, 6, x_dtype="f32"), norm),
            "linear": (lambda: Linear(600, 200, "none", "f32"), linear)}


@pytest.mark.parametrize("warm", [True, False], ids=["after_a_call", "first_call_captured"])
@pytest.mark.parametrize("name", ["decay", "norm", "linear"])
def test_graph_survives_a_larger_call(gpu_lib, name, warm):
    """A graph of a small size, then calls of larger sizes on the same handle (and
    others on another one, which take the memory that is free): its replays still
    give the direct call's bits, in any order with captures of the larger sizes."""
    import torch
    make, call = _ops()[name]
    op, other = make(), make()
    cases = [call(op, size, seed=size) for size in (1, 4, 9)]
    want = []
    for size, (run, outs) in zip((1, 4, 9), cases):
        ref = make()                         # a handle of its own: the captured one has not seen the size
        direct, o = call(ref, size, seed=size)
        direct()
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
    graphs = []
    for run, _ in cases:
        if warm:
            run()
            torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
        call(other, 4, seed=77)[0]()
    for k in (0, 2, 1, 0):
        for t in cases[k][1]:
            t.zero_()
        call(other, 9, seed=78)[0]()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cases[k][1], want[k])), k
    if name != "norm":
        op.status()


@pytest.mark.parametrize("C,G,S,layout", [(48, 1, 1, "channels_last"), (510, 6, 1, "channels_last"), (2000, 2, 1, "channels_last"),
                                          (96, 2, 200, "heads"), (85, 1, 7, "heads"), (96, 2, 200, "channels_last"),
                                          (85, 1, 600, "channels_last")])
@pytest.mark.parametrize("value", [1000.3, -77777.0])
def test_norm_of_a_large_common_offset(gpu_lib, C, G, S, layout, value):
    """A set of one value has variance 0: y is the bias, though 1 / sqrt(eps) = 316
    stands before every error of the mean.  The rounded mean is off by up to a few
    units in the last place of the value (0.03 at 77777); the centred values' own
    mean takes that back to 2^-23 of it, 316 times which is 1.2e-6: 1e-5 allowed.
    With noise of 1 on the offset the result keeps the digits of x: the mean to a
    few units in the last place, 6 of them allowed."""
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    N = 3
    shape = (N, G, S, C // G) if layout == "heads" else (N, S, C)
    op = GroupNorm(C, G, x_dtype="f32", layout=layout)
    bias = torch.randn(C, generator=torch.Generator().manual_seed(3)).cuda()
    flat = op.forward(dict(x=torch.full(shape, value, device="cuda"), bias=bias))["y"]
    x = (value + torch.randn(shape, generator=torch.Generator().manual_seed(4))).cuda()
    noisy = op.forward(dict(x=x))["y"]
    torch.cuda.synchronize()
    assert float((flat - bias).abs().max()) <= 1e-5
    ref = layer.group_norm(_host(x), G, layout=layout)
    assert np.abs(_host(noisy) - ref).max() <= 6 * np.spacing(np.float32(abs(value)))


# ------------------------------------------------- the tensor-core kernels' variants
# fp32 results at fp32 accuracy, on max|gpu - ref| / max|ref|.  An accumulator loses 1.1e-9 of the result per value of K
# (tensor cores cut off): 5.6e-7 in a pass of 512, fp32 sums of the passes a few 6e-8 more; 2e-6 allowed.  An operand
# without its third term (2^-17 of each product, signs at random) or K in one accumulator from 4096 on would exceed it.
FP32 = 2e-6


def _product(M, K, N, act, in_dtype, out_dtype, bias=True, residual=True, inplace=False):
    import torch
    from test_learned_neural_gb300.runner import Linear
    g = torch.Generator().manual_seed(51)
    x = torch.randn(M, K, generator=g).to(_dt(in_dtype)).cuda()
    W = (torch.randn(K, N, generator=g) / K ** 0.5).to(_dt(in_dtype)).cuda()
    b = torch.randn(N, generator=g).cuda() if bias else None
    r = torch.randn(M, N, generator=g).to(_dt(out_dtype)).cuda() if residual else None
    ref = layer.linear(_host(x), _host(W), _host(b), _host(r), act)
    op = Linear(K, N, act, in_dtype, out_dtype)
    y = op.forward(dict(x=x, W=W, bias=b, residual=r), out=dict(y=r) if inplace else None)["y"]
    torch.cuda.synchronize()
    op.status()
    assert op.last_path() == 1
    err = maxrel(_host(y), ref)
    print(f"{err:.2e}")
    assert err <= (FP32 if out_dtype == "f32" else TOL["bf16"]), err


# 17 row tiles (a second band of 16) and more tiles than pairs: 256 columns a tile, 128, and rows off 16 bytes
@pytest.mark.parametrize("M,K,N", [(4200, 96, 2048), (4200, 96, 1300), (4200, 96, 1301), (4097, 200, 2056)], ids=str)
@pytest.mark.parametrize("in_dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("residual", ["none", "own", "in place"])
def test_linear_several_tiles_per_pair(gpu_lib, M, K, N, in_dtype, out_dtype, residual):
    _product(M, K, N, "none", in_dtype, out_dtype, N % 2 == 0, residual != "none", residual == "in place")


# passes of K: one, a whole number and a rest; with and without a split
@pytest.mark.parametrize("M,K,N", [(300, 8192, 4096), (300, 517, 264), (40, 8192, 136), (700, 2100, 1160)], ids=str)
@pytest.mark.parametrize("in_dtype", ["bf16", "f32"])
def test_linear_fp32_accuracy(gpu_lib, M, K, N, in_dtype):
    _product(M, K, N, "none", in_dtype, "f32")


@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (48, 48)], ids=str)
@pytest.mark.parametrize("B,T", [(2, 2050), (160, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_fp32_accuracy(gpu_lib, dims, B, T, dtype):
    """As the product: chunks of at most 128 tokens and 128 keys per accumulator."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    (dk, dv), H = dims, 2
    t = _decay_inputs(B, H, T, dk, dv, dtype, 1, "heads", False, True, seed=52, gammas=[1.0, 0.97])
    op = DecayAttention(H, dk, dv, qkv_dtype=dtype, y_dtype="f32")
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    rows = min(B, 3)
    y, S = _decay_ref({n: v if n == "decay" else v[:rows] for n, v in t.items()}, "heads", "heads")
    ey, eS = maxrel(_host(out["y"][:rows]), y), maxrel(_host(out["S"][:rows]), S)
    print(f"y {ey:.2e} S {eS:.2e}")
    assert ey <= FP32 and eS <= FP32


# clusters of 2, 4 and 8 (both types); groups that do not fill the last tile
@pytest.mark.parametrize("N,S,C,G", [(40, 500, 256, 8), (40, 900, 256, 8), (20, 1900, 256, 8), (20, 4000, 256, 8),
                                     (60, 1025, 80, 5), (40, 700, 96, 6)], ids=str)
@pytest.mark.parametrize("x_dtype,y_dtype,act", [("bf16", "bf16", "silu"), ("f32", "f32", "none"), ("f32", "bf16", "gelu")])
def test_norm_clusters(gpu_lib, N, S, C, G, x_dtype, y_dtype, act):
    _norm_check(N, S, C, G, x_dtype, act, y_dtype, rows=slice(0, N, N // 3))


@pytest.mark.parametrize("N,S,C,G,dtype", [(320, 60000, 16, 2, "f32"), (320, 20000, 15, 1, "f32"), (200, 47, 255, 3, "f32"),
                                           (40, 900, 256, 8, "f32"), (1, 30000, 64, 2, "f32"), (320, 60000, 16, 2, "bf16")])
def test_norm_behind_an_outlier(gpu_lib, N, S, C, G, dtype):
    """Position 0 of channel 0 is 1000 standard deviations away (a token that
    attention collects on): the variance keeps its digits.  Squares of 1000 in
    blocks of up to 64 values under one shift: 64 of them lose a few 2^-24 of 6e7
    each, 20 of 1e6 and half of that in the inverse deviation, 1e-5.  The
    largest value is the outlier's own; the others, of order 1 / (1000 / sqrt(S)), are
    held to 1e-5 of themselves as a whole."""
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    g = torch.Generator(device="cuda").manual_seed(61)
    x = torch.randn(N, S, C, generator=g, device="cuda")
    x[:, 0, 0] = 1000
    x = x.to(_dt(dtype))
    y = GroupNorm(C, G, x_dtype=dtype, y_dtype="f32").forward(dict(x=x))["y"]
    torch.cuda.synchronize()
    pick = slice(0, N, max(1, N // 3))
    got, ref = _host(y[pick]), layer.group_norm(_host(x[pick]), G)
    for part in (np.s_[:, 0], np.s_[:, 1:]):
        err = _rms(got[part] - ref[part]) / _rms(ref[part])
        print(f"{err:.2e}")
        assert err <= 1e-5


# ------------------------------------------------------------------ chained
def test_behind_the_memory_itself(gpu_lib):
    """The memory's own read-out through the head norm and the output projection:
    each stage against the oracle on what it was given (2^-8 of the values, as
    the operators' own tests)."""
    import torch
    from harness import WORKLOADS, make_inputs
    from test_learned_neural_gb300.runner import GroupNorm, Linear, Memory, tensors_from_numpy
    w = WORKLOADS["titans_mlp"].scaled(B=2, H=4, T=192)
    mem = Memory(w)
    y = mem.forward(tensors_from_numpy(make_inputs(w)))["y"]
    B, H, T, d = y.shape
    g = torch.Generator().manual_seed(71)
    weight, W_o = (1 + 0.1 * torch.randn(H * d, generator=g)).cuda(), (torch.randn(H * d, 96, generator=g) / 16).bfloat16().cuda()
    x = torch.randn(B * T, 96, generator=g).bfloat16().cuda()
    n = GroupNorm(H * d, H, "silu", x_dtype="f32", y_dtype="bf16", layout="heads").forward(dict(x=y, weight=weight))["y"]
    out = Linear(H * d, 96).forward(dict(x=n.view(B * T, H * d), W=W_o, residual=x))["y"]
    torch.cuda.synchronize()
    mem.status()
    assert n.shape == (B, T, H * d)
    assert maxrel(_host(n), layer.group_norm(_host(y), H, _host(weight), None, "silu", layout="heads")) <= TOL["bf16"]
    assert maxrel(_host(out), layer.linear(_host(n).reshape(B * T, H * d), _host(W_o), residual=_host(x))) <= TOL["bf16"]
