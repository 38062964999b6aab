"""The layer operators around the memory on the GPU against their fp64 oracle
on the same inputs.

Tolerances are on max|gpu - ref| / max|ref| of a tensor:
  bf16 outputs of the norm and of the product are fp32 values rounded once:
    2^-9 of the largest value, doubled for the fp32 error at a tie: 4e-3;
  bf16 read-outs of the decay attention may also round the masked scores and
    the state to bf16 (2^-9 each, of sums whose terms exceed the result by at
    most a small factor on random inputs): 1e-2;
  fp32 outputs: sums of up to about 1000 products, each rounded to 2^-24 of
    partial sums of the order of the result: about sqrt(1000) 6e-8 = 2e-6 for
    random signs, 1e-5 allowed; operands split into two bf16 halves carry
    2^-17 = 7.6e-6 each, inside the same 1e-5.
"""
import numpy as np
import pytest

from oracle import layer
from tests.gpu_common import maxrel

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 4e-3}
TOL_DECAY = {"f32": 1e-5, "bf16": 1e-2}


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _offset(t, on):
    """The same values at an address that is a multiple of the element size only."""
    import torch
    if not on:
        return t
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    flat.copy_(t.reshape(-1))
    return flat.view(t.shape)


# --------------------------------------------------------- decay attention
def _decay_inputs(B, H, T, dk, dv, dtype, share, layout, ragged, state, seed=0, gammas=None, unaligned=False):
    import torch
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    def heads(n, d, unit):
        x = normal(*((B, n, T, d) if layout == "heads" else (B, T, n, d)))
        x = x / x.norm(dim=-1, keepdim=True) if unit else x
        return _offset(x.to(_dt(dtype)).cuda(), unaligned)

    t = dict(q=heads(H // share, dk, True), k=heads(H // share, dk, True), v=heads(H, dv, False))
    if gammas is None:
        gammas = [0.9, 1.0, 0.0, 0.97, 0.5, 0.999]
    t["decay"] = torch.tensor([gammas[h % len(gammas)] for h in range(H)]).cuda()
    if ragged:
        t["lens"] = torch.tensor([(T * b) // max(1, B - 1) for b in range(B)], dtype=torch.int32).cuda()
    if state:
        t["S0"] = _offset(normal(B, H, dk, dv).cuda(), unaligned)
    return t


def _decay_ref(t, layout, y_layout, scale=1.0):
    q, k, v = (_host(t[n]) if layout == "heads" else _host(t[n]).transpose(0, 2, 1, 3) for n in ("q", "k", "v"))
    y, S = layer.decay_attention(q, k, v, _host(t["decay"]), None if t.get("lens") is None else t["lens"].cpu().numpy(),
                                 _host(t.get("S0")), scale)
    return (y if y_layout == "heads" else y.transpose(0, 2, 1, 3)), S


def _decay_check(t, H, dk, dv, dtype, y_dtype, share, layout, y_layout, scale=1.0, tol=None):
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    op = DecayAttention(H, dk, dv, share, dtype, y_dtype, layout, y_layout, scale)
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    y, S = _decay_ref(t, layout, y_layout, scale)
    ey, eS = maxrel(_host(out["y"]), y), maxrel(_host(out["S"]), S)
    print(f"path {op.last_path()} y {ey:.2e} S {eS:.2e}")
    tol = tol or TOL_DECAY
    assert ey <= tol[y_dtype] and eS <= tol["f32"], (ey, eS)
    op.close()
    return out


# B, H, share, T, d_k, d_v
DECAY = [
    (1, 1, 1, 1, 64, 64), (3, 4, 2, 1, 128, 128), (2, 3, 1, 1, 5, 7), (2, 2, 1, 1, 200, 65), (1, 2, 1, 2, 16, 16),
    (2, 2, 2, 16, 64, 48), (2, 2, 1, 17, 64, 64), (1, 3, 1, 63, 48, 48), (2, 2, 1, 64, 64, 64), (1, 2, 1, 65, 64, 64),
    (2, 2, 1, 127, 64, 64), (1, 6, 2, 128, 64, 128), (1, 6, 3, 129, 128, 64), (3, 2, 1, 300, 24, 80),
    (1, 2, 1, 200, 3, 130), (1, 2, 1, 150, 136, 72), (1, 1, 1, 257, 256, 65), (1, 1, 1, 2050, 64, 64),
    (2, 1, 1, 1111, 128, 128), (160, 1, 1, 140, 32, 32), (2, 6, 1, 700, 96, 40),
    # rings of stages that turn more than once: many chunks per block, whole (more rows than SMs) and in segments
    (160, 1, 1, 900, 64, 64), (40, 1, 1, 2300, 64, 64), (20, 2, 1, 1500, 128, 64),
]


@pytest.mark.parametrize("case", DECAY, ids=str)
@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_decay_parity(gpu_lib, case, dtype, y_dtype):
    B, H, share, T, dk, dv = case
    t = _decay_inputs(B, H, T, dk, dv, dtype, share, "heads", ragged=False, state=T % 2 == 0 or T == 1)
    _decay_check(t, H, dk, dv, dtype, y_dtype, share, "heads", "heads", scale=0.5 if T == 64 else 1.0)


@pytest.mark.parametrize("T", [1, 9, 64, 333, 1500])
@pytest.mark.parametrize("layout,y_layout", [("heads", "tokens"), ("tokens", "heads"), ("tokens", "tokens")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_ragged_layouts(gpu_lib, T, layout, y_layout, dtype):
    """Lengths from 0 to T; what lies past a row's length is never read."""
    B, H, dk, dv = 4, 4, 64, 64
    t = _decay_inputs(B, H, T, dk, dv, dtype, 2, layout, ragged=True, state=True, seed=1)
    for n in ("q", "k", "v"):
        for b in range(B):
            (t[n][b, :, int(t["lens"][b]):] if layout == "heads" else t[n][b, int(t["lens"][b]):]).fill_(float("nan"))
    out = _decay_check(t, H, dk, dv, dtype, dtype, 2, layout, y_layout)
    assert bool((out["y"][0] == 0).all()) and bool((out["S"][0] == t["S0"][0]).all())


@pytest.mark.parametrize("T", [1, 5, 100, 900])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_unaligned(gpu_lib, T, dtype):
    t = _decay_inputs(2, 2, T, 64, 64, dtype, 1, "heads", False, True, seed=2, unaligned=True)
    _decay_check(t, 2, 64, 64, dtype, "f32", 1, "heads", "heads")


@pytest.mark.parametrize("gammas", [[0.0], [1.0], [1e-30], [0.25], [1 - 2.0 ** -20]], ids=str)
@pytest.mark.parametrize("T", [3, 400])
def test_decay_extremes(gpu_lib, gammas, T):
    t = _decay_inputs(1, 2, T, 64, 64, "bf16", 1, "heads", False, True, seed=3, gammas=gammas)
    _decay_check(t, 2, 64, 64, "bf16", "f32", 1, "heads", "heads")


@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (48, 200)], ids=str)
@pytest.mark.parametrize("T", [300, 900, 2000, 5000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_state_in_place_of_split_rows(gpu_lib, dims, T, dtype):
    """Long rows beside short and empty ones, split along the tokens: S_out in
    S0's buffer gives the bits that a buffer of its own gives."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    (dk, dv), B, H = dims, 5, 4
    t = _decay_inputs(B, H, T, dk, dv, dtype, 2, "tokens", False, True, seed=T)
    t["lens"] = torch.tensor([T, 0, 1, T // 2, T - 1], dtype=torch.int32).cuda()
    op = DecayAttention(H, dk, dv, 2, dtype, "f32", "tokens", "tokens")
    own = op.forward(t)
    S = t["S0"].clone()
    out = dict(y=torch.empty_like(own["y"]), S=S)
    op.forward(dict(t, S0=S), out=out)
    torch.cuda.synchronize()
    op.status()
    assert torch.equal(out["y"], own["y"]) and torch.equal(S, own["S"])
    assert torch.equal(S[1], t["S0"][1])


@pytest.mark.parametrize("cuts", [(1,), (40, 41), (64,), (130, 500)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_continues_in_place(gpu_lib, cuts, dtype):
    """Pieces with the state continued in its own buffer equal one call."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    B, H, T, d = 2, 2, 777, 64
    t = _decay_inputs(B, H, T, d, d, dtype, 1, "heads", False, True, seed=4)
    op = DecayAttention(H, d, d, qkv_dtype=dtype, y_dtype="f32")
    whole = op.forward(t)
    S = t["S0"].clone()
    ys, edges = [], (0, *cuts, T)
    for a, b in zip(edges, edges[1:]):
        part = {n: t[n][:, :, a:b].contiguous() for n in ("q", "k", "v")}
        out = dict(y=torch.empty(B, H, b - a, d, device="cuda"), S=S)
        op.forward(dict(part, decay=t["decay"], S0=S), out=out)
        ys.append(out["y"])
    torch.cuda.synchronize()
    op.status()
    # each side is within the fp32 tolerance of the formula
    assert maxrel(_host(torch.cat(ys, 2)), _host(whole["y"])) <= 2 * TOL_DECAY["f32"]
    assert maxrel(_host(S), _host(whole["S"])) <= 2 * TOL_DECAY["f32"]


def test_decay_other_stream_and_repeat(gpu_lib):
    """On a side stream, twice: the same bits."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    t = _decay_inputs(1, 4, 3000, 64, 64, "bf16", 1, "heads", False, True, seed=5)
    op = DecayAttention(4, 64, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = op.alloc_outputs(1, 3000, "cuda"), op.alloc_outputs(1, 3000, "cuda")
    with torch.cuda.stream(s):
        op.forward(t, out=a)
    op.forward(t, out=b, stream=s.cuda_stream)
    s.synchronize()
    op.status()
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["S"], b["S"])
    y, S = _decay_ref(t, "heads", "heads")
    assert maxrel(_host(a["y"]), y) <= TOL_DECAY["bf16"] and maxrel(_host(a["S"]), S) <= TOL_DECAY["f32"]


# -------------------------------------------------------------- group norm
# N, S, C, groups
NORM = [
    (1, 1, 1, 1), (3, 1, 64, 8), (2, 1, 512, 8), (5, 1, 1024, 1), (2, 1, 2048, 1), (3, 1, 70, 7), (2, 1, 768, 16),
    (1, 2, 6, 3), (2, 33, 24, 3), (3, 64, 256, 8), (2, 1000, 64, 4), (1, 4097, 48, 2), (2, 257, 510, 6),
    (700, 9, 96, 6), (640, 30, 40, 5), (610, 2, 80, 10), (630, 16, 96, 2),   # several groups per tile
    (1, 20000, 16, 2), (4, 7, 5, 5), (2, 50, 8192, 2), (70000, 1, 8, 2), (300, 3, 32, 4), (1, 100, 1030, 2),
]


def _norm_check(x, C, groups, act, x_dtype, y_dtype, layout, affine, tol=None, inplace=False):
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    g = torch.Generator().manual_seed(9)
    w = (1 + 0.2 * torch.randn(C, generator=g)).cuda() if affine else None
    b = (0.2 * torch.randn(C, generator=g)).cuda() if affine else None
    ref = layer.group_norm(_host(x), groups, _host(w), _host(b), act, layout=layout)
    op = GroupNorm(C, groups, act, x_dtype=x_dtype, y_dtype=y_dtype, layout=layout)
    out = op.forward(dict(x=x, weight=w, bias=b), out=dict(y=x) if inplace else None)
    torch.cuda.synchronize()
    err = maxrel(_host(out["y"]), ref)
    print(f"{err:.2e}")
    assert err <= (tol or TOL[y_dtype]), err
    op.close()


@pytest.mark.parametrize("case", NORM, ids=str)
@pytest.mark.parametrize("act,x_dtype,y_dtype", [("silu", "bf16", "bf16"), ("none", "f32", "f32"),
                                                 ("gelu", "bf16", "f32"), ("silu", "f32", "bf16")])
def test_norm_parity(gpu_lib, case, act, x_dtype, y_dtype):
    import torch
    N, S, C, G = case
    x = (torch.randn(N, S, C, generator=torch.Generator().manual_seed(6)) * 1.5 + 0.3).to(_dt(x_dtype)).cuda()
    _norm_check(x, C, G, act, x_dtype, y_dtype, "channels_last", affine=C % 3 != 0)


@pytest.mark.parametrize("case", [(1, 1, 64, 8), (2, 100, 512, 8), (3, 77, 96, 2), (2, 5, 35, 5), (1, 9, 1500, 2), (9000, 2, 64, 8)], ids=str)
@pytest.mark.parametrize("x_dtype,y_dtype", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
def test_norm_heads(gpu_lib, case, x_dtype, y_dtype):
    import torch
    N, S, C, G = case
    x = torch.randn(N, G, S, C // G, generator=torch.Generator().manual_seed(7)).to(_dt(x_dtype)).cuda()
    _norm_check(x, C, G, "silu", x_dtype, y_dtype, "heads", affine=True)


@pytest.mark.parametrize("case", [(3, 1, 64, 4), (2, 500, 64, 4)], ids=str)
def test_norm_unaligned_in_place_and_constant(gpu_lib, case):
    import torch
    N, S, C, G = case
    x = torch.randn(N, S, C, generator=torch.Generator().manual_seed(8)).cuda()
    _norm_check(_offset(x, True), C, G, "none", "f32", "f32", "channels_last", True)
    _norm_check(x.clone(), C, G, "gelu", "f32", "f32", "channels_last", True, inplace=True)
    # a constant set has variance 0: y = act(bias)
    _norm_check(torch.full_like(x, 3.0), C, G, "none", "f32", "f32", "channels_last", True)
    # a common offset of 1000 leaves the mean an error of a few 2^-24 1000 = 6e-5 times log2 of the terms' depth
    # (32000 values: 15), so 1e-3 of values of order 1
    _norm_check(x + 1000, C, G, "none", "f32", "f32", "channels_last", True, tol=1e-3)


def test_norm_nonfinite_stays_in_its_set(gpu_lib):
    import torch
    from test_learned_neural_gb300.runner import GroupNorm
    for S in (1, 300):
        x = torch.randn(2, S, 64, generator=torch.Generator().manual_seed(10)).cuda()
        op = GroupNorm(64, 4, x_dtype="f32")
        want = op.forward(dict(x=x))["y"]
        y2 = x.clone()
        y2[1, 0, 17] = float("inf")
        got = op.forward(dict(x=y2))["y"]
        torch.cuda.synchronize()
        mask = torch.ones_like(x, dtype=torch.bool)
        mask[1, :, 16:32] = False
        assert torch.equal(got[mask], want[mask])
        assert not bool(torch.isfinite(got[1, :, 16:32]).all())


# ---------------------------------------------------------- matrix product
# M, K, N
LINEAR = [
    (1, 512, 512), (1, 1, 1), (1, 77, 300), (2, 768, 768), (5, 520, 264), (8, 64, 4096), (17, 512, 136), (33, 1024, 512),
    (64, 256, 512), (100, 51, 67), (127, 192, 128), (128, 64, 256), (129, 100, 72), (300, 768, 200), (700, 96, 1031),
    (1000, 517, 264), (520, 1000, 1160),
    (40, 8192, 136), (300, 6500, 70), (30, 2100, 100), (5, 2048, 2050),     # K split over the idle blocks (fp32 from about K = 1024)
]


def _linear_check(M, K, N, act, in_dtype, out_dtype, bias=True, residual=True, inplace=False, unaligned=False, x=None):
    import torch
    from test_learned_neural_gb300.runner import Linear
    g = torch.Generator().manual_seed(11)
    x = torch.randn(M, K, generator=g) if x is None else x
    x = _offset(x.to(_dt(in_dtype)).cuda(), unaligned)
    W = _offset((torch.randn(K, N, generator=g) / K ** 0.5).to(_dt(in_dtype)).cuda(), unaligned)
    b = torch.randn(N, generator=g).cuda() if bias else None
    r = _offset(torch.randn(M, N, generator=g).to(_dt(out_dtype)).cuda(), unaligned) if residual else None
    ref = layer.linear(_host(x), _host(W), _host(b), _host(r), act)
    op = Linear(K, N, act, in_dtype, out_dtype)
    out = op.forward(dict(x=x, W=W, bias=b, residual=r), out=dict(y=r) if inplace else None)
    torch.cuda.synchronize()
    op.status()
    err = maxrel(_host(out["y"]), ref)
    print(f"path {op.last_path()} {err:.2e}")
    assert err <= TOL[out_dtype], err
    op.close()
    return out["y"]


@pytest.mark.parametrize("case", LINEAR, ids=str)
@pytest.mark.parametrize("act,in_dtype,out_dtype", [("none", "bf16", "bf16"), ("silu", "bf16", "f32"),
                                                    ("gelu", "f32", "f32"), ("gelu", "bf16", "bf16")])
def test_linear_parity(gpu_lib, case, act, in_dtype, out_dtype):
    M, K, N = case
    _linear_check(M, K, N, act, in_dtype, out_dtype, bias=N % 8 == 0, residual=M % 2 == 0)


@pytest.mark.parametrize("case", [(1, 512, 512), (40, 128, 256), (300, 512, 768)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_in_place_and_unaligned(gpu_lib, case, dtype):
    _linear_check(*case, "silu", dtype, dtype, inplace=True)
    _linear_check(*case, "none", dtype, dtype, unaligned=True)


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_nonfinite_rows_stay_alone(gpu_lib, M, dtype):
    import torch
    from test_learned_neural_gb300.runner import Linear
    g = torch.Generator().manual_seed(12)
    x, W = torch.randn(M, 256, generator=g).to(_dt(dtype)).cuda(), torch.randn(256, 256, generator=g).to(_dt(dtype)).cuda()
    op = Linear(256, 256, in_dtype=dtype)
    want = op.forward(dict(x=x, W=W))["y"]
    x2 = x.clone()
    x2[1, 5] = float("inf")
    got = op.forward(dict(x=x2, W=W))["y"]
    torch.cuda.synchronize()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(got[keep], want[keep]) and not bool(torch.isfinite(got[1]).any())


def test_linear_large_values(gpu_lib):
    """Activations far from zero: exp overflows inside them, the result does not."""
    import torch
    x = torch.tensor([[200.0, -200.0, 1.0, 0.0]]).repeat(40, 1)
    for act in ("silu", "gelu"):
        y = _linear_check(40, 4, 8, act, "f32", "f32", residual=False, x=x)
        assert bool(torch.isfinite(y).all())


# ------------------------------------------------------- graphs and streams
def test_captured_in_a_graph(gpu_lib):
    """After one call of a size (which allocates the workspace) the operators
    can be captured; a replay gives the same bits, on new inputs too."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention, GroupNorm, Linear
    B, H, T, d = 1, 4, 600, 64
    t = _decay_inputs(B, H, T, d, d, "bf16", 1, "heads", False, True, seed=6)
    mix, norm = DecayAttention(H, d, d, y_layout="tokens"), GroupNorm(H * d, H, act="silu")
    pos, lin = GroupNorm(H * d, H), Linear(H * d, 264)
    W = (torch.randn(H * d, 264, generator=torch.Generator().manual_seed(3)) / 16).bfloat16().cuda()
    a, n, p, y = (mix.alloc_outputs(B, T, "cuda"), norm.alloc_outputs(B * T, 1, "cuda"), pos.alloc_outputs(B, T, "cuda"),
                  lin.alloc_outputs(B * T, "cuda"))

    def run():
        mix.forward(t, out=a)
        norm.forward(dict(x=a["y"].view(B * T, 1, H * d)), out=n)
        pos.forward(dict(x=n["y"].view(B, T, H * d)), out=p)
        lin.forward(dict(x=p["y"].view(B * T, H * d), W=W), out=y)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (7, 8):
        fresh = _decay_inputs(B, H, T, d, d, "bf16", 1, "heads", False, True, seed=seed)
        for k in ("q", "k", "v", "S0"):
            t[k].copy_(fresh[k])
        run()
        torch.cuda.synchronize()
        want = [a["y"].clone(), a["S"].clone(), y["y"].clone()]
        for o in (a["y"], a["S"], n["y"], p["y"], y["y"]):
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, (a["y"], a["S"], y["y"])))


# ------------------------------------------------------------------ chained
def _layer_reference(la, x):
    """The example layer in 64 bits, nothing rounded in between."""
    import oracle
    f = {n: _host(v) for n, v in la.w.items()}
    xs = _host(x)
    B, T, D = xs.shape
    rows = [oracle.prologue_row(la.cfg, xs[b], f["W_in"], f["conv_w"], f["gate_b"]) for b in range(B)]
    q, k, v = (np.stack([r[n] for r in rows]) for n in ("q", "k", "v"))
    a, _ = layer.decay_attention(q, k, v, f["decay"])
    n = layer.group_norm(a, la.H, f["norm_w"], f["norm_b"], "silu", layout="heads").reshape(B * T, -1)
    h = layer.linear(n, f["W_o"], residual=xs.reshape(B * T, D))
    y = layer.linear(layer.linear(h, f["W_1"], f["b_1"], act="silu"), f["W_2"], f["b_2"], residual=h)
    return y.reshape(B, T, D)


def test_layer_example(gpu_lib):
    """The example layer: a prompt and then single tokens equal one longer
    prompt, and both equal the chained oracles."""
    import torch
    from examples.decay_layer import DecayLayer, random_weights
    torch.manual_seed(0)
    B, T, D, H, d = 2, 90, 128, 4, 32
    layer_ = DecayLayer(D, H, d, random_weights(D, H, d, hidden=256, device="cuda"))
    x = torch.randn(B, T, D, device="cuda").bfloat16()
    whole, _ = layer_.forward(x)
    first, state = layer_.forward(x[:, :T - 5].contiguous())
    rows = [first]
    for t in range(T - 5, T):
        y, state = layer_.forward(x[:, t:t + 1].contiguous(), state)
        rows.append(y)
    torch.cuda.synchronize()
    ref = _layer_reference(layer_, x)
    # six bf16 roundings lie between x and the result, each 2^-9 of values of the result's order: 6 * 2^-9 = 1.2e-2,
    # through two products that mix them at unit gain
    assert maxrel(_host(whole), ref) <= 2.5e-2
    assert maxrel(_host(torch.cat(rows, 1)), ref) <= 2.5e-2
