"""The selective scan on the GPU against its fp64 oracle on the same inputs.

Tolerances, on max|gpu - ref| / max|ref| of a tensor, as derived for the decay
attention (tests/test_gpu_layer.py): fp32 read-outs and states 1e-5 (sums of about a
thousand products, 2e-6 for random signs; a product of up to 128 decays adds 128
roundings of 2^-24 at most, 8e-6, about 7e-7 for random ones); bf16 read-outs
half a step of 2^-8 of the largest value and the weighted scores' and the
state's 2^-16: 4.1e-3.
"""
import numpy as np
import pytest

from oracle import layer
from tests.gpu_common import maxrel
from tests.test_gpu_selective import _dt, _host, _offset

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 4.1e-3}


def _inputs(B, H, T, dk, dv, dtype="bf16", gates="memory", share=1, layout="heads", ragged=False, state=True, skip=False, seed=0,
            unaligned=False, apart=0, reset=0.0):
    """apart: values between a token's last and the next one's first (tokens layout: v, k and q side by side in one row)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    Hq = H // share
    q, k = (torch.nn.functional.normalize(n(B, T, Hq, dk), dim=-1) for _ in range(2))
    v, t = n(B, T, H, dv), {}
    if gates == "memory":
        t["theta"], t["alpha"] = torch.rand(B, T, H, generator=g) + 0.1, torch.sigmoid(2 * n(B, T, H) - 4)
        if reset:
            t["alpha"][torch.rand(B, T, H, generator=g) < reset] = 1.0
    else:
        t["dt"], t["dt_bias"], t["A"] = n(B, T, H), n(H) - 3, -torch.rand(H, generator=g) * 8
    if layout == "heads":
        t = {m: a.transpose(1, 2).contiguous() if m in ("theta", "alpha", "dt") else a for m, a in t.items()}
        q, k, v = (_offset(a.transpose(1, 2).to(_dt(dtype)).contiguous().cuda(), unaligned) for a in (q, k, v))
    elif apart:
        row = torch.cat([v.flatten(2), k.flatten(2), q.flatten(2), torch.full((B, T, apart), float("nan"))], 2)
        row = _offset(row.to(_dt(dtype)).cuda(), unaligned)
        a, b = H * dv, H * dv + Hq * dk
        v, k, q = (row[..., i:j].unflatten(2, (-1, d)) for i, j, d in ((0, a, dv), (a, b, dk), (b, b + Hq * dk, dk)))
        wide = torch.cat([t[m] for m in ("theta", "alpha", "dt") if m in t] + [torch.full((B, T, 3), float("nan"))], 2).cuda()
        for i, m in enumerate([m for m in ("theta", "alpha", "dt") if m in t]):
            t[m] = wide[..., i * H:(i + 1) * H]
    else:
        q, k, v = (_offset(a.to(_dt(dtype)).cuda(), unaligned) for a in (q, k, v))
    t = {m: a.cuda() for m, a in t.items()}
    t.update(q=q, k=k, v=v)
    if skip:
        t["D"] = n(H).cuda()
    if ragged:
        t["lens"] = torch.tensor([(T * b) // max(1, B - 1) for b in range(B)], dtype=torch.int32).cuda()
    if state:
        t["S0"] = _offset(n(B, H, dk, dv).cuda(), unaligned)
    return t


def _ref(t, layout="heads", y_layout="heads", scale=1.0):
    first = lambda a: _host(a) if layout == "heads" else _host(a).swapaxes(1, 2)  # noqa: E731
    q, k, v = (first(t[n]) for n in ("q", "k", "v"))
    if "theta" in t:
        s, g = first(t["theta"]), 1 - first(t["alpha"])
    else:
        s, g = layer.step_gates(first(t["dt"]), _host(t.get("dt_bias")), _host(t["A"]))
    y, S = layer.selective_scan(q, k, v, s, g, _host(t.get("D")), None if t.get("lens") is None else t["lens"].cpu().numpy(),
                                _host(t.get("S0")), scale)
    return (y if y_layout == "heads" else y.swapaxes(1, 2)), S


def _op(t, H, dk, dv, dtype, y_dtype, share=1, layout="heads", y_layout="heads", scale=1.0):
    from test_learned_neural_gb300.runner import SelectiveScan
    return SelectiveScan(H, dk, dv, share, "memory" if "theta" in t else "step", dtype, y_dtype, layout, y_layout, scale)


def _check(t, H, dk, dv, dtype, y_dtype, share=1, layout="heads", y_layout="heads", scale=1.0, out=None, ref=None):
    import torch
    op = _op(t, H, dk, dv, dtype, y_dtype, share, layout, y_layout, scale)
    y, S = ref or _ref(t, layout, y_layout, scale)
    out = op.forward(t, out=out)
    torch.cuda.synchronize()
    op.status()
    ey, eS = maxrel(_host(out["y"]), y), maxrel(_host(out["S"]), S)
    print(f"path {op.last_path()} y {ey:.2e} S {eS:.2e}")
    assert ey <= TOL[y_dtype] and eS <= TOL["f32"], (ey, eS)
    return out


# B, H, share, T, d_k, d_v
SCAN = [
    (1, 1, 1, 1, 64, 64), (3, 4, 2, 1, 128, 64), (2, 3, 1, 1, 5, 7), (2, 2, 1, 1, 200, 65), (1, 2, 1, 2, 16, 16),
    (2, 2, 2, 16, 64, 48), (2, 2, 1, 17, 64, 64), (1, 3, 1, 63, 48, 48), (2, 2, 1, 64, 64, 64), (1, 2, 1, 65, 64, 64),
    (2, 2, 1, 127, 64, 64), (1, 6, 2, 128, 64, 128), (1, 6, 3, 129, 128, 64), (3, 2, 1, 300, 24, 80),
    (1, 2, 1, 200, 3, 130), (1, 2, 1, 150, 136, 72), (1, 1, 1, 257, 256, 65), (1, 1, 1, 2050, 64, 64),
    (2, 1, 1, 1111, 128, 128), (160, 1, 1, 140, 32, 32), (2, 6, 1, 700, 96, 40),
    # rings of stages that turn more than once: many chunks per block, whole (more rows than SMs) and in segments
    (160, 1, 1, 900, 64, 64), (40, 1, 1, 2300, 64, 64), (20, 2, 1, 1500, 128, 64),
]


@pytest.mark.parametrize("case", SCAN, ids=str)
@pytest.mark.parametrize("dtype,y_dtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_scan_parity(gpu_lib, case, dtype, y_dtype):
    B, H, share, T, dk, dv = case
    t = _inputs(B, H, T, dk, dv, dtype, "step" if (T + dk) % 3 == 0 else "memory", share, state=T % 2 == 0 or T == 1, skip=T % 3 != 1,
                reset=0.02 if T % 5 == 0 else 0.0)
    _check(t, H, dk, dv, dtype, y_dtype, share, scale=0.5 if T == 64 else 1.0)


@pytest.mark.parametrize("T", [1, 9, 64, 333, 1500])
@pytest.mark.parametrize("layout,y_layout", [("heads", "tokens"), ("tokens", "heads"), ("tokens", "tokens")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gates", ["memory", "step"])
def test_scan_ragged_layouts(gpu_lib, T, layout, y_layout, dtype, gates):
    """Lengths from 0 to T; what lies past a row's length is never read."""
    B, H, dk, dv = 4, 4, 64, 64
    t = _inputs(B, H, T, dk, dv, dtype, gates, 2, layout, ragged=True, skip=True, seed=1)
    ref = _ref(t, layout, y_layout)
    for b, n in enumerate(t["lens"].tolist()):
        for m in ("q", "k", "v", "theta", "alpha", "dt"):
            if m in t:
                (t[m][b, :, n:] if layout == "heads" else t[m][b, n:]).fill_(float("nan"))
    out = _check(t, H, dk, dv, dtype, "f32" if dtype == "f32" else "bf16", 2, layout, y_layout, ref=ref)
    y = out["y"] if y_layout == "heads" else out["y"].transpose(1, 2)
    for b, n in enumerate(t["lens"].tolist()):
        assert not y[b, :, n:].any()


@pytest.mark.parametrize("T", [1, 7, 200, 1000])
@pytest.mark.parametrize("dtype,dk,dv,apart,unaligned", [
    ("bf16", 64, 64, 24, False), ("bf16", 128, 64, 8, False), ("bf16", 64, 48, 3, False), ("bf16", 20, 12, 4, False),
    ("bf16", 64, 64, 8, True), ("f32", 64, 48, 4, False), ("f32", 33, 17, 1, True)])
def test_scan_rows_inside_wider_ones(gpu_lib, T, dtype, dk, dv, apart, unaligned):
    """q, k, v and the gates as slices: of the convolution's rows, of a projection's."""
    t = _inputs(3, 4, T, dk, dv, dtype, "step" if apart % 8 else "memory", 4, "tokens", apart=apart, unaligned=unaligned, skip=True,
                ragged=True, seed=2)
    _check(t, 4, dk, dv, dtype, "f32", 4, "tokens", "tokens")


@pytest.mark.parametrize("dtype,dk,dv,T", [("bf16", 64, 64, 700), ("bf16", 128, 128, 700), ("bf16", 50, 30, 300), ("f32", 48, 48, 700),
                                           ("bf16", 64, 64, 3), ("f32", 130, 64, 300)])
def test_scan_unaligned_and_in_place(gpu_lib, dtype, dk, dv, T):
    t = _inputs(2, 2, T, dk, dv, dtype, unaligned=True, skip=True)
    ref = _ref(t)
    import torch
    out = dict(y=_offset(torch.empty((2, 2, T, dv), dtype=_dt(dtype)).cuda()), S=t["S0"])
    _check(t, 2, dk, dv, dtype, dtype, out=out, ref=ref)


@pytest.mark.parametrize("dtype,T", [("bf16", 500), ("f32", 500), ("bf16", 12)])
def test_scan_extreme_gates(gpu_lib, dtype, T):
    """Resets, no decay at all, decays that leave fp32's range within a chunk, steps of zero and below."""
    import torch
    t = _inputs(1, 6, T, 64, 64, dtype, state=True)
    a = t["alpha"]
    a[0, 0] = 0.0
    a[0, 1] = 1.0
    a[0, 2] = 1 - 1e-6
    a[0, 3, ::7] = 1.0
    a[0, 4, :T // 2] = 1.0
    t["theta"][0, 5] *= -1
    t["theta"][0, 3, ::3] = 0.0
    t["theta"][0, 0] *= 0.01
    y, S = _ref(t)
    op = _op(t, 6, 64, 64, dtype, "f32")
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    for h in range(6):   # head by head: their sizes differ
        assert maxrel(_host(out["y"])[:, h], y[:, h]) <= 1e-5 and maxrel(_host(out["S"])[:, h], S[:, h]) <= 1e-5, h


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk", [64, 128])
def test_scan_calls_continue_one_another(gpu_lib, dtype, dk):
    """A prompt in pieces, down to single tokens, against the whole."""
    import torch
    t = _inputs(2, 2, 330, dk, 64, dtype, "step", skip=True)
    op = _op(t, 2, dk, 64, dtype, "f32")
    whole = op.forward(t)
    S, ys, at = t["S0"], [], 0
    for n in (1, 200, 1, 1, 27, 100):
        cut = {m: a[:, :, at:at + n].contiguous() if m in ("q", "k", "v", "dt") else a for m, a in t.items()}
        out = op.forward({**cut, "S0": S})
        S, at = out["S"], at + n
        ys.append(out["y"])
    assert maxrel(_host(torch.cat(ys, 2)), _host(whole["y"])) <= 1e-5 and maxrel(_host(S), _host(whole["S"])) <= 1e-5


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("dtype,dk", [("bf16", 64), ("bf16", 96), ("f32", 48)])
def test_scan_non_finite_values_stay_in_their_row_and_head(gpu_lib, T, dtype, dk):
    import torch
    t = _inputs(3, 4, T, dk, 40, dtype, share=2, skip=True)
    op = _op(t, 4, dk, 40, dtype, "f32", 2)
    clean = {n: a.clone() for n, a in op.forward(t).items()}
    at = T // 2
    t["k"][0, 1, at, 3] = float("nan")       # heads 2 and 3 of row 0
    t["v"][1, 2, at, 5] = float("inf")
    t["alpha"][2, 0, at] = float("nan")
    t["theta"][2, 3, at] = float("inf")
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    for n in ("y", "S"):
        hit = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
        for b, h in ((0, 2), (0, 3), (1, 2), (2, 0), (2, 3)):
            hit[b, h] = True
        assert torch.equal(out[n][~hit], clean[n][~hit])
    assert torch.isnan(out["S"][2, 0]).all() and not torch.isfinite(out["S"][0, 2, 3]).any()
    first = max(0, at - 127)
    assert torch.equal(out["y"][0, 2, :first], clean["y"][0, 2, :first])


@pytest.mark.parametrize("T", [1, 600])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_repeated_streamed_and_captured_calls_give_the_same_bits(gpu_lib, T, dtype):
    import torch
    t = _inputs(2, 2, T, 64, 64, dtype, skip=True)
    op = _op(t, 2, 64, 64, dtype, "f32")
    out, graph = op.alloc_outputs(2, T, "cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):        # the first call of the handle
        op.forward(t, out=out)
    graph.replay()
    torch.cuda.synchronize()
    ref = {n: a.clone() for n, a in out.items()}
    big = _inputs(2, 2, 2 * T + 900, 64, 64, dtype, skip=True)
    op.forward(big)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = op.forward(t)
    side.synchronize()
    for a in out.values():
        a.zero_()
    graph.replay()
    torch.cuda.synchronize()
    op.status()
    for n in ref:
        assert torch.equal(ref[n], other[n]) and torch.equal(ref[n], out[n])
    y, S = _ref(t)
    assert maxrel(_host(ref["y"]), y) <= 1e-5 and maxrel(_host(ref["S"]), S) <= 1e-5


def test_scan_takes_the_stage_in_fronts_outputs(gpu_lib):
    """Prologue's q, k, v and gates as they are."""
    import torch
    from types import SimpleNamespace
    from test_learned_neural_gb300.runner import Prologue
    B, T, D, H, d = 2, 300, 96, 3, 32
    cfg = SimpleNamespace(D=D, H=H, d_k=d, d_v=d, conv=4, with_gamma=0, theta_max=0.1, qkv_dtype="bf16", Nc=3 * H * d)
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = Prologue(cfg).forward(dict(x=n(B, T, D).bfloat16().cuda(), W_in=(n(D, cfg.Nc + 3 * H) / D ** 0.5).bfloat16().cuda(),
                                   conv_w=n(cfg.Nc, 4).cuda(), gate_b=n(3, H).cuda()))
    t = {m: p[m] for m in ("q", "k", "v", "theta", "alpha")}
    _check(t, H, d, d, "bf16", "bf16")


@pytest.mark.parametrize("scale", [0.0, -0.25])
@pytest.mark.parametrize("dtype,y_dtype,dk,T", [("bf16", "bf16", 64, 300), ("bf16", "f32", 64, 300), ("bf16", "bf16", 128, 300),
                                                ("bf16", "f32", 128, 300), ("f32", "f32", 48, 300), ("bf16", "f32", 64, 2)])
def test_scan_scale_is_not_of_the_skip_term(gpu_lib, scale, dtype, y_dtype, dk, T):
    """A factor of 0 leaves D v; a negative one turns the read-outs alone."""
    t = _inputs(2, 2, T, dk, 64, dtype, "step", skip=True, seed=3)
    _check(t, 2, dk, 64, dtype, y_dtype, scale=scale)


def test_scan_steps_that_vanish_or_saturate(gpu_lib):
    """dt of -inf (a token that is left out), of 80 and of 1e4 with A = 0 and A far below 0."""
    import torch
    for T, dtype in ((4, "f32"), (300, "bf16"), (300, "f32")):
        t = _inputs(1, 3, T, 64, 32, dtype, "step", seed=4)
        t["dt_bias"].zero_()
        t["A"].copy_(torch.tensor([0.0, -1.0, -1e30]))
        t["dt"][0, :, 1::3] = -float("inf")
        t["dt"][0, 1, 2::7] = 80.0
        t["dt"][0, 2, 2::11] = 1e4
        y, S = _ref(t)
        out = _op(t, 3, 64, 32, dtype, "f32").forward(t)
        for h in range(3):
            assert maxrel(_host(out["y"])[:, h], y[:, h]) <= 1e-5 and maxrel(_host(out["S"])[:, h], S[:, h]) <= 1e-5, (T, dtype, h)


def test_scans_of_two_handles_on_two_streams_at_once(gpu_lib):
    import torch
    calls = []
    for i, (dk, T) in enumerate(((64, 900), (128, 700))):
        t = _inputs(2, 4, T, dk, 64, "bf16", skip=True, seed=6 + i)
        op = _op(t, 4, dk, 64, "bf16", "f32")
        calls.append((op, t, {n: a.clone() for n, a in op.forward(t).items()}, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (op, t, _, st) in enumerate(calls):
            with torch.cuda.stream(st):
                outs[i].append(op.forward(t))
    torch.cuda.synchronize()
    for (op, _, ref, _), many in zip(calls, outs):
        op.status()
        for out in many:
            assert all(torch.equal(out[n], ref[n]) for n in ref)


@pytest.mark.parametrize("T", [21, 31, 32, 33, 63, 64, 65, 96, 200])
@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("f32", 16, 8), ("f32", 63, 31), ("f32", 65, 33), ("f32", 96, 66), ("f32", 128, 128),
                                         ("f32", 129, 12), ("f32", 256, 64), ("bf16", 160, 64), ("bf16", 131, 70)])
@pytest.mark.parametrize("state", [False, True])
def test_scan_split_chunks_at_their_edges(gpu_lib, T, dtype, dk, dv, state):
    """Chunks of 64 and 32 tokens from split operands: whole, a token less and more, with and without a state to
    carry on; many units, so that a block takes several chunks."""
    B = 1 if T < 64 else 80
    t = _inputs(B, 4, T, dk, dv, dtype, "step" if dk % 2 else "memory", 2, "tokens", state=state, skip=state, seed=T + dk)
    _check(t, 4, dk, dv, dtype, "f32", 2, "tokens", "heads")


def test_scan_split_accuracy(gpu_lib):
    """Two parts of 11 bits, the first one rounded: 2^-23 of a factor is cut off, 2^-22 of a product left out, 2^-21 of it
    altogether.  A read-out has two such products in a row, so that sums without cancellation, positive values, come
    within 2^-20, and another 2^-19 for the weights' products and the sums' roundings."""
    import torch
    for dk, T in ((64, 640), (128, 640), (256, 320)):
        t = _inputs(2, 2, T, dk, 64, "f32", seed=9)
        for n in ("q", "k", "v", "S0"):
            t[n].abs_()
        y, S = _ref(t)
        out = _op(t, 2, dk, 64, "f32", "f32").forward(t)
        for got, want in ((out["y"], y), (out["S"], S)):
            worst = (np.abs(_host(got) - want) / want).max()
            assert worst <= 2.0 ** -19 + 2.0 ** -20, (dk, worst)
