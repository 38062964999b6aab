"""The operators of a selective layer run together, as examples/selective_layer.py
does: against their oracles chained, a prompt against its tokens one by one, and a
serving step captured in a graph."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import layer as oracle
from tests.gpu_common import maxrel
from tests.test_gpu_selective import _host

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("selective_layer", os.path.join(ROOT, "examples", "selective_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _silu(z):
    return z / (1 + np.exp(-z))


def _bf16(a):
    import torch
    return torch.from_numpy(a).to(torch.bfloat16).double().numpy()


def _ref(lay, x, stream, state=None):
    """The oracles one behind the other, rounded where the operators round."""
    import torch
    B, T, D = x.shape
    H, d, dk, w = lay.H, lay.d, lay.d_k, {n: _host(a) for n, a in lay.w.items()}
    n, h = oracle.rms_norm(_host(x).reshape(-1, D), _host(stream).reshape(-1, D), w["norm"])
    s = oracle.e4m3_scales(n, 128)
    wide = np.repeat(s, 128, axis=1)[:, :D]
    q8 = torch.from_numpy(n / wide).float().to(torch.float8_e4m3fn).double().numpy()

    def weights(op, W):
        q = op.quantize(W)
        return oracle.quant_weights(q["q"].cpu().numpy(), _host(q["scales"]), None, op.cfg.K, op.cfg.group)

    p = oracle.quant_linear(q8, weights(lay.proj, lay.w["W_in"]), s, 128).reshape(B, T, -1)
    Hd = H * d
    c, cache = oracle.short_conv(_bf16(p[..., Hd:Hd + lay.C]), w["taps"], w["taps_b"], state and state["cache"], act="silu")
    c = _bf16(c)
    v, k, q = (c[..., a:b].reshape(B, T, m, -1).transpose(0, 2, 1, 3) for a, b, m in ((0, Hd, H), (Hd, Hd + dk, 1), (Hd + dk, lay.C, 1)))
    step, decay = oracle.step_gates(p[..., Hd + lay.C:].transpose(0, 2, 1), w["dt_bias"], w["A"])
    a, S = oracle.selective_scan(q, k, v, step, decay, w["skip"], S0=state and state["S"])
    a = _bf16(a.transpose(0, 2, 1, 3).reshape(B * T, 1, Hd))
    g = _bf16(oracle.group_norm(a, H, w["head"])).reshape(B, T, Hd)
    z = p[..., :Hd]
    y = oracle.quant_linear(_bf16(g * _silu(z)).reshape(B * T, Hd), weights(lay.out, lay.w["W_out"])).reshape(B, T, D)
    return y, h.reshape(B, T, D), dict(S=S, cache=cache)


@pytest.mark.parametrize("T,D,H,d,d_k", [(150, 96, 4, 32, 80), (37, 256, 2, 64, 64), (1, 200, 3, 24, 128)])
def test_layer_against_the_oracles_chained(gpu_lib, T, D, H, d, d_k):
    """Each rounding (8-bit norm 2^-4, bf16 2^-8) may fall on the other side of a
    border than the oracle's: one value in e4m3 moves a projection of D values by 2^-4
    / sqrt(D) of its size at most, 6e-3 for D = 96, the states and read-outs as much."""
    import torch
    lay = _example().SelectiveLayer(D, H, d, d_k, seed=1)
    g = torch.Generator().manual_seed(2)
    x, stream = (torch.randn(2, T, D, generator=g).bfloat16().cuda() for _ in range(2))
    y, h, st = lay.forward(x, stream)
    torch.cuda.synchronize()
    lay.scan.status(), lay.proj.status(), lay.out.status()
    ry, rh, rst = _ref(lay, x, stream)
    assert maxrel(_host(h), rh) <= 4e-3 and maxrel(_host(st["S"]), rst["S"]) <= 2e-2 and maxrel(_host(y), ry) <= 3e-2


def test_prompt_equals_its_tokens(gpu_lib):
    """Rows, tokens and heads are computed alike in a prompt and in steps: the
    operators' fp32 sums in another order move a rounding (2^-4 of a value in 8 bits) now and then."""
    import torch
    lay = _example().SelectiveLayer(96, 4, 32, 80, seed=3)
    g = torch.Generator().manual_seed(4)
    x, stream = (torch.randn(2, 24, 96, generator=g).bfloat16().cuda() for _ in range(2))
    y, h, st = lay.forward(x, stream)
    state, ys, hs = None, [], []
    for t in range(24):
        a, b, state = lay.forward(x[:, t:t + 1].contiguous(), stream[:, t:t + 1].contiguous(), state)
        ys.append(a), hs.append(b)
    assert torch.equal(torch.cat(hs, 1), h)
    assert maxrel(_host(torch.cat(ys, 1)), _host(y)) <= 3e-2 and maxrel(_host(state["S"]), _host(st["S"])) <= 2e-2
    assert maxrel(_host(state["cache"]), _host(st["cache"])) <= 2e-2


def test_step_in_a_graph(gpu_lib):
    """A serving step replayed from a graph, the state continued in place."""
    import torch
    lay = _example().SelectiveLayer(128, 2, 64, 64, seed=5)
    g = torch.Generator().manual_seed(6)
    x, stream = (torch.randn(3, 40, 128, generator=g).bfloat16().cuda() for _ in range(2))
    _, _, st0 = lay.forward(x, stream)
    tok, one = x[:, :1].contiguous(), stream[:, :1].contiguous()
    ref, state = [], {n: a.clone() for n, a in st0.items()}
    for _ in range(4):
        y, _, state = lay.forward(tok, one, state)
        ref.append(y.clone())
    cur = {n: a.clone() for n, a in st0.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _, new = lay.forward(tok, one, cur)
        for n in cur:
            cur[n].copy_(new[n])
    for n in cur:
        cur[n].copy_(st0[n])
    for r in ref:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, r)


def test_example_runs(gpu_lib, capsys):
    _example().main()
    assert "tokens/s" in capsys.readouterr().out
