"""CPU checks of the layer operators: the fp64 oracle against closed forms and
torch's fp64 functions, and what the C entry points refuse before any CUDA
call."""
import ctypes
import os

import numpy as np
import pytest

import test_learned_neural_gb300 as tln
from oracle import layer
from test_learned_neural_gb300 import build as tln_build

RNG = np.random.default_rng


# --------------------------------------------------------------- the oracle
@pytest.mark.parametrize("share", [1, 2])
def test_decay_oracle_is_the_sum_over_past_tokens(share):
    r = RNG(0)
    B, H, T, dk, dv = 2, 4, 9, 3, 5
    q, k = r.normal(size=(2, B, H // share, T, dk))
    v, S0 = r.normal(size=(B, H, T, dv)), r.normal(size=(B, H, dk, dv))
    g = np.array([0.0, 1.0, 0.5, 0.9])
    y, S = layer.decay_attention(q, k, v, g, S0=S0, scale=0.7)
    for h in range(H):
        w = np.array([[g[h] ** (t - j) if j <= t else 0.0 for j in range(T)] for t in range(T)])
        qh, kh = q[:, h // share], k[:, h // share]
        want = 0.7 * ((np.einsum("btk,bjk->btj", qh, kh) * w) @ v[:, h]
                      + (g[h] ** np.arange(1, T + 1))[None, :, None] * (qh @ S0[:, h]))
        np.testing.assert_allclose(y[:, h], want, rtol=1e-12, atol=1e-12)
        want = g[h] ** T * S0[:, h] + np.einsum("bjk,j,bjv->bkv", kh, w[T - 1], v[:, h])
        np.testing.assert_allclose(S[:, h], want, rtol=1e-12, atol=1e-12)


def test_decay_oracle_lengths():
    r = RNG(1)
    q, k, v = r.normal(size=(3, 3, 1, 6, 4))
    S0 = r.normal(size=(3, 1, 4, 4))
    y, S = layer.decay_attention(q, k, v, [0.8], lens=[0, 4, 6], S0=S0)
    assert not y[0].any() and not y[1, :, 4:].any()
    np.testing.assert_array_equal(S[0], S0[0])
    y4, S4 = layer.decay_attention(q[1:2, :, :4], k[1:2, :, :4], v[1:2, :, :4], [0.8], S0=S0[1:2])
    np.testing.assert_array_equal(y[1, :, :4], y4[0])
    np.testing.assert_array_equal(S[1], S4[0])


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_norm_and_linear_oracles_against_torch(act):
    import torch
    import torch.nn.functional as F
    r = RNG(2)
    x, w, b = r.normal(size=(2, 7, 12)), r.normal(size=12), r.normal(size=12)
    f = {"none": lambda a: a, "silu": F.silu, "gelu": F.gelu}[act]
    want = f(F.group_norm(torch.tensor(x).transpose(1, 2), 3, torch.tensor(w), torch.tensor(b), 1e-5))
    np.testing.assert_allclose(layer.group_norm(x, 3, w, b, act), want.transpose(1, 2).numpy(), rtol=1e-10, atol=1e-12)
    heads = x.reshape(2, 7, 3, 4).transpose(0, 2, 1, 3)          # [N, G, S, Cg]
    rows = x.reshape(14, 1, 12)
    np.testing.assert_array_equal(layer.group_norm(heads, 3, w, b, act, layout="heads"),
                                  layer.group_norm(rows, 3, w, b, act).reshape(2, 7, 12))
    W, res = r.normal(size=(12, 5)), r.normal(size=(7, 5))
    want = f(F.linear(torch.tensor(x[0]), torch.tensor(W.T), torch.tensor(b[:5]))) + torch.tensor(res)
    np.testing.assert_allclose(layer.linear(x[0], W, b[:5], res, act), want.numpy(), rtol=1e-10, atol=1e-12)


# ----------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tln.LIB_PATH):
        tln_build.build()
    return tln.load()


BAD, UNS = tln.ATLAS_ERR_INVALID_ARG, tln.ATLAS_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(H=0), BAD), (dict(d_k=0), BAD), (dict(d_v=-1), BAD), (dict(share=0), BAD), (dict(share=3), BAD),
    (dict(qkv_dtype=2), BAD), (dict(y_dtype=-1), BAD), (dict(qkv_layout=2), BAD), (dict(y_layout=7), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(d_k=257), UNS), (dict(d_v=1025), UNS),
    (dict(H=65536), UNS),
])
def test_decay_create_rejects(lib, kw, code):
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_decay_create(tln.make_decay_config(**{**dict(H=4, d_k=8, d_v=8), **kw}))
    assert ei.value.code == code and tln.atlas_decay_last_error(None)


@pytest.mark.parametrize("kw,code", [
    (dict(C=0), BAD), (dict(groups=0), BAD), (dict(groups=5), BAD), (dict(act=3), BAD), (dict(eps=0.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(x_dtype=2), BAD), (dict(y_dtype=9), BAD), (dict(layout=2), BAD),
    (dict(C=65537, groups=1), UNS), (dict(C=2048, groups=1, layout="heads"), UNS),
])
def test_norm_create_rejects(lib, kw, code):
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_norm_create(tln.make_norm_config(**{**dict(C=12, groups=3), **kw}))
    assert ei.value.code == code and tln.atlas_norm_last_error(None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), BAD), (dict(N=0), BAD), (dict(act=-1), BAD), (dict(in_dtype=2), BAD), (dict(out_dtype=2), BAD),
    (dict(K=(1 << 20) + 1), UNS), (dict(N=(1 << 20) + 1), UNS),
])
def test_linear_create_rejects(lib, kw, code):
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_linear_create(tln.make_linear_config(**{**dict(K=8, N=8), **kw}))
    assert ei.value.code == code and tln.atlas_linear_last_error(None)


def _refuses(lib, op, h, io, code, word):
    assert getattr(lib, f"atlas_{op}_forward")(h, ctypes.byref(io), None) == code
    assert word in getattr(tln, f"atlas_{op}_last_error")(h)


def test_decay_forward_validates_before_any_cuda_call(lib):
    h = tln.atlas_decay_create(tln.make_decay_config(H=4, d_k=8, d_v=8))
    assert lib.atlas_decay_forward(None, None, None) == BAD and lib.atlas_decay_forward(h, None, None) == BAD
    io = tln.atlas_decay_io(0, 5)
    _refuses(lib, "decay", h, io, BAD, "B and T")
    io.B, io.T = 1, 0
    _refuses(lib, "decay", h, io, BAD, "B and T")
    io.T = 5
    _refuses(lib, "decay", h, io, BAD, "non-NULL")
    io.q = io.k = io.v = io.decay = 64            # never dereferenced: validation fails first
    _refuses(lib, "decay", h, io, BAD, "non-NULL")
    io.y = 64
    _refuses(lib, "decay", h, io, BAD, "alias")
    io.y, io.B, io.T = 128, 1 << 20, 100
    _refuses(lib, "decay", h, io, UNS, "65535")
    assert tln.atlas_decay_last_path(h) == -1 and tln.atlas_decay_status(h) == tln.ATLAS_OK
    assert tln.atlas_decay_workspace_bytes(h, 1, 1) == 0 and tln.atlas_decay_workspace_bytes(h, 0, 1) == 0
    tln.atlas_decay_destroy(h)
    lib.atlas_decay_destroy(None)
    assert lib.atlas_decay_status(None) == BAD


def test_norm_forward_validates_before_any_cuda_call(lib):
    h = tln.atlas_norm_create(tln.make_norm_config(C=12, groups=3, layout="heads"))
    assert lib.atlas_norm_forward(None, None, None) == BAD and lib.atlas_norm_forward(h, None, None) == BAD
    io = tln.atlas_norm_io(0, 5)
    _refuses(lib, "norm", h, io, BAD, "N and S")
    io.N = 2
    _refuses(lib, "norm", h, io, BAD, "non-NULL")
    io.x = io.y = 64
    _refuses(lib, "norm", h, io, BAD, "y may be x")
    tln.atlas_norm_destroy(h)
    lib.atlas_norm_destroy(None)


def test_linear_forward_validates_before_any_cuda_call(lib):
    h = tln.atlas_linear_create(tln.make_linear_config(K=8, N=8))
    assert lib.atlas_linear_forward(None, None, None) == BAD and lib.atlas_linear_forward(h, None, None) == BAD
    io = tln.atlas_linear_io(0)
    _refuses(lib, "linear", h, io, BAD, "M must")
    io.M = 3
    _refuses(lib, "linear", h, io, BAD, "non-NULL")
    io.x = io.W = io.y = 64
    _refuses(lib, "linear", h, io, BAD, "alias")
    assert tln.atlas_linear_last_path(h) == -1 and tln.atlas_linear_status(h) == tln.ATLAS_OK
    tln.atlas_linear_destroy(h)
    lib.atlas_linear_destroy(None)


def test_sizes_beyond_a_call_are_refused(lib):
    """The documented limits, one past each."""
    lin = tln.atlas_linear_create(tln.make_linear_config(K=8, N=8))
    io = tln.atlas_linear_io(4194241)
    io.x, io.W, io.y = 64, 128, 192
    _refuses(lib, "linear", lin, io, UNS, "4194240")
    dec = tln.atlas_decay_create(tln.make_decay_config(H=4, d_k=64, d_v=64))
    io = tln.atlas_decay_io(1 << 14, 21)
    io.q = io.k = io.v = io.decay = 64
    io.y = 128
    _refuses(lib, "decay", dec, io, UNS, "at most 20 tokens")
    nrm = tln.atlas_norm_create(tln.make_norm_config(C=12, groups=3))
    io = tln.atlas_norm_io(1 << 15, 1 << 14)
    io.x, io.y = 64, 128
    _refuses(lib, "norm", nrm, io, UNS, "2^30")
    tln.atlas_linear_destroy(lin)
    tln.atlas_decay_destroy(dec)
    tln.atlas_norm_destroy(nrm)


def test_runner_refuses_wrong_tensors(lib):
    import torch
    from test_learned_neural_gb300.runner import DecayAttention, GroupNorm, Linear
    z = torch.zeros
    lin, nrm, dec = Linear(8, 4), GroupNorm(8, 2), DecayAttention(2, 4, 4)
    for t in (dict(x=z(3, 8), W=z(8, 4)),                                         # fp32 for bf16
              dict(x=z(3, 8).bfloat16(), W=z(8, 4).bfloat16())):                  # host tensors
        with pytest.raises(ValueError):
            lin.forward(t, out=dict(y=z(3, 4).bfloat16()))
    with pytest.raises(ValueError):
        nrm.forward(dict(x=z(2, 3, 9).bfloat16()), out=dict(y=z(2, 3, 8).bfloat16()))
    with pytest.raises(ValueError):
        dec.forward(dict(q=z(1, 2, 5, 4).bfloat16(), k=z(1, 2, 5, 4), v=z(1, 2, 5, 4), decay=z(2)),
                    out=dict(y=None, S=None))
