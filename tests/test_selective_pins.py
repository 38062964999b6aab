"""CPU checks of the selective layer's operators: the fp64 oracle against closed
forms and torch, and what the C entry points and the binding refuse before any
CUDA call."""
import numpy as np
import pytest

import test_learned_neural_gb300 as tln
from oracle import layer
from tests.test_layer_pins import BAD, UNS, _refuses, lib  # noqa: F401

RNG = np.random.default_rng


# --------------------------------------------------------------- the oracle
@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_oracle_is_torchs_convolution(K):
    import torch
    import torch.nn.functional as F
    r = RNG(0)
    x, w, b = r.normal(size=(2, 9, 5)), r.normal(size=(5, K)), r.normal(size=5)
    y, keep = layer.short_conv(x, w, b, act="silu")
    pad = F.pad(torch.tensor(x).transpose(1, 2), (K - 1, 0))
    want = F.silu(F.conv1d(pad, torch.tensor(w)[:, None], torch.tensor(b), groups=5))
    np.testing.assert_allclose(y, want.transpose(1, 2).numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(keep, x[:, 9 - (K - 1):])


def test_conv_oracle_cut_and_lengths():
    r = RNG(1)
    x, w, c = r.normal(size=(3, 6, 4)), r.normal(size=(4, 4)), r.normal(size=(3, 3, 4))
    y, keep = layer.short_conv(x, w, cache=c)
    y1, k1 = layer.short_conv(x[:, :2], w, cache=c)
    y2, k2 = layer.short_conv(x[:, 2:], w, cache=k1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-12)
    np.testing.assert_array_equal(k2, keep)
    yr, kr = layer.short_conv(x, w, cache=c, lens=[0, 2, 6])
    np.testing.assert_array_equal(kr[0], c[0])
    np.testing.assert_array_equal(kr[1], k1[1])
    assert not yr[0].any() and not yr[1, 2:].any()


def test_rms_oracle_and_scales():
    import torch
    r = RNG(2)
    x, res, w = r.normal(size=(4, 300)), r.normal(size=(4, 300)), r.normal(size=300)
    y, h = layer.rms_norm(x, res, w, 1e-5)
    want = torch.nn.functional.rms_norm(torch.tensor(x + res), (300,), torch.tensor(w), 1e-5)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-12)
    s = layer.e4m3_scales(y, 128)
    assert s.shape == (4, 3) and s[2, 2] == np.abs(y[2, 256:]).max() / 448
    assert layer.e4m3_scales(0 * y, 0).tolist() == [[2.0 ** -100 / 448]] * 4


def test_quant_weights_by_hand():
    q = np.array([[0x1f, 0x80], [0x07, 0x9a]], np.uint8)          # K = 3: the last high half is not looked at
    W = layer.quant_weights(q, np.array([[0.5, 2.0]]), None, 3, 32)
    np.testing.assert_array_equal(W, [[3.5, -16.0], [-3.5, 0.0], [-0.5, 4.0]])
    W = layer.quant_weights(q, np.array([[0.5, 2.0]]), np.array([[15, 0]], np.uint8), 3, 32)
    np.testing.assert_array_equal(W, [[0.0, 0.0], [-7.0, 16.0], [-4.0, 20.0]])
    y = layer.quant_linear([[1.0, 2.0, 4.0]], W, [[10.0]], 0)
    np.testing.assert_array_equal(y, [[10 * (-14 - 16), 10 * (32 + 80)]])


@pytest.mark.parametrize("share", [1, 2])
def test_scan_oracle_is_the_sum_over_past_tokens(share):
    r = RNG(3)
    B, H, T, dk, dv = 2, 4, 7, 3, 5
    q, k = r.normal(size=(2, B, H // share, T, dk))
    v, S0, D = r.normal(size=(B, H, T, dv)), r.normal(size=(B, H, dk, dv)), r.normal(size=H)
    s, g = layer.step_gates(r.normal(size=(B, H, T)), r.normal(size=H), -np.exp(r.normal(size=H)))
    y, S = layer.selective_scan(q, k, v, s, g, D, S0=S0, scale=0.7)
    for b in range(B):
        for h in range(H):
            for t in range(T):
                past = sum(np.prod(g[b, h, j + 1:t + 1]) * s[b, h, j] * (q[b, h // share, t] @ k[b, h // share, j]) * v[b, h, j]
                           for j in range(t + 1))
                past = past + np.prod(g[b, h, :t + 1]) * (q[b, h // share, t] @ S0[b, h])
                np.testing.assert_allclose(y[b, h, t], 0.7 * past + D[h] * v[b, h, t], rtol=1e-10, atol=1e-12)
    const = layer.selective_scan(q, k, v, np.ones((B, H, T)), np.full((B, H, T), 0.8))
    want = layer.decay_attention(q, k, v, np.full(H, 0.8))
    np.testing.assert_allclose(const[0], want[0], rtol=1e-12)
    np.testing.assert_allclose(const[1], want[1], rtol=1e-12)


# ----------------------------------------------------------------- refusals
@pytest.mark.parametrize("kw,code", [
    (dict(C=0), BAD), (dict(K=0), BAD), (dict(act=3), BAD), (dict(dtype=2), BAD), (dict(K=9), UNS), (dict(C=(1 << 20) + 1), UNS)])
def test_conv_create_rejects(lib, kw, code):  # noqa: F811
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_conv_create(tln.make_conv_config(**{**dict(C=8, K=4), **kw}))
    assert ei.value.code == code and tln.atlas_conv_last_error(None)


@pytest.mark.parametrize("kw,code", [
    (dict(C=0), BAD), (dict(eps=0.0), BAD), (dict(eps=float("inf")), BAD), (dict(eps=float("nan")), BAD), (dict(x_dtype=2), BAD),
    (dict(residual_dtype=2), BAD), (dict(y_dtype=3), BAD), (dict(block=128), BAD), (dict(y_dtype="e4m3", block=64), BAD),
    (dict(C=32769), UNS)])
def test_rms_create_rejects(lib, kw, code):  # noqa: F811
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_rms_create(tln.make_rms_config(**{**dict(C=8), **kw}))
    assert ei.value.code == code and tln.atlas_rms_last_error(None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), BAD), (dict(N=0), BAD), (dict(group=16), BAD), (dict(group=0), BAD), (dict(zeros=2), BAD), (dict(act=-1), BAD),
    (dict(x_dtype=3), BAD), (dict(x_block=128), BAD), (dict(x_dtype="e4m3", x_block=32), BAD), (dict(out_dtype=2), BAD),
    (dict(K=(1 << 20) + 1), UNS), (dict(N=(1 << 20) + 1), UNS)])
def test_qlinear_create_rejects(lib, kw, code):  # noqa: F811
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_qlinear_create(tln.make_qlinear_config(**{**dict(K=8, N=8), **kw}))
    assert ei.value.code == code and tln.atlas_qlinear_last_error(None)


def test_conv_forward_validates_before_any_cuda_call(lib):  # noqa: F811
    h = tln.atlas_conv_create(tln.make_conv_config(8, 4))
    assert lib.atlas_conv_forward(None, None, None) == BAD and lib.atlas_conv_forward(h, None, None) == BAD
    io = tln.atlas_conv_io(0, 5)
    _refuses(lib, "conv", h, io, BAD, "B and T")
    io.B = 2
    _refuses(lib, "conv", h, io, BAD, "non-NULL")
    io.x, io.w, io.y, io.ld_x = 1 << 20, 1 << 10, 1 << 21, 7         # never dereferenced: validation fails first
    _refuses(lib, "conv", h, io, BAD, "ld_x")
    io.ld_x = 16
    io.y = (1 << 20) + (2 * 5 - 1) * 32 + 8                          # inside x's last row
    _refuses(lib, "conv", h, io, BAD, "overlap")
    io.y, io.cache, io.cache_out = 1 << 21, 1 << 22, (1 << 22) + 16   # a shifted cache
    _refuses(lib, "conv", h, io, BAD, "cache itself")
    io.cache_out = (1 << 21) + 32
    _refuses(lib, "conv", h, io, BAD, "overlap")
    io.cache_out, io.T = None, (1 << 30) + 1
    _refuses(lib, "conv", h, io, UNS, "2^30")
    tln.atlas_conv_destroy(h)
    lib.atlas_conv_destroy(None)


def test_rms_forward_validates_before_any_cuda_call(lib):  # noqa: F811
    h = tln.atlas_rms_create(tln.make_rms_config(16, y_dtype="e4m3", block=128))
    assert lib.atlas_rms_forward(None, None, None) == BAD and lib.atlas_rms_forward(h, None, None) == BAD
    io = tln.atlas_rms_io(0)
    _refuses(lib, "rms", h, io, BAD, "M must")
    io.M = 3
    _refuses(lib, "rms", h, io, BAD, "non-NULL")
    io.x, io.y = 1 << 20, 1 << 21
    _refuses(lib, "rms", h, io, BAD, "scale goes with")
    io.scale, io.y = 1 << 22, 1 << 20
    _refuses(lib, "rms", h, io, BAD, "y may be x")
    io.y, io.h, io.residual = 1 << 21, (1 << 23) + 32, 1 << 23
    _refuses(lib, "rms", h, io, BAD, "h may be")
    io.h, io.scale = 1 << 23, (1 << 23) + 4
    _refuses(lib, "rms", h, io, BAD, "scale must not")
    tln.atlas_rms_destroy(h)
    h = tln.atlas_rms_create(tln.make_rms_config(16))
    _refuses(lib, "rms", h, io, BAD, "scale goes with")
    tln.atlas_rms_destroy(h)
    lib.atlas_rms_destroy(None)


def test_qlinear_validates_before_any_cuda_call(lib):  # noqa: F811
    h = tln.atlas_qlinear_create(tln.make_qlinear_config(100, 40, group=32, zeros=True, x_dtype="e4m3"))
    assert lib.atlas_qlinear_forward(None, None, None) == BAD and lib.atlas_qlinear_forward(h, None, None) == BAD
    io = tln.atlas_qlinear_io(0)
    _refuses(lib, "qlinear", h, io, BAD, "M must")
    io.M = 3
    _refuses(lib, "qlinear", h, io, BAD, "non-NULL")
    io.x, io.y, io.W = 1 << 20, 1 << 21, (1 << 22) + 8
    _refuses(lib, "qlinear", h, io, BAD, "x_scale goes with")
    io.x_scale = 1 << 23
    _refuses(lib, "qlinear", h, io, BAD, "aligned")
    io.W, io.residual = 1 << 22, (1 << 21) + 2
    _refuses(lib, "qlinear", h, io, BAD, "residual itself")
    io.residual, io.M = None, 4194241
    _refuses(lib, "qlinear", h, io, UNS, "4194240")
    # a block of 128 columns by 128 of K: codes, four groups of scales and zero points
    assert tln.atlas_qlinear_packed_bytes(h) == 128 * 64 + 4 * 128 * 2 + 4 * 64
    assert tln.atlas_qlinear_workspace_bytes(h, 3) == 8 * 128 * 2 and tln.atlas_qlinear_workspace_bytes(h, 0) == 0
    Q, P = lib.atlas_qlinear_quantize, lib.atlas_qlinear_pack
    assert Q(None, 64, 0, 64, 64, 64, None) == BAD and P(None, 64, 64, 64, 64, None) == BAD
    for args in ((None, 0, 64, 1 << 20, 1 << 21), (1 << 30, 2, 64, 1 << 20, 1 << 21), (1 << 30, 0, 64, 1 << 20, None),
                 (1 << 20, 0, 64, (1 << 20) + 100, 1 << 25)):
        assert Q(h, *args, None) == BAD and tln.atlas_qlinear_last_error(h)
    f32 = tln.atlas_qlinear_create(tln.make_qlinear_config(100, 40, x_dtype="f32"))
    io = tln.atlas_qlinear_io(2097121)
    io.x, io.y, io.W = 1 << 40, 1 << 41, 1 << 42
    _refuses(lib, "qlinear", f32, io, UNS, "2097120")
    tln.atlas_qlinear_destroy(f32)
    for args in ((64, 1 << 20, 1 << 21, None), (64, 1 << 20, None, 1 << 22), (64, 1 << 20, 1 << 21, (1 << 22) + 4),
                 (1 << 22, 1 << 20, 1 << 21, 1 << 22)):
        assert P(h, *args, None) == BAD and tln.atlas_qlinear_last_error(h)
    assert tln.atlas_qlinear_status(h) == tln.ATLAS_OK and lib.atlas_qlinear_status(None) == BAD
    tln.atlas_qlinear_destroy(h)
    lib.atlas_qlinear_destroy(None)


def test_runner_refuses_wrong_tensors(lib):  # noqa: F811
    import torch
    from test_learned_neural_gb300.runner import QuantLinear, RmsNorm, ShortConv
    z = torch.zeros
    with pytest.raises(ValueError):
        ShortConv(8, 4).forward(dict(x=z(1, 5, 8).bfloat16(), w=z(8, 4)), out=dict(y=z(1, 5, 8).bfloat16(), cache=None))
    with pytest.raises(ValueError):
        RmsNorm(8).forward(dict(x=z(3, 9).bfloat16()), out=dict(y=z(3, 8).bfloat16()))
    with pytest.raises(ValueError):
        QuantLinear(8, 4).forward(dict(x=z(3, 8).bfloat16(), W=z(10)), out=dict(y=z(3, 4).bfloat16()))
    with pytest.raises(ValueError):
        QuantLinear(8, 4).quantize(z(8, 4).half())


class Strided:
    """A tensor on a device that this machine need not have, with strides."""

    def __init__(self, shape, stride):
        import torch
        self.shape, self._stride, self.dtype, self.is_cuda, self.device = shape, stride, torch.bfloat16, True, "cuda"

    def is_contiguous(self):
        return False

    def stride(self):
        return self._stride

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("shape,stride,ld", [
    ((2, 5, 8), (100, 20, 1), 20), ((2, 1, 8), (20, 999, 1), 20), ((1, 5, 8), (7, 20, 1), 20), ((1, 1, 8), (3, 2, 1), 8),
    ((2, 5, 3, 4), (100, 20, 4, 1), 20), ((2, 5, 1, 4), (100, 20, 77, 1), 20)])
def test_rows_inside_wider_ones(shape, stride, ld):
    from test_learned_neural_gb300 import runner
    import torch
    assert runner._check_rows("x", Strided(shape, stride), torch.bfloat16, shape, None) == (1 << 20, ld)


@pytest.mark.parametrize("shape,stride", [
    ((2, 5, 8), (100, 20, 2)), ((2, 5, 8), (99, 20, 1)), ((2, 5, 8), (40, 4, 1)), ((2, 5, 3, 4), (100, 20, 5, 1)),
    ((2, 5, 8), (0, 0, 1)), ((2, 5, 8), (5 << 31, 1 << 31, 1))])
def test_other_strides_are_refused(shape, stride):
    from test_learned_neural_gb300 import runner
    import torch
    with pytest.raises(ValueError, match="slice"):
        runner._check_rows("x", Strided(shape, stride), torch.bfloat16, shape, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=0), BAD), (dict(d_k=0), BAD), (dict(d_v=-1), BAD), (dict(share=3), BAD), (dict(gates=2), BAD), (dict(qkv_dtype=2), BAD),
    (dict(y_dtype=2), BAD), (dict(qkv_layout=2), BAD), (dict(y_layout=-1), BAD), (dict(scale=float("nan")), BAD), (dict(d_k=257), UNS),
    (dict(d_v=1025), UNS), (dict(H=65536), UNS)])
def test_scan_create_rejects(lib, kw, code):  # noqa: F811
    with pytest.raises(tln.AtlasError) as ei:
        tln.atlas_scan_create(tln.make_scan_config(**{**dict(H=4, d_k=8, d_v=8), **kw}))
    assert ei.value.code == code and tln.atlas_scan_last_error(None)


def test_scan_forward_validates_before_any_cuda_call(lib):  # noqa: F811
    h = tln.atlas_scan_create(tln.make_scan_config(4, 8, 8, gates="memory", qkv_layout="tokens"))
    assert lib.atlas_scan_forward(None, None, None) == BAD and lib.atlas_scan_forward(h, None, None) == BAD
    io = tln.atlas_scan_io(0, 5)
    _refuses(lib, "scan", h, io, BAD, "B and T")
    io.B = 2
    _refuses(lib, "scan", h, io, BAD, "non-NULL")
    io.q, io.k, io.v, io.step, io.y = (i << 20 for i in range(1, 6))     # never dereferenced: validation fails first
    _refuses(lib, "scan", h, io, BAD, "takes alpha")
    io.alpha = io.A = 6 << 20
    _refuses(lib, "scan", h, io, BAD, "takes alpha")
    io.A = None
    for name, value in (("ld_qk", 31), ("ld_v", 31), ("ld_gates", 3)):
        setattr(io, name, value)
        _refuses(lib, "scan", h, io, BAD, "at least")
        setattr(io, name, 0)
    io.ld_v, io.y = 100, (3 << 20) + 9 * 200 + 60                        # the last token's values
    _refuses(lib, "scan", h, io, BAD, "y must not")
    io.y, io.S_out = 5 << 20, 6 << 20
    _refuses(lib, "scan", h, io, BAD, "S_out")
    io.S0, io.S_out = 7 << 20, (7 << 20) + 4
    _refuses(lib, "scan", h, io, BAD, "S_out")
    io.S_out, io.T = None, (1 << 30) + 1
    _refuses(lib, "scan", h, io, UNS, "2^30")
    io.T, io.B, io.S0 = 50, 1 << 14, None
    for i, n in enumerate(("q", "k", "v", "step", "alpha", "y")):
        setattr(io, n, (i + 1) << 40)
    _refuses(lib, "scan", h, io, UNS, "65535")
    assert tln.atlas_scan_last_path(h) == -1 and tln.atlas_scan_status(h) == tln.ATLAS_OK
    assert tln.atlas_scan_workspace_bytes(h, 1, 1) == 0 and tln.atlas_scan_workspace_bytes(h, 0, 1) == 0
    assert tln.atlas_scan_workspace_bytes(h, 1, 100000) >= 4 * 2 * 8 * 8 * 4      # states at the segments' starts
    tln.atlas_scan_destroy(h)
    h = tln.atlas_scan_create(tln.make_scan_config(4, 8, 8, gates="step"))
    io = tln.atlas_scan_io(1, 5)
    io.q, io.k, io.v, io.step, io.y = (i << 20 for i in range(1, 6))
    _refuses(lib, "scan", h, io, BAD, "ATLAS_GATES_STEP A")
    io.A, io.ld_qk = 6 << 20, 40
    _refuses(lib, "scan", h, io, BAD, "ATLAS_LAYOUT_TOKENS")
    tln.atlas_scan_destroy(h)
    lib.atlas_scan_destroy(None)
    assert lib.atlas_scan_status(None) == BAD
