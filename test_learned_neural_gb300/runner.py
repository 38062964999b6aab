"""Tensor marshalling around the C entry points for whole workloads.

``Memory`` owns one library handle for a memory configuration; ``forward``
takes torch tensors (device or pinned host) in the layouts of
include/atlas_mem.h and returns the outputs.  No arithmetic of the method
happens here.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (ATLAS_BF16, ATLAS_F32, ATLAS_LAYOUT_HEADS, ATLAS_NORM_HEADS, atlas_decay_create, atlas_decay_destroy,
               atlas_decay_forward, atlas_decay_io, atlas_decay_last_path, atlas_decay_status, atlas_linear_create,
               atlas_linear_destroy, atlas_linear_forward, atlas_linear_io, atlas_linear_last_path,
               atlas_linear_status, atlas_mem_create, atlas_mem_destroy, atlas_mem_forward,
               atlas_mem_forward_host, atlas_mem_status, atlas_norm_create, atlas_norm_destroy, atlas_norm_forward,
               atlas_norm_io, atlas_prologue_create, atlas_prologue_destroy,
               atlas_prologue_forward, atlas_prologue_io, atlas_prologue_last_gemm, atlas_prologue_status,
               current_stream, make_config, make_decay_config, make_io, make_linear_config, make_norm_config,
               make_prologue_config, AtlasError)


def matrix_shapes(cfg):
    F = cfg.proj_dim if cfg.proj_dim else (cfg.d_k if cfg.p == 1 else (cfg.d_k + 1) * (cfg.d_k + 2) // 2)
    if cfg.depth == 1:
        return [(F, cfg.d_v)]
    return [(F, cfg.hidden), (cfg.hidden, cfg.d_v)]


class Memory:
    """A configured memory layer (one library handle)."""

    def __init__(self, cfg):
        self.cfg = cfg
        self.shapes = matrix_shapes(cfg)
        self.qkv_torch = torch.float32 if cfg.qkv_dtype in ("f32", ATLAS_F32) else torch.bfloat16
        self.h = atlas_mem_create(make_config(cfg.depth, cfg.d_k, cfg.d_v, cfg.hidden if cfg.depth == 2 else 0,
                                              cfg.C, cfg.c, cfg.p, cfg.proj_dim, cfg.ns_iters, cfg.qkv_dtype,
                                              getattr(cfg, "readout", "post"),
                                              getattr(cfg, "ns_target", "momentum"),
                                              getattr(cfg, "update", "per_token")))

    def close(self):
        if self.h is not None:
            atlas_mem_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_outputs(self, B, H, T, device):
        f32 = torch.float32
        out = dict(
            y=torch.empty((B, H, T, self.cfg.d_v), dtype=f32, device=device),
            W=[torch.empty((B, H, r, c), dtype=f32, device=device) for r, c in self.shapes],
            S=[torch.empty((B, H, r, c), dtype=f32, device=device) for r, c in self.shapes],
        )
        nc = max(self.cfg.c - 1, 0)
        if nc:
            out["win_k"] = torch.zeros((B, H, nc, self.cfg.d_k), dtype=self.qkv_torch, device=device)
            out["win_v"] = torch.zeros((B, H, nc, self.cfg.d_v), dtype=self.qkv_torch, device=device)
            out["win_gamma"] = torch.zeros((B, H, nc), dtype=f32, device=device)
        return out

    def forward(self, t, out=None, win=None, host=False, stream=None):
        """t: dict of tensors (q, k, v, theta, eta, alpha, gamma, P, W0, S0);
        win: optional (win_len, win_k, win_v, win_gamma).  Returns the outputs."""
        B, H, T = t["q"].shape[:3]
        dev = "cpu" if host else t["q"].device
        if out is None:
            out = self.alloc_outputs(B, H, T, dev)
            if host:
                for key, val in list(out.items()):
                    out[key] = [x.pin_memory() for x in val] if isinstance(val, list) else val.pin_memory()
        win_len, wk, wv, wg = win if win is not None else (0, None, None, None)
        io = make_io(B, H, T, t["q"], t["k"], t["v"], t["theta"], t["eta"], t["alpha"], t.get("gamma"),
                     t.get("P"), t["W0"], t["S0"], out["y"], out["W"], out["S"],
                     win_len=win_len, win_k=wk, win_v=wv, win_gamma=wg,
                     win_k_out=out.get("win_k"), win_v_out=out.get("win_v"), win_gamma_out=out.get("win_gamma"))
        s = current_stream() if stream is None else stream
        if host:
            atlas_mem_forward_host(self.h, io, s)
        else:
            atlas_mem_forward(self.h, io, s)
        return out

    def status(self):
        rc = atlas_mem_status(self.h)
        if rc:
            raise AtlasError(rc, "device status")
        return rc


def tensors_from_numpy(inp: dict, device="cuda", pin=False):
    """Harness-style numpy inputs (bf16 as uint16 bit patterns) -> torch."""
    def conv(a):
        if a is None:
            return None
        a = np.ascontiguousarray(a)
        if a.dtype == np.uint16:
            t = torch.from_numpy(a.view(np.int16)).view(torch.bfloat16)
        else:
            t = torch.from_numpy(a)
        if device == "cpu":
            return t.pin_memory() if pin else t
        return t.to(device, non_blocking=False)

    out = {k: conv(inp[k]) for k in ("q", "k", "v", "theta", "eta", "alpha", "gamma", "P")}
    out["W0"] = [conv(m) for m in inp["W0"]]
    out["S0"] = [conv(m) for m in inp["S0"]]
    return out


class Prologue:
    """A configured stage in front of the memory (one library handle):
    x [B, T, D] -> q, k, v [B, H, T, d] and the gates [B, H, T]."""

    def __init__(self, cfg):
        self.cfg = cfg
        self.qkv_torch = torch.float32 if cfg.qkv_dtype in ("f32", ATLAS_F32) else torch.bfloat16
        self.h = atlas_prologue_create(make_prologue_config(cfg.D, cfg.H, cfg.d_k, cfg.d_v, cfg.conv,
                                                            cfg.with_gamma, cfg.theta_max, cfg.qkv_dtype))

    def close(self):
        if self.h is not None:
            atlas_prologue_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_outputs(self, B, T, device):
        c, f32 = self.cfg, torch.float32
        out = dict(q=torch.empty((B, c.H, T, c.d_k), dtype=self.qkv_torch, device=device),
                   k=torch.empty((B, c.H, T, c.d_k), dtype=self.qkv_torch, device=device),
                   v=torch.empty((B, c.H, T, c.d_v), dtype=self.qkv_torch, device=device))
        for g in ("theta", "eta", "alpha") + (("gamma",) if c.with_gamma else ()):
            out[g] = torch.empty((B, c.H, T), dtype=f32, device=device)
        if c.conv > 1:
            out["cache"] = torch.empty((B, c.conv - 1, c.Nc), dtype=f32, device=device)
        return out

    def forward(self, t, out=None, stream=None):
        """t: dict of device tensors x, W_in, conv_w, gate_b and optional cache."""
        B, T = t["x"].shape[:2]
        if out is None:
            out = self.alloc_outputs(B, T, t["x"].device)

        def ptr(a):
            return None if a is None else a.data_ptr()

        io = atlas_prologue_io(B, T, ptr(t["x"]), ptr(t["W_in"]), ptr(t["conv_w"]), ptr(t["gate_b"]),
                               ptr(t.get("cache")), ptr(out["q"]), ptr(out["k"]), ptr(out["v"]), ptr(out["theta"]),
                               ptr(out["eta"]), ptr(out["alpha"]), ptr(out.get("gamma")), ptr(out.get("cache")))
        atlas_prologue_forward(self.h, io, current_stream() if stream is None else stream)
        return out

    def status(self):
        rc = atlas_prologue_status(self.h)
        if rc:
            raise AtlasError(rc, "device status of the stage in front of the memory")
        return rc

    def last_gemm(self):
        """1: the projection ran on the tensor cores (TMA + tcgen05), 0: fp32 SIMT."""
        return atlas_prologue_last_gemm(self.h)


def prologue_tensors_from_numpy(inp: dict, device="cuda"):
    """Seeded prologue inputs (bf16 as uint16 bit patterns) -> torch."""
    def conv(a):
        if a is None:
            return None
        a = np.ascontiguousarray(a)
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
        return torch.from_numpy(a).to(device)
    return {k: conv(inp.get(k)) for k in ("x", "W_in", "conv_w", "gate_b", "cache")}


def _torch_dtype(t):
    return torch.bfloat16 if t == ATLAS_BF16 else torch.float32


def _check(name, t, dtype, shape, device):
    """Device address of a tensor of the layer operators, which must have the
    type and shape that the configuration and the call's sizes give, and lie
    on the call's device (its index; None: there is only one)."""
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda
            or device is not None and t.get_device() != device):
        raise ValueError(f"{name}: want a contiguous CUDA tensor {dtype} {shape} on one device with the others, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


# The current stream's handle of a device: torch.cuda.current_stream() builds a
# Python object for it, 3 us of a serving step's 10 on the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_devices = None


def _device_of(t):
    """Index of a tensor's device; None where there is only one, so that the
    checks of a serving step's tensors cost nothing there (else 1 us of 7)."""
    global _devices
    if _devices is None:
        _devices = torch.cuda.device_count()
    return t.get_device() if _devices > 1 else None


def _stream_of(device, stream):
    """The stream of a call whose tensors are on `device`.  The kernels go to
    the current device: any other would read the tensors' addresses as its own."""
    if device is None:
        return _raw_stream(0) if stream is None else stream
    now = _current_device()
    if now != device:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{now}: make the call under "
                         f"torch.cuda.device({device})")
    return _raw_stream(device) if stream is None else stream


class _Layer:
    """One library handle of a layer operator."""
    _destroy = None
    h = None

    def close(self):
        if self.h is not None:
            type(self)._destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DecayAttention(_Layer):
    """Linear attention with a decay for each head (include/atlas_decay.h):
    S_t = g S_{t-1} + k_t^T v_t, y_t = scale q_t S_t."""
    _destroy = staticmethod(atlas_decay_destroy)

    def __init__(self, H, d_k, d_v, share=1, qkv_dtype="bf16", y_dtype=None, qkv_layout="heads", y_layout="heads",
                 scale=1.0):
        self.cfg = make_decay_config(H, d_k, d_v, share, qkv_dtype, y_dtype, qkv_layout, y_layout, scale)
        self.h = atlas_decay_create(self.cfg)
        c = self.cfg
        self._qkv, self._y = _torch_dtype(c.qkv_dtype), _torch_dtype(c.y_dtype)
        self._heads_first, self._y_heads_first = c.qkv_layout == ATLAS_LAYOUT_HEADS, c.y_layout == ATLAS_LAYOUT_HEADS

    def _y_shape(self, B, T):
        c = self.cfg
        return (B, c.H, T, c.d_v) if self._y_heads_first else (B, T, c.H, c.d_v)

    def alloc_outputs(self, B, T, device):
        c = self.cfg
        return dict(y=torch.empty(self._y_shape(B, T), dtype=self._y, device=device),
                    S=torch.empty((B, c.H, c.d_k, c.d_v), dtype=torch.float32, device=device))

    def forward(self, t, out=None, stream=None):
        """t: dict of device tensors q, k, v, decay and optional lens (int32
        [B]) and S0 (fp32 [B, H, d_k, d_v]; may be out["S"]: the state is then
        continued in place)."""
        c, q, v = self.cfg, t["q"], t["v"]
        B, T = (q.shape[0], q.shape[2]) if self._heads_first else q.shape[:2]
        hq = c.H // c.share
        qs, vs = ((B, hq, T, c.d_k), (B, c.H, T, c.d_v)) if self._heads_first else (
            (B, T, hq, c.d_k), (B, T, c.H, c.d_v))
        if out is None:
            out = self.alloc_outputs(B, T, q.device)
        lens, S0, sq, f32, dev = t.get("lens"), t.get("S0"), (B, c.H, c.d_k, c.d_v), torch.float32, _device_of(q)
        io = atlas_decay_io(B, T, _check("q", q, self._qkv, qs, dev), _check("k", t["k"], self._qkv, qs, dev),
                            _check("v", v, self._qkv, vs, dev), _check("decay", t["decay"], f32, (c.H,), dev),
                            None if lens is None else _check("lens", lens, torch.int32, (B,), dev),
                            None if S0 is None else _check("S0", S0, f32, sq, dev),
                            _check("y", out["y"], self._y, self._y_shape(B, T), dev),
                            _check("S", out["S"], f32, sq, dev))
        atlas_decay_forward(self.h, io, _stream_of(dev, stream))
        return out

    def status(self):
        rc = atlas_decay_status(self.h)
        if rc:
            raise AtlasError(rc, "device status of the decay attention")
        return rc

    def last_path(self):
        """0: token by token, 1: fp32 chunks, 2: tensor-core chunks."""
        return atlas_decay_last_path(self.h)


class GroupNorm(_Layer):
    """Group norm with an activation, channels last (include/atlas_norm.h).
    layout "heads": x is a read-out [N, groups, S, C / groups], y [N, S, C]."""
    _destroy = staticmethod(atlas_norm_destroy)

    def __init__(self, C, groups, act="none", eps=1e-5, x_dtype="bf16", y_dtype=None, layout="channels_last"):
        self.cfg = make_norm_config(C, groups, act, eps, x_dtype, y_dtype, layout)
        self.h = atlas_norm_create(self.cfg)
        self._x, self._y = _torch_dtype(self.cfg.x_dtype), _torch_dtype(self.cfg.y_dtype)

    def alloc_outputs(self, N, S, device):
        return dict(y=torch.empty((N, S, self.cfg.C), dtype=self._y, device=device))

    def forward(self, t, out=None, stream=None):
        """t: dict of device tensors x and optional weight, bias (fp32 [C])."""
        c, x = self.cfg, t["x"]
        if c.layout == ATLAS_NORM_HEADS:
            N, S = x.shape[0], x.shape[2]
            shape = (N, c.groups, S, c.C // c.groups)
        else:
            N, S = x.shape[:2]
            shape = (N, S, c.C)
        if out is None:
            out = self.alloc_outputs(N, S, x.device)
        w, b, f32, dev = t.get("weight"), t.get("bias"), torch.float32, _device_of(x)
        io = atlas_norm_io(N, S, _check("x", x, self._x, shape, dev),
                           None if w is None else _check("weight", w, f32, (c.C,), dev),
                           None if b is None else _check("bias", b, f32, (c.C,), dev),
                           _check("y", out["y"], self._y, (N, S, c.C), dev))
        atlas_norm_forward(self.h, io, _stream_of(dev, stream))
        return out


class Linear(_Layer):
    """y = act(x W + bias) + residual (include/atlas_linear.h)."""
    _destroy = staticmethod(atlas_linear_destroy)

    def __init__(self, K, N, act="none", in_dtype="bf16", out_dtype=None):
        self.cfg = make_linear_config(K, N, act, in_dtype, out_dtype)
        self.h = atlas_linear_create(self.cfg)
        self._in, self._out = _torch_dtype(self.cfg.in_dtype), _torch_dtype(self.cfg.out_dtype)

    def alloc_outputs(self, M, device):
        return dict(y=torch.empty((M, self.cfg.N), dtype=self._out, device=device))

    def forward(self, t, out=None, stream=None):
        """t: dict of device tensors x [M, K], W [K, N] and optional bias
        (fp32 [N]) and residual [M, N] (may be out["y"]: added in place)."""
        c, x = self.cfg, t["x"]
        M = x.shape[0]
        if out is None:
            out = self.alloc_outputs(M, x.device)
        b, r, dev = t.get("bias"), t.get("residual"), _device_of(x)
        io = atlas_linear_io(M, _check("x", x, self._in, (M, c.K), dev), _check("W", t["W"], self._in, (c.K, c.N), dev),
                             None if b is None else _check("bias", b, torch.float32, (c.N,), dev),
                             None if r is None else _check("residual", r, self._out, (M, c.N), dev),
                             _check("y", out["y"], self._out, (M, c.N), dev))
        atlas_linear_forward(self.h, io, _stream_of(dev, stream))
        return out

    def status(self):
        rc = atlas_linear_status(self.h)
        if rc:
            raise AtlasError(rc, "device status of the matrix product")
        return rc

    def last_path(self):
        """1: tensor cores, 2: few rows."""
        return atlas_linear_last_path(self.h)
