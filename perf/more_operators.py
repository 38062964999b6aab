"""Cases of the operators of a selective layer around a plain matrix memory:
the scan whose decay and step come with every token, its short causal
convolution, the root-mean-square norm with the residual's addition, and the
matrix product with 4-bit weights.

`listed()` and `draw()` give cases, `prepare()` their inputs, `run()` one pass:
through the library's entry points where `own` is true, else in plain torch
(fp32 whatever the inputs' type, the decays' sums in 64 bits, rounded once at
the end).  `exact()` gives the same outputs in 64 bits from the operators'
definitions.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def _scan(B, H, T, d_k, d_v, gates="memory", dtype="bf16", y="bf16", share=1, ragged=False, layout="heads",
          y_layout="heads", state=True, skip=False):
    return dict(op="scan", B=B, H=H, T=T, d_k=d_k, d_v=d_v, gates=gates, dtype=dtype, y=y, share=share, ragged=ragged,
                layout=layout, y_layout=y_layout, state=state, skip=skip)


def _conv(B, T, C, K=4, act="silu", dtype="bf16", bias=True, extra=0, ragged=False, cache=True):
    return dict(op="conv", B=B, T=T, C=C, K=K, act=act, dtype=dtype, bias=bias, extra=extra, ragged=ragged, cache=cache)


def _rms(M, C, x="bf16", y="bf16", residual="bf16", block=0, affine=True):
    return dict(op="rms", M=M, C=C, x=x, y=y, residual=residual, block=block, affine=affine)


def _qlinear(M, K, N, group=128, zeros=False, act="none", x="bf16", x_block=0, out="bf16", bias=False, residual=False):
    return dict(op="qlinear", M=M, K=K, N=N, group=group, zeros=zeros, act=act, x=x, x_block=x_block, out=out,
                bias=bias, residual=residual)


def listed():
    return [
        # one token for many sequences, two heads' widths of a state-space layer: all time goes to the states
        dict(_scan(256, 16, 1, 128, 64, "step", share=16, layout="tokens", y_layout="tokens", skip=True),
             name="scan_step_many"),
        # a batch of prompts of the Titans workload's shape behind the stage in front of the memory, tokens first
        # for the head norm behind it
        dict(_scan(4, 8, 4096, 64, 64, y_layout="tokens", state=False), name="scan_prompt"),
        # ragged prompts at a state-space layer's widths: one query/key head for all, rows of the convolution's output
        dict(_scan(2, 16, 8192, 128, 64, "step", share=16, ragged=True, layout="tokens", y_layout="tokens", skip=True),
             name="scan_wide"),
        # the long-context workload's shape in one call, the read-out kept in fp32 as the memory's
        dict(_scan(1, 16, 131072, 64, 64, y="f32"), name="scan_long"),
        # a ragged fp32 batch at the configuration example's head width, two value heads per query/key head
        dict(_scan(3, 6, 1501, 48, 48, dtype="f32", y="f32", share=2, ragged=True), name="scan_ragged_f32"),
        # one token for a batch of sequences, the q/k/v channels of the configuration example
        dict(_conv(256, 1, 2304), name="conv_step"),
        # prompts, a slice of the projection's rows
        dict(_conv(4, 4096, 1536, extra=24), name="conv_prompt"),
        # the norm in front of a layer, one token of a few sequences
        dict(_rms(8, 2048), name="rms_token"),
        # prompts, quantised for the product behind it
        dict(_rms(16384, 2048, y="e4m3", block=128), name="rms_e4m3"),
        # the widening half of a feed-forward block, one token
        dict(_qlinear(1, 2048, 8192, act="silu"), name="q4_token"),
        # a batch of tokens out of the quantising norm
        dict(_qlinear(16, 8192, 8192, x="e4m3", x_block=128, residual=True), name="q4_batch"),
        # fp32, zero points, short groups, no size a multiple of anything
        dict(_qlinear(37, 1031, 2517, group=32, zeros=True, x="f32", out="f32", bias=True), name="q4_odd_f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _size(rng, lo, hi, step):
    """A size of [lo, hi]: half of the time a multiple of `step`, else any."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.5:
        v = max(step, v // step * step)
    return v


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "conv", "rms", "qlinear", "qlinear"])
    if op == "scan":
        dt = rng.choice(["bf16", "bf16", "f32"])
        d_k = rng.choice([16, 24, 32, 48, 64, 64, 96, 128, 128, rng.randint(3, 128)])
        d_v = d_k if rng.random() < 0.4 else rng.choice([32, 48, 64, 64, 80, 128, rng.randint(3, 128)])
        T = 1 if rng.random() < 0.3 else _log(rng, 2, 65536)
        share = rng.choice([1, 1, 2, 4, 8])
        most = (1 << 21) // T * 64 // max(d_k, d_v, 64) // (1 if dt == "bf16" else 4)
        units = max(share, _log(rng, 1, max(1, min(4096 if T == 1 else 512, most))))
        H = share * rng.randint(1, max(1, min(16, units) // share))
        B = max(1, units // H)
        return _scan(B, H, T, d_k, d_v, rng.choice(["memory", "step"]), dt, rng.choice(["f32", dt]), share,
                     B > 1 and rng.random() < 0.4, rng.choice(["heads", "tokens", "tokens"]),
                     rng.choice(["heads", "tokens"]), rng.random() < 0.7, rng.random() < 0.5)
    if op == "conv":
        T = 1 if rng.random() < 0.3 else _log(rng, 2, 16384)
        C = _size(rng, 16, 4096, 8)
        B = _log(rng, 1, max(1, min(1024, (1 << 25) // (T * C))))
        return _conv(B, T, C, rng.choice([2, 3, 4, 4, 4, 8]), rng.choice(["none", "silu"]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5, rng.choice([0, 0, 8, 24, 5]),
                     B > 1 and rng.random() < 0.4, rng.random() < 0.7)
    if op == "rms":
        C = _size(rng, 64, 16384, 128)
        M = _log(rng, 1, max(1, min(32768, (1 << 25) // C)))
        y = rng.choice(["bf16", "f32", "e4m3", "e4m3"])
        return _rms(M, C, rng.choice(["bf16", "bf16", "f32"]), y, rng.choice(["bf16", "f32", "none"]),
                    rng.choice([0, 128]) if y == "e4m3" else 0, rng.random() < 0.8)
    K, N, M = _size(rng, 64, 8192, 64), _size(rng, 64, 8192, 64), _log(rng, 1, 128)
    x = rng.choice(["bf16", "bf16", "f32", "e4m3"])
    return _qlinear(M, K, N, rng.choice([32, 64, 128, 128]), rng.random() < 0.4, rng.choice(["none", "silu", "gelu"]), x,
                    rng.choice([0, 128]) if x == "e4m3" else 0, rng.choice(["f32", "bf16"]), rng.random() < 0.5,
                    rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _lens(case, g):
    """Ragged lengths: evenly spread from 0 (an empty row) to T, in an order of the seed's."""
    B, T = case["B"], case["T"]
    v = torch.tensor([T * b // (B - 1) if B > 1 else T // 2 for b in range(B)], dtype=torch.int32)
    return v.cuda()[torch.randperm(B, generator=g, device="cuda")].contiguous()


def _silu(x):
    return x / (1 + torch.exp(-x))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] == "scan":
        B, H, T, dk, dv = (case[n] for n in ("B", "H", "T", "d_k", "d_v"))
        Hq, heads = H // case["share"], case["layout"] == "heads"
        if case["gates"] == "memory":
            # queries and keys come out of the stage in front with unit norm, its gates as the workloads draw them
            q, k = (torch.nn.functional.normalize(normal(B, T, Hq, dk), dim=-1) for _ in range(2))
            v = normal(B, T, H, dv)
            s["theta"] = (0.1 * torch.sigmoid(normal(B, T, H)))
            s["alpha"] = torch.sigmoid(normal(B, T, H) - 4)
        else:
            # behind a convolution with SiLU; steps of 0.001 to 0.1, decays of one token to hundreds
            q, k, v = (_silu(normal(B, T, n, d)) for n, d in ((Hq, dk), (Hq, dk), (H, dv)))
            s["dt"] = 0.5 * normal(B, T, H)
            step = torch.exp(uniform(math.log(0.001), math.log(0.1), H))
            s["dt_bias"] = step + torch.log(-torch.expm1(-step))
            s["A"] = -uniform(1, 16, H)
        for n in ("theta", "alpha", "dt"):
            if n in s and heads:
                s[n] = s[n].transpose(1, 2).contiguous()
        if heads:
            s["q"], s["k"], s["v"] = (x.transpose(1, 2).to(DT[case["dtype"]]).contiguous() for x in (q, k, v))
        else:
            # rows of the convolution's output: v, k, q side by side
            row = torch.cat([x.reshape(B, T, -1) for x in (v, k, q)], 2).to(DT[case["dtype"]])
            s["v"] = row[..., :H * dv].unflatten(2, (H, dv))
            s["k"] = row[..., H * dv:H * dv + Hq * dk].unflatten(2, (Hq, dk))
            s["q"] = row[..., H * dv + Hq * dk:].unflatten(2, (Hq, dk))
        s["D"] = 1 + 0.1 * normal(H) if case["skip"] else None
        s["lens"] = _lens(case, g) if case["ragged"] else None
        s["S0"] = normal(B, H, dk, dv) if case["state"] else None
    elif case["op"] == "conv":
        B, T, C, K = (case[n] for n in ("B", "T", "C", "K"))
        s["x"] = normal(B, T, C + case["extra"]).to(DT[case["dtype"]])[..., :C]
        s["w"] = normal(C, K) / K ** 0.5
        s["bias"] = 0.1 * normal(C) if case["bias"] else None
        s["cache"] = normal(B, K - 1, C).to(DT[case["dtype"]]) if case["cache"] else None
        s["lens"] = _lens(case, g) if case["ragged"] else None
    elif case["op"] == "rms":
        M, C = case["M"], case["C"]
        s["x"] = normal(M, C).to(DT[case["x"]])
        # the stream that the layers add to: wider, some channels far wider than the others
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = (2 * normal(M, C) * torch.exp(0.5 * normal(C))).to(DT[case["residual"]])
        s["weight"] = 1 + 0.2 * normal(C) if case["affine"] else None
    else:
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        n = -(-K // G)
        W = torch.nn.functional.pad(normal(K, N) / K ** 0.5, (0, 0, 0, n * G - K)).view(n, G, N)
        if case["zeros"]:
            lo, hi = W.amin(1), W.amax(1)
            s["scales"] = ((hi - lo) / 15).to(torch.bfloat16)
            step = s["scales"].float()
            s["zeros"] = torch.round(-lo / step).clamp(0, 15).to(torch.uint8)
            q = torch.round(W / step[:, None]) + s["zeros"].float()[:, None]
        else:
            s["scales"], s["zeros"] = (W.abs().amax(1) / 7).to(torch.bfloat16), None
            q = torch.round(W / s["scales"].float()[:, None]) + 8
        q = q.clamp(0, 15).to(torch.uint8).view(n * G, N)
        q[K:] = 0
        s["q"] = (q[0::2] | (q[1::2] << 4))[:-(-K // 2)].contiguous()
        x = normal(M, K)
        s["x_scale"] = None
        if case["x"] == "e4m3":
            b = case["x_block"] or K
            pad = torch.nn.functional.pad(x, (0, -K % b)).view(M, -1, b)
            s["x_scale"] = pad.abs().amax(2) / E4M3_MAX
            x = (pad / s["x_scale"][..., None]).view(M, -1)[:, :K]
        s["x"] = x.to(DT[case["x"]]).contiguous()
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        s["residual"] = normal(M, N).to(DT[case["out"]]) if case["residual"] else None
    if own:
        from test_learned_neural_gb300 import runner
        if case["op"] == "scan":
            h = runner.SelectiveScan(case["H"], case["d_k"], case["d_v"], share=case["share"], gates=case["gates"],
                                     qkv_dtype=case["dtype"], y_dtype=case["y"], qkv_layout=case["layout"],
                                     y_layout=case["y_layout"])
        elif case["op"] == "conv":
            h = runner.ShortConv(case["C"], case["K"], act=case["act"], dtype=case["dtype"])
        elif case["op"] == "rms":
            h = runner.RmsNorm(case["C"], x_dtype=case["x"], y_dtype=case["y"], block=case["block"],
                               residual_dtype=None if case["residual"] == "none" else case["residual"])
        else:
            h = runner.QuantLinear(case["K"], case["N"], group=case["group"], zeros=case["zeros"], act=case["act"],
                                   x_dtype=case["x"], x_block=case["x_block"], out_dtype=case["out"])
            # the weights in the kernels' order, once
            s["W"] = h.pack(s["q"], s["scales"], s["zeros"])
        s["handle"] = h
        # the buffers that a serving loop keeps for its outputs
        size = {"scan": ("B", "T"), "conv": ("B", "T"), "rms": ("M",), "qlinear": ("M",)}[case["op"]]
        s["out"] = h.alloc_outputs(*(case[n] for n in size), "cuda")
    return s


# ------------------------------------------------------------- plain forms
def _act(x, act):
    if act == "silu":
        return _silu(x)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x / math.sqrt(2.0)))
    return x


def _heads_first(s, name):
    return s[name] if s["case"]["layout"] == "heads" else s[name].transpose(1, 2)


def _plain_scan(s):
    """Chunks of 64 tokens: products inside a chunk under the mask of decays, and the chunk-start states from one
    product over chunks.  Sums of the decays' logarithms in 64 bits."""
    case, C = s["case"], 64
    B, H, T, R = (case[n] for n in ("B", "H", "T", "share"))
    D = torch.float64
    q, k, v = (_heads_first(s, n).float() for n in ("q", "k", "v"))
    q, k = (x.repeat_interleave(R, dim=1) for x in (q, k))
    if case["gates"] == "memory":
        step, log_g = _heads_first(s, "theta"), torch.log1p(-_heads_first(s, "alpha").to(D))
    else:
        x = _heads_first(s, "dt").to(D) + s["dt_bias"].to(D)[:, None]
        step = torch.where(x > 30, x, torch.log1p(torch.exp(x)))
        log_g = step * s["A"].to(D)[:, None]
        step = step.float()
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    live = (torch.arange(T, device="cuda") < lens[:, None])[:, None]                # [B, 1, T]
    skip = s["D"][:, None, None] * v * live[..., None] if s["D"] is not None else 0.0
    q = q * live[..., None]
    k = k * (step * live)[..., None]
    log_g = log_g * live
    v = v * live[..., None]
    S0 = s["S0"] if s["S0"] is not None else torch.zeros(B, H, case["d_k"], case["d_v"], device="cuda")
    n = -(-T // C)
    C = C if n > 1 else T
    pad = n * C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, n, C, -1) for x in (q, k, v))
    cum = torch.nn.functional.pad(log_g, (0, pad)).reshape(B, H, n, C).cumsum(3)    # from each chunk's start
    i = torch.arange(C, device="cuda")
    mask = torch.where(i[:, None] >= i, torch.exp(cum[..., :, None] - cum[..., None, :]), 0.0).float()
    y = ((q @ k.transpose(3, 4)) * mask) @ v
    add = (k * torch.exp(cum[..., -1:] - cum).float()[..., None]).transpose(3, 4) @ v   # [B, H, n, d_k, d_v]
    total = cum[..., -1].cumsum(2)                                                  # [B, H, n], behind each chunk
    before = total - cum[..., -1]
    c = torch.arange(n, device="cuda")
    carry = torch.where(c[:, None] > c, torch.exp(before[..., :, None] - total[..., None, :]), 0.0).float()
    start = (carry @ add.reshape(B, H, n, -1)).reshape(add.shape)
    start = start + torch.exp(before).float()[..., None, None] * S0[:, :, None]
    y = y + (q * torch.exp(cum).float()[..., None]) @ start
    S = torch.exp(cum[:, :, -1, -1]).float()[..., None, None] * start[:, :, -1] + add[:, :, -1]
    y = y.reshape(B, H, n * C, -1)[:, :, :T] + skip
    if case["y_layout"] == "tokens":
        y = y.transpose(1, 2)
    return dict(y=y.to(DT[case["y"]]).contiguous(), S=S)


def _rows_before(s, x):
    """The K - 1 rows before the call and the call's own (zero past a row's length), and the next call's cache."""
    case = s["case"]
    B, T, K = case["B"], case["T"], case["K"]
    cache = s["cache"] if s["cache"] is not None else x.new_zeros(B, K - 1, case["C"])
    rows = torch.cat([cache.to(x.dtype), x], 1)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    at = lens[:, None] + torch.arange(K - 1, device="cuda")
    keep = torch.cat([cache, s["x"]], 1).gather(1, at[..., None].expand(-1, -1, case["C"]))
    return rows, keep, (torch.arange(T, device="cuda") < lens[:, None])[..., None]


def _plain_conv(s):
    case = s["case"]
    rows, keep, live = _rows_before(s, s["x"].float())
    y = (rows.unfold(1, case["K"], 1) * s["w"]).sum(3)
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, case["act"])
    return dict(y=torch.where(live, y, 0.0).to(DT[case["dtype"]]), cache=keep)


def _plain_rms(s):
    case = s["case"]
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["h"] = h.to(DT[case["residual"]])
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    if s["weight"] is not None:
        y = y * s["weight"]
    if case["y"] == "e4m3":
        M, C, b = case["M"], case["C"], case["block"] or case["C"]
        y = torch.nn.functional.pad(y, (0, -C % b)).view(M, -1, b)
        out["scale"] = y.abs().amax(2).clamp(min=2.0 ** -100) / E4M3_MAX
        y = (y / out["scale"][..., None]).view(M, -1)[:, :C].contiguous()
    out["y"] = y.to(DT[case["y"]])
    return out


def _weights(s, dtype):
    """scale (q - zero), [K, N]."""
    case = s["case"]
    K, N, G = case["K"], case["N"], case["group"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], 1).view(-1, N)[:K].to(dtype)
    group = torch.arange(K, device="cuda") // G
    zero = s["zeros"].to(dtype)[group] if s["zeros"] is not None else 8.0
    return s["scales"].to(dtype)[group] * (q - zero)


def _x_values(s, dtype):
    x = s["x"].to(torch.float32).to(dtype)
    if s["x_scale"] is not None:
        b = s["case"]["x_block"] or s["case"]["K"]
        x = x * s["x_scale"].to(dtype)[:, torch.arange(s["case"]["K"], device="cuda") // b]
    return x


def _plain_qlinear(s):
    case = s["case"]
    y = _x_values(s, torch.float32) @ _weights(s, torch.float32)
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return dict(y=y.to(DT[case["out"]]))


def run(s):
    if own:
        return s["handle"].forward(s, out=s["out"])
    return {"scan": _plain_scan, "conv": _plain_conv, "rms": _plain_rms, "qlinear": _plain_qlinear}[s["case"]["op"]](s)


# -------------------------------------------------------- definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "scan":
        # token by token: S = g S + step k v^T, y = q S + D v
        B, H, T = case["B"], case["H"], case["T"]
        if T > 140000:
            return None
        S = torch.zeros(B, H, case["d_k"], case["d_v"], dtype=D, device="cuda") if s["S0"] is None else s["S0"].to(D)
        gates = [_heads_first(s, n).to(D) for n in (("theta", "alpha") if case["gates"] == "memory" else ("dt",))]
        if case["gates"] == "memory":
            step, decay = gates[0], 1 - gates[1]
        else:
            step = torch.nn.functional.softplus(gates[0] + s["dt_bias"].to(D)[:, None], threshold=700)
            decay = torch.exp(step * s["A"].to(D)[:, None])
        if s["lens"] is not None:
            on = (torch.arange(T, device="cuda") < s["lens"][:, None])[:, None]
            step, decay = step * on, torch.where(on, decay, 1.0)
        at = 2 if case["layout"] == "heads" else 1
        head = torch.arange(H, device="cuda") // case["share"]
        rows = []
        for t in range(T):
            q, k, v = (s[n].select(at, t).to(D) for n in ("q", "k", "v"))
            w = step[:, :, t, None] * k[:, head]
            S = torch.addcmul(decay[:, :, t, None, None] * S, w[..., None], v[:, :, None])
            y = torch.einsum("bhk,bhkv->bhv", q[:, head], S)
            if s["D"] is not None:
                y = torch.addcmul(y, s["D"].to(D)[:, None], v)
            rows.append(y)
        y = torch.stack(rows, 2)
        if s["lens"] is not None:
            y = torch.where(on[..., None], y, 0.0)
        return dict(y=y if case["y_layout"] == "heads" else y.transpose(1, 2), S=S)
    if case["op"] == "conv":
        rows, keep, live = _rows_before(s, s["x"].to(D))
        y = torch.zeros(case["B"], case["T"], case["C"], dtype=D, device="cuda")
        if s["bias"] is not None:
            y = y + s["bias"].to(D)
        for j in range(case["K"]):
            y = torch.addcmul(y, rows[:, j:j + case["T"]], s["w"][:, j].to(D))
        return dict(y=torch.where(live, _exact_act(y, case["act"]), 0.0), cache=keep.to(D))
    if case["op"] == "rms":
        out, h = {}, s["x"].to(D)
        if s["residual"] is not None:
            out["h"] = h = h + s["residual"].to(D)
        y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["C"] + 1e-6)
        if s["weight"] is not None:
            y = y * s["weight"].to(D)
        if case["y"] == "e4m3":
            b = case["block"] or case["C"]
            parts = torch.split(y, b, 1)
            out["scale"] = torch.stack([p.abs().amax(1).clamp(min=2.0 ** -100) / E4M3_MAX for p in parts], 1)
            y = torch.cat([p / out["scale"][:, i:i + 1] for i, p in enumerate(parts)], 1)
        out["y"] = y
        return out
    y = torch.mm(_x_values(s, D), _weights(s, D))
    if s["bias"] is not None:
        y = y + s["bias"].to(D)
    y = _exact_act(y, case["act"])
    return dict(y=y if s["residual"] is None else y + s["residual"].to(D))


def _exact_act(x, act):
    if act == "silu":
        return x * torch.special.expit(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x


# ---------------------------------------------------------------- the least
def _live(case):
    B, T = case["B"], case["T"]
    return sum(T * b // (B - 1) if B > 1 else T // 2 for b in range(B)) if case["ragged"] else B * T


def work(case):
    if case["op"] == "scan":
        B, H, T, R, d_k, d_v = (case[n] for n in ("B", "H", "T", "share", "d_k", "d_v"))
        gates = 8 * H if case["gates"] == "memory" else 4 * H
        read = _live(case) * ((2 * (H // R) * d_k + H * d_v) * SIZE[case["dtype"]] + gates)
        states = B * H * d_k * d_v * 4 * (2 if case["state"] else 1)
        return dict(bytes=read + B * T * H * d_v * SIZE[case["y"]] + states, flops=4.0 * _live(case) * H * d_k * d_v)
    if case["op"] == "conv":
        B, T, C, K = (case[n] for n in ("B", "T", "C", "K"))
        cache = B * (K - 1) * C * (2 if case["cache"] else 1)
        return dict(bytes=(_live(case) * C + B * T * C + cache) * SIZE[case["dtype"]] + 4 * C * (K + case["bias"]),
                    flops=2.0 * K * _live(case) * C)
    if case["op"] == "rms":
        n = case["M"] * case["C"]
        res = 2 * SIZE[case["residual"]] if case["residual"] != "none" else 0
        scales = 4 * case["M"] * (-(-case["C"] // (case["block"] or case["C"]))) if case["y"] == "e4m3" else 0
        return dict(bytes=n * (SIZE[case["x"]] + SIZE[case["y"]] + res) + scales + 4 * case["C"] * case["affine"],
                    flops=4.0 * n)
    M, K, N, G = (case[n] for n in ("M", "K", "N", "group"))
    weights = -(-K // 2) * N + -(-K // G) * N * (2.5 if case["zeros"] else 2)
    out = M * N * SIZE[case["out"]] * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
    x = M * K * SIZE[case["x"]] + (4 * M * (-(-K // (case["x_block"] or K))) if case["x"] == "e4m3" else 0)
    return dict(bytes=weights + out + x, flops=2.0 * M * K * N)
