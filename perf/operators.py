"""Cases of the layer operators around the memory: attention with a decay per
head, group norm with an activation, and the matrix product with bias,
activation and residual.

`listed()` and `draw()` give cases, `prepare()` their inputs, `run()` one pass:
through the library's entry points where `own` is true, else in plain torch
(fp32 whatever the inputs' type, rounded once at the end).  `exact()` gives the
same outputs in 64 bits from the operators' definitions.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def _decay(B, H, T, d_k, d_v, dtype="bf16", y="bf16", share=1, ragged=False, layout="heads", y_layout="heads",
           state=True):
    return dict(op="decay", B=B, H=H, T=T, d_k=d_k, d_v=d_v, dtype=dtype, y=y, share=share, ragged=ragged,
                layout=layout, y_layout=y_layout, state=state)


def _norm(N, S, C, G, act="silu", x="bf16", y="bf16", layout="channels_last", affine=True):
    return dict(op="norm", N=N, S=S, C=C, G=G, act=act, x=x, y=y, layout=layout, affine=affine)


def _linear(M, K, N, act="none", dtype="bf16", out="bf16", bias=True, residual=True):
    return dict(op="linear", M=M, K=K, N=N, act=act, dtype=dtype, out=out, bias=bias, residual=residual)


def listed():
    return [
        # one token for a handful of sequences: the latency of a serving step
        dict(_decay(8, 8, 1, 64, 64), name="decay_step"),
        # one token for many sequences with wide heads: all time goes to the states
        dict(_decay(256, 16, 1, 128, 128), name="decay_step_many"),
        # a batch of prompts of the Titans workload's shape, tokens first for the head norm behind it
        dict(_decay(4, 8, 4096, 64, 64, y_layout="tokens", state=False), name="decay_prompt"),
        # the long-context workload's shape in one call, the read-out kept in fp32 as the memory's
        dict(_decay(1, 16, 131072, 64, 64, y="f32"), name="decay_long"),
        # a ragged fp32 batch at the configuration example's head width, two value heads per query/key head
        dict(_decay(3, 6, 1501, 48, 48, dtype="f32", y="f32", share=2, ragged=True), name="decay_ragged_f32"),
        # the head norm behind the memory's fp32 read-out of the Titans workload
        dict(_norm(4, 4096, 512, 8, x="f32", layout="heads"), name="norm_heads"),
        # statistics over all positions of a sample, channels last
        dict(_norm(8, 4096, 1024, 32), name="norm_positions"),
        # odd positions and group width in fp32, no affine
        dict(_norm(5, 1023, 510, 6, act="gelu", x="f32", y="f32", affine=False), name="norm_odd_f32"),
        # the output projection of one token
        dict(_linear(1, 512, 512), name="linear_token"),
        # the output projection of a batch of sequences at the configuration example's width
        dict(_linear(16384, 768, 768, bias=False), name="linear_out"),
        # the widening half of a feed-forward block
        dict(_linear(16384, 2048, 8192, act="gelu", residual=False), name="linear_wide"),
        # fp32, no size a multiple of anything
        dict(_linear(1999, 517, 1031, act="silu", dtype="f32", out="f32"), name="linear_odd_f32"),
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
    op = rng.choice(["decay", "decay", "norm", "linear", "linear"])
    if op == "decay":
        dt = rng.choice(["bf16", "bf16", "f32"])
        d_k, d_v = (rng.choice([16, 24, 32, 48, 64, 64, 80, 96, 128, 128, rng.randint(3, 128)]) for _ in range(2))
        if rng.random() < 0.5:
            d_v = d_k
        T = 1 if rng.random() < 0.3 else _log(rng, 2, 65536)
        share = rng.choice([1, 1, 2, 4])
        most = (1 << 21) // T * 64 // max(d_k, d_v, 64) // (1 if dt == "bf16" else 4)
        units = max(share, _log(rng, 1, max(1, min(4096 if T == 1 else 512, most))))
        H = share * rng.randint(1, max(1, min(16, units) // share))
        B = max(1, units // H)
        return _decay(B, H, T, d_k, d_v, dt, rng.choice(["f32", dt]), share, B > 1 and rng.random() < 0.4,
                      rng.choice(["heads", "heads", "tokens"]), rng.choice(["heads", "tokens"]), rng.random() < 0.7)
    if op == "norm":
        G = rng.choice([1, 2, 4, 6, 8, 16, 32])
        Cg = rng.choice([4, 8, 16, 32, 48, 64, 128, rng.randint(3, 160)])
        layout = rng.choice(["channels_last", "channels_last", "heads"])
        S = 1 if layout == "channels_last" and rng.random() < 0.3 else _log(rng, 2, 16384)
        N = _log(rng, 1, max(1, min(16384, (1 << 25) // (S * G * Cg))))
        return _norm(N, S, G * Cg, G, rng.choice(["none", "silu", "gelu"]), rng.choice(["bf16", "f32"]),
                     rng.choice(["bf16", "f32"]), layout, rng.random() < 0.8)
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    while True:
        M, K, N = _log(rng, 1, 16384), _size(rng, 64, 8192, 64), _size(rng, 64, 8192, 64)
        if M * K * N <= (1 << 37) and 3072 not in (M, K, N):
            break
    return _linear(M, K, N, rng.choice(["none", "silu", "gelu"]), dt, rng.choice(["f32", dt]), rng.random() < 0.7,
                   rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _lens(case, g):
    """Ragged lengths: evenly spread from 0 (an empty row) to T, in an order of the seed's."""
    B, T = case["B"], case["T"]
    v = torch.tensor([T * b // (B - 1) if B > 1 else T // 2 for b in range(B)], dtype=torch.int32)
    return v.cuda()[torch.randperm(B, generator=g, device="cuda")].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] == "decay":
        B, H, T, R = case["B"], case["H"], case["T"], case["share"]

        def heads(n, d, unit):
            # queries and keys come out of the stage in front with unit norm
            x = normal(*((B, n, T, d) if case["layout"] == "heads" else (B, T, n, d)))
            return (x / x.norm(dim=-1, keepdim=True) if unit else x).to(DT[case["dtype"]])

        s["q"], s["k"] = heads(H // R, case["d_k"], True), heads(H // R, case["d_k"], True)
        s["v"] = heads(H, case["d_v"], False)
        # memories of about 4 to 500 tokens
        s["decay"] = 1 - torch.exp2(-(2 + 7 * torch.rand(H, generator=g, device="cuda")))
        s["lens"] = _lens(case, g) if case["ragged"] else None
        s["S0"] = normal(B, H, case["d_k"], case["d_v"]) if case["state"] else None
    elif case["op"] == "norm":
        N, S, C, G = case["N"], case["S"], case["C"], case["G"]
        shape = (N, S, C) if case["layout"] == "channels_last" else (N, G, S, C // G)
        s["x"] = (normal(*shape) * 1.5 + 0.3).to(DT[case["x"]])
        s["weight"] = 1 + 0.2 * normal(C) if case["affine"] else None
        s["bias"] = 0.2 * normal(C) if case["affine"] else None
    else:
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = normal(M, K).to(DT[case["dtype"]])
        s["W"] = (normal(K, N) / K ** 0.5).to(DT[case["dtype"]])
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        s["residual"] = normal(M, N).to(DT[case["out"]]) if case["residual"] else None
    if own:
        from test_learned_neural_gb300 import runner
        if case["op"] == "decay":
            s["handle"] = runner.DecayAttention(case["H"], case["d_k"], case["d_v"], qkv_dtype=case["dtype"],
                                                y_dtype=case["y"], share=case["share"], qkv_layout=case["layout"],
                                                y_layout=case["y_layout"])
        elif case["op"] == "norm":
            s["handle"] = runner.GroupNorm(case["C"], case["G"], act=case["act"], x_dtype=case["x"],
                                           y_dtype=case["y"], layout=case["layout"])
        else:
            s["handle"] = runner.Linear(case["K"], case["N"], act=case["act"], in_dtype=case["dtype"],
                                        out_dtype=case["out"])
        # the buffers that a serving loop keeps for its outputs
        size = {"decay": ("B", "T"), "norm": ("N", "S"), "linear": ("M",)}[case["op"]]
        s["out"] = s["handle"].alloc_outputs(*(case[n] for n in size), "cuda")
    return s


# ------------------------------------------------------------- plain forms
def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x / math.sqrt(2.0)))
    return x


def _plain_decay(s):
    """Chunks of 64 tokens: products inside a chunk under the decay mask, and the chunk-start states from one product
    over chunks."""
    case, C = s["case"], 64
    B, H, T, R, d_k, d_v = (case[n] for n in ("B", "H", "T", "share", "d_k", "d_v"))
    q, k, v = (s[n].float() if case["layout"] == "heads" else s[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    q, k = (x.repeat_interleave(R, dim=1) for x in (q, k))
    dec = s["decay"]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    t = torch.arange(T, device="cuda")
    live = (t < lens[:, None]).float()[:, None, :, None]
    k, v, q = k * live, v * live, q * live
    S0 = s["S0"] if s["S0"] is not None else torch.zeros(B, H, d_k, d_v, device="cuda")
    # final state: every token at its distance from its sequence's end
    left = (lens[:, None] - 1 - t).clamp(min=0)                                     # [B, T]
    w = dec[None, :, None] ** left[:, None, :]                                      # [B, H, T]
    S = (dec[None, :] ** lens[:, None])[..., None, None] * S0 + (k * w[..., None]).transpose(2, 3) @ v
    n = -(-T // C)
    C = C if n > 1 else T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).reshape(B, H, n, C, -1) for x in (q, k, v))
    i = torch.arange(C, device="cuda")
    gap = i[:, None] - i
    mask = torch.where(gap >= 0, dec[:, None, None] ** gap.clamp(min=0), 0.0)       # [H, C, C]
    y = ((q @ k.transpose(3, 4)) * mask[:, None]) @ v
    add = (k * (dec[:, None] ** (C - 1 - i))[:, None, :, None]).transpose(3, 4) @ v  # [B, H, n, d_k, d_v]
    c = torch.arange(n, device="cuda")
    gap = c[:, None] - 1 - c
    carry = torch.where(gap >= 0, dec[:, None, None] ** (C * gap.clamp(min=0)), 0.0)  # [H, n, n]
    start = (carry @ add.reshape(B, H, n, -1)).reshape(add.shape)
    start = start + (dec[:, None] ** (C * c))[:, :, None, None] * S0[:, :, None]
    y = y + (q * (dec[:, None] ** (i + 1))[:, None, :, None]) @ start
    y = y.reshape(B, H, n * C, d_v)[:, :, :T]
    if case["y_layout"] == "tokens":
        y = y.transpose(1, 2)
    return dict(y=y.to(DT[case["y"]]).contiguous(), S=S)


def _plain_norm(s):
    case = s["case"]
    N, S, C, G = (case[n] for n in ("N", "S", "C", "G"))
    x = s["x"].float()
    if case["layout"] == "heads":
        x = x.permute(0, 2, 1, 3).reshape(N, S, G, C // G)
        over = (3,)
    else:
        x = x.reshape(N, S, G, C // G)
        over = (1, 3)
    x = x - x.mean(over, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(over, keepdim=True) + 1e-5)
    x = x.reshape(N, S, C)
    if s["weight"] is not None:
        x = x * s["weight"] + s["bias"]
    return _act(x, case["act"]).to(DT[case["y"]])


def _plain_linear(s):
    case = s["case"]
    y = s["x"].float() @ s["W"].float()
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[case["out"]])


def run(s):
    op = s["case"]["op"]
    if own:
        out = s["handle"].forward(s, out=s["out"])
        return out if op == "decay" else out["y"]
    return {"decay": _plain_decay, "norm": _plain_norm, "linear": _plain_linear}[op](s)


# -------------------------------------------------------- definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "decay":
        # token by token: S = decay S + k v^T, y = q S
        B, H, T, R = case["B"], case["H"], case["T"], case["share"]
        if T > 140000:
            return None
        S = torch.zeros(B, H, case["d_k"], case["d_v"], dtype=D, device="cuda") if s["S0"] is None else s["S0"].to(D)
        dec = s["decay"].to(D)[:, None, None]
        at = 2 if case["layout"] == "heads" else 1
        head = torch.arange(H, device="cuda") // R
        rows = []
        for t in range(T):
            q, k, v = (s[n].select(at, t).to(D) for n in ("q", "k", "v"))
            q, k = q[:, head], k[:, head]
            new = torch.addcmul(dec * S, k[..., None], v[:, :, None])
            y = torch.einsum("bhk,bhkv->bhv", q, new)
            if s["lens"] is not None:
                on = (t < s["lens"])[:, None, None]
                y = torch.where(on, y, 0.0)
                new = torch.where(on[..., None], new, S)
            S = new
            rows.append(y)
        return dict(y=torch.stack(rows, 2 if case["y_layout"] == "heads" else 1), S=S)
    if case["op"] == "norm":
        N, S, C, G = (case[n] for n in ("N", "S", "C", "G"))
        x = s["x"].to(D)
        x = x.reshape(N, S, G, C // G) if case["layout"] == "channels_last" else x.transpose(1, 2)
        over = [1, 3] if case["layout"] == "channels_last" else [3]
        var, mean = torch.var_mean(x, over, correction=0, keepdim=True)
        x = ((x - mean) / torch.sqrt(var + 1e-5)).reshape(N, S, C)
        if s["weight"] is not None:
            x = torch.addcmul(s["bias"].to(D), x, s["weight"].to(D))
        return _exact_act(x, case["act"])
    y = torch.mm(s["x"].to(D), s["W"].to(D))
    if s["bias"] is not None:
        y = y + s["bias"].to(D)
    y = _exact_act(y, case["act"])
    return y if s["residual"] is None else y + s["residual"].to(D)


def _exact_act(x, act):
    if act == "silu":
        return x * torch.special.expit(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x


# ---------------------------------------------------------------- the least
def work(case):
    if case["op"] == "decay":
        B, H, T, R, d_k, d_v = (case[n] for n in ("B", "H", "T", "share", "d_k", "d_v"))
        live = sum(T * b // (B - 1) if B > 1 else T // 2 for b in range(B)) if case["ragged"] else B * T
        read = live * (2 * (H // R) * d_k + H * d_v) * SIZE[case["dtype"]]
        states = B * H * d_k * d_v * 4 * (2 if case["state"] else 1)
        return dict(bytes=read + B * T * H * d_v * SIZE[case["y"]] + states, flops=4.0 * live * H * d_k * d_v)
    if case["op"] == "norm":
        n = case["N"] * case["S"] * case["C"]
        return dict(bytes=n * (SIZE[case["x"]] + SIZE[case["y"]]) + (8 * case["C"] if case["affine"] else 0),
                    flops=8.0 * n)
    M, K, N = case["M"], case["K"], case["N"]
    out = M * N * SIZE[case["out"]] * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
    return dict(bytes=(M * K + K * N) * SIZE[case["dtype"]] + out, flops=2.0 * M * K * N)
