"""A token-mixing layer from the library's operators, for prompts and single
tokens:

    q, k, v = the stage in front of the memory (projection, short convolution, q/k normalisation)
    a = attention with a decay for each head            DecayAttention
    a = SiLU(norm of each head)                         GroupNorm
    h = x + a W_o                                       Linear with residual
    y = h + SiLU(h W_1 + b_1) W_2 + b_2                 Linear with bias and activation, Linear with residual

    python examples/decay_layer.py                      # a prompt, then single tokens, with times
"""
import os
import sys
import time
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from test_learned_neural_gb300.runner import DecayAttention, GroupNorm, Linear, Prologue  # noqa: E402

CONV = 4


def random_weights(D, H, d, hidden, device):
    Nc, bf = 3 * H * d, torch.bfloat16
    n = lambda *s: torch.randn(*s, device=device)  # noqa: E731
    return dict(W_in=(n(D, Nc + 3 * H) / D ** 0.5).to(bf), conv_w=n(Nc, CONV) / CONV ** 0.5,
                gate_b=torch.zeros(3, H, device=device),
                decay=1 - torch.exp2(-2 - 6 * torch.arange(H, device=device) / H),
                norm_w=1 + 0.1 * n(H * d), norm_b=0.1 * n(H * d),
                W_o=(n(H * d, D) / (H * d) ** 0.5).to(bf),
                W_1=(n(D, hidden) / D ** 0.5).to(bf), b_1=0.1 * n(hidden),
                W_2=(n(hidden, D) / hidden ** 0.5).to(bf), b_2=0.1 * n(D))


class DecayLayer:
    def __init__(self, D, H, d, weights):
        self.D, self.H, self.d, self.w = D, H, d, weights
        self.cfg = SimpleNamespace(D=D, H=H, d_k=d, d_v=d, conv=CONV, with_gamma=0, theta_max=0.1, qkv_dtype="bf16",
                                   Nc=3 * H * d)
        self.front = Prologue(self.cfg)
        self.mix = DecayAttention(H, d, d, y_layout="tokens")
        self.norm = GroupNorm(H * d, H, act="silu")
        self.out = Linear(H * d, D)
        hidden = weights["W_1"].shape[1]
        self.up, self.down = Linear(D, hidden, act="silu"), Linear(hidden, D)

    def forward(self, x, state=None):
        """x [B, T, D] bf16; state from the last call on this sequence, or
        None.  Returns y [B, T, D] and the state for the next call."""
        B, T, D = x.shape
        w, st = self.w, state or {}
        p = self.front.forward(dict(x=x, W_in=w["W_in"], conv_w=w["conv_w"], gate_b=w["gate_b"], cache=st.get("cache")))
        a = self.mix.forward(dict(q=p["q"], k=p["k"], v=p["v"], decay=w["decay"], S0=st.get("S")))
        n = self.norm.forward(dict(x=a["y"].view(B * T, 1, -1), weight=w["norm_w"], bias=w["norm_b"]))
        h = self.out.forward(dict(x=n["y"].view(B * T, -1), W=w["W_o"], residual=x.reshape(B * T, D)))["y"]
        u = self.up.forward(dict(x=h, W=w["W_1"], bias=w["b_1"]))["y"]
        y = self.down.forward(dict(x=u, W=w["W_2"], bias=w["b_2"], residual=h))["y"]
        return y.view(B, T, D), dict(S=a["S"], cache=p["cache"])


def main():
    torch.manual_seed(0)
    B, T, D, H, d, steps = 4, 4096, 512, 8, 64, 64
    layer = DecayLayer(D, H, d, random_weights(D, H, d, hidden=2048, device="cuda"))
    x = torch.randn(B, T, D, device="cuda").bfloat16()
    for _ in range(3):
        y, state = layer.forward(x)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    y, state = layer.forward(x)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    tok = y[:, -1:].contiguous()
    for _ in range(steps):
        tok, state = layer.forward(tok, state)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    print(f"prompt of {B} x {T} tokens: {1e3 * (t1 - t0):.3f} ms ({B * T / (t1 - t0):.3g} tokens/s); "
          f"one token for {B} sequences: {1e6 * (t2 - t1) / steps:.0f} us")


if __name__ == "__main__":
    main()
