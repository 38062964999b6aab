"""A selective state-space layer from the library's operators, for prompts and
single tokens, with 4-bit weights:

    h, n = h + x, norm of the sum in 8 bits             RmsNorm
    z, c, dt = n W_in                                   QuantLinear (one projection)
    v, k, q = SiLU(short convolution of c)              ShortConv
    a = matrix memory with dt's steps and decays        SelectiveScan
    g = norm of each head of a, times SiLU(z)           GroupNorm
    y = g W_out                                         QuantLinear

    python examples/selective_layer.py                  # a prompt, then single tokens, with times
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from test_learned_neural_gb300.runner import GroupNorm, QuantLinear, RmsNorm, SelectiveScan, ShortConv  # noqa: E402

TAPS = 4


class SelectiveLayer:
    """D wide, H heads of d values, one query/key head of d_k for all of them."""

    def __init__(self, D, H, d, d_k, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g).to(device)  # noqa: E731
        self.D, self.H, self.d, self.d_k = D, H, d, d_k
        self.C = H * d + 2 * d_k                      # v, k, q side by side, as the convolution takes them
        wide = H * d + self.C + H                     # z, the convolution's channels, dt
        self.norm = RmsNorm(D, y_dtype="e4m3", block=128)
        # dt is wanted in fp32, so the projection's results are; the convolution's channels go back to bf16
        self.proj = QuantLinear(D, wide, x_dtype="e4m3", x_block=128, out_dtype="f32")
        self.conv = ShortConv(self.C, TAPS, dtype="bf16")
        self.scan = SelectiveScan(H, d_k, d, share=H, gates="step", qkv_layout="tokens", y_layout="tokens")
        self.head_norm = GroupNorm(H * d, H)
        self.out = QuantLinear(H * d, D)
        self.w = dict(norm=1 + 0.1 * n(D), taps=n(self.C, TAPS) / TAPS ** 0.5, taps_b=0.1 * n(self.C),
                      dt_bias=n(H) - 3, A=-1 - 7 * torch.rand(H, generator=g).to(device), skip=1 + 0.1 * n(H),
                      head=1 + 0.1 * n(H * d), W_in=n(D, wide) / D ** 0.5, W_out=n(H * d, D) / (H * d) ** 0.5)
        self.W_in, self.W_out = (op.pack(**op.quantize(self.w[name])) for op, name in ((self.proj, "W_in"), (self.out, "W_out")))

    def forward(self, x, stream, state=None):
        """x [B, T, D] bf16, what the layer before adds to the stream [B, T, D]
        (bf16); state from the last call on these sequences, or None.  Returns y
        and the new stream, [B, T, D] each, and the state for the next call."""
        B, T, D = x.shape
        w, st, Hd = self.w, state or {}, self.H * self.d
        n = self.norm.forward(dict(x=x.reshape(B * T, D), residual=stream.reshape(B * T, D), weight=w["norm"]))
        p = self.proj.forward(dict(x=n["y"], x_scale=n["scale"], W=self.W_in))["y"].view(B, T, -1)
        c = self.conv.forward(dict(x=p[..., Hd:Hd + self.C].bfloat16(), w=w["taps"], bias=w["taps_b"], cache=st.get("cache")))
        v, k, q = c["y"].split([Hd, self.d_k, self.d_k], dim=2)
        a = self.scan.forward(dict(q=q.unflatten(2, (1, -1)), k=k.unflatten(2, (1, -1)), v=v.unflatten(2, (self.H, -1)),
                                   dt=p[..., Hd + self.C:], dt_bias=w["dt_bias"], A=w["A"], D=w["skip"], S0=st.get("S")))
        g = self.head_norm.forward(dict(x=a["y"].view(B * T, 1, Hd), weight=w["head"]))["y"].view(B, T, Hd)
        z = p[..., :Hd]
        g = (g * (z * torch.sigmoid(z))).bfloat16()
        y = self.out.forward(dict(x=g.view(B * T, Hd), W=self.W_out))["y"].view(B, T, D)
        return y, n["h"].view(B, T, D), dict(S=a["S"], cache=c["cache"])


def main():
    B, T, D, H, d, d_k, steps = 4, 4096, 512, 16, 64, 128, 64
    layer = SelectiveLayer(D, H, d, d_k)
    x, stream = torch.randn(B, T, D, device="cuda").bfloat16(), torch.randn(B, T, D, device="cuda").bfloat16()
    for _ in range(3):
        y, _, state = layer.forward(x, stream)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    y, _, state = layer.forward(x, stream)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    tok, one = y[:, -1:].contiguous(), stream[:, -1:].contiguous()
    for _ in range(steps):
        tok, one, state = layer.forward(tok, one, state)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    print(f"prompt of {B} x {T} tokens: {1e3 * (t1 - t0):.3f} ms ({B * T / (t1 - t0):.3g} tokens/s); "
          f"one token for {B} sequences: {1e6 * (t2 - t1) / steps:.0f} us")


if __name__ == "__main__":
    main()
