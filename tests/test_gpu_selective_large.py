"""Offsets that pass 32 bits: the last rows of tensors of more than 2^32 values, and of
more than 2^31, against the same rows computed on their own."""
import pytest

pytestmark = pytest.mark.gpu


def test_norm_past_32_bits(gpu_lib):
    import torch
    from test_learned_neural_gb300.runner import RmsNorm
    M, C = (1 << 21) + 5, 2048
    op = RmsNorm(C, y_dtype="e4m3", block=128)
    x = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    r = torch.empty_like(x).fill_(0.25)
    x[-3:] = torch.randn(3, C, device="cuda").bfloat16()
    out = op.forward(dict(x=x, residual=r))
    ref = op.forward(dict(x=x[-5:].clone(), residual=r[-5:].clone()))
    for n in ref:
        assert torch.equal(out[n][-5:].view(torch.uint8), ref[n].view(torch.uint8)), n


def test_convolution_past_32_bits(gpu_lib):
    import torch
    from test_learned_neural_gb300.runner import ShortConv
    B, T, C = 3, (1 << 19) + 7, 4096
    x = torch.empty(B, T, C, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    x[-1, -40:] = torch.randn(40, C, device="cuda").bfloat16()
    t = dict(w=torch.randn(C, 4, device="cuda"))
    op = ShortConv(C, 4)
    out = op.forward(dict(x=x, **t))
    ref = op.forward(dict(x=x[-1:, -40:].contiguous(), cache=x[-1:, -43:-40].contiguous(), **t))
    assert torch.equal(out["y"][-1:, -40:], ref["y"]) and torch.equal(out["cache"][-1:], ref["cache"])


@pytest.mark.parametrize("dk", [64, 128])
def test_scan_past_32_bits(gpu_lib, dk):
    """The last tokens of a long call, from the state that the call on those before them leaves."""
    import torch
    from test_learned_neural_gb300.runner import SelectiveScan
    H, T, last = 16, (1 << 21) + 300, 1000
    if dk == 128:
        T = (1 << 20) + 300
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k = (torch.empty(1, T, H, dk, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(dk ** -0.5) for _ in range(2))
    v = torch.empty(1, T, H, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    theta, alpha = (torch.rand(1, T, H, device="cuda", generator=g) for _ in range(2))
    t = dict(q=q, k=k, v=v, theta=theta, alpha=alpha.mul_(0.1))
    assert max(q.numel(), v.numel()) > 1 << 31
    op = SelectiveScan(H, dk, 64, qkv_layout="tokens", y_layout="tokens")
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    first = op.forward({n: a[:, :T - last] for n, a in t.items()})
    tail = op.forward(dict({n: a[:, T - last:].contiguous() for n, a in t.items()}, S0=first["S"]))
    torch.cuda.synchronize()
    op.status()
    # fp32 states and decays, in other chunks: 1e-5; bf16 read-outs twice half a step
    S, y = tail["S"], tail["y"].float()
    assert (out["S"] - S).abs().max() <= 1e-5 * S.abs().max()
    assert (out["y"][:, T - last:].float() - y).abs().max() <= 2 * 4.1e-3 * y.abs().max()


def test_4_bit_product_past_32_bits(gpu_lib):
    """More than 2^31 codes, and more than 2^31 values of x."""
    import torch
    from test_learned_neural_gb300.runner import QuantLinear
    K, N = 65536 + 128, 65536
    op = QuantLinear(K, N, out_dtype="f32")
    q = torch.full((K // 2, N), 0x88, dtype=torch.uint8, device="cuda")
    q[-1, -1], q[0, -1], q[-1, 0] = 0x9a, 0x78, 0x89
    scales = torch.ones(K // 128, N, device="cuda").bfloat16()
    x = torch.randn(2, K, device="cuda").bfloat16()
    y = op.forward(dict(x=x, W=op.pack(q, scales)))["y"]
    f = x.float()
    assert torch.allclose(y[:, -1], 2 * f[:, -2] + f[:, -1] - f[:, 1], atol=1e-5)
    assert torch.allclose(y[:, 0], f[:, -2], atol=1e-5) and not y[:, 1:-1].any()
    M = 33000
    op = QuantLinear(K, 32, out_dtype="f32")
    W = op.pack(torch.randint(0, 256, (K // 2, 32), dtype=torch.uint8, device="cuda"),
                torch.rand(K // 128, 32, device="cuda").bfloat16())
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").fill_(0.01)
    x[-5:] = torch.randn(5, K, device="cuda").bfloat16()
    y, ref = op.forward(dict(x=x, W=W))["y"][-5:], op.forward(dict(x=x[-5:].clone(), W=W))["y"]
    assert (y - ref).abs().max() <= 1e-5 * ref.abs().max()      # (K is split otherwise for few rows)
