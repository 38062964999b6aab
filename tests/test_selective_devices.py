"""The selective layer's operators refuse tensors of several devices, of one that
is not the current one, and host tensors, before any call of the library."""
import pytest
import torch

from test_learned_neural_gb300 import runner
from tests.test_layer_devices import Fake as Plain
from tests.test_layer_pins import lib  # noqa: F401


class Fake(Plain):
    def stride(self):
        return torch.empty(self.shape, device="meta").stride()


def _cases():
    f, h, e, u = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8
    qk, v, g, S = (2, 5, 1, 8), (2, 5, 2, 4), (2, 5, 2), (2, 2, 8, 4)
    return {
        "scan": (lambda: runner.SelectiveScan(2, 8, 4, share=2, gates="step", qkv_layout="tokens"),
                 dict(q=(qk, h), k=(qk, h), v=(v, h), dt=(g, f), A=((2,), f), dt_bias=((2,), f), D=((2,), f),
                      lens=((2,), torch.int32), S0=(S, f)), dict(y=((2, 2, 5, 4), h), S=(S, f))),
        "conv": (lambda: runner.ShortConv(8, 4), dict(x=((2, 5, 8), h), w=((8, 4), f), bias=((8,), f), cache=((2, 3, 8), h),
                                                      lens=((2,), torch.int32)), dict(y=((2, 5, 8), h), cache=((2, 3, 8), h))),
        "rms": (lambda: runner.RmsNorm(8, y_dtype="e4m3"), dict(x=((3, 8), h), residual=((3, 8), h), weight=((8,), f)),
                dict(y=((3, 8), e), h=((3, 8), h), scale=((3, 1), f))),
        "qlinear": (lambda: runner.QuantLinear(8, 4, x_dtype="e4m3"),
                    dict(x=((3, 8), e), x_scale=((3, 1), f), W=((8448,), u), bias=((4,), f), residual=((3, 4), h)),
                    dict(y=((3, 4), h))),
    }


@pytest.fixture
def no_calls(monkeypatch):
    """The library's forwards record their calls and launch nothing."""
    calls = []
    for op in _cases():
        monkeypatch.setattr(runner, f"atlas_{op}_forward", lambda *a, op=op: calls.append((op, a[2])))
    monkeypatch.setattr(runner, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(runner, "_devices", 2, raising=False)
    monkeypatch.setattr(runner, "_raw_stream", lambda index: 100 + index)
    return calls


@pytest.mark.parametrize("op", list(_cases()))
def test_tensors_of_another_device_are_refused(lib, no_calls, op):  # noqa: F811
    make, ins, outs = _cases()[op]
    h = make()

    def call(at, **kw):
        t = {n: Fake(*ins[n], at.get(n, at["all"])) for n in ins}
        return h.forward(t, out={n: Fake(*outs[n], at.get("out " + n, at["all"])) for n in outs}, **kw)

    call({"all": 0})
    call({"all": 0}, stream=7)
    assert no_calls == [(op, 100), (op, 7)]
    for n in (*ins, *("out " + m for m in outs)):
        for index in (1, -1):
            with pytest.raises(ValueError, match="device"):
                call({"all": 0, n: index})
    for kw in ({}, dict(stream=7)):
        with pytest.raises(ValueError, match="current device"):
            call({"all": 1}, **kw)
    with pytest.raises(ValueError):
        call({"all": -1})
    assert len(no_calls) == 2


def test_quantize_and_pack_refuse_host_tensors(lib):  # noqa: F811
    op = runner.QuantLinear(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        op.quantize(torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        op.pack(torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(1, 4).bfloat16())


def test_scan_refuses_tokens_that_lie_unequally_apart(lib, no_calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(runner, "_check_rows", lambda name, *a: (1 << 20, {"k": 9}.get(name, 8)))
    make, ins, outs = _cases()["scan"]
    t = {n: Fake(*ins[n], 0) for n in ins}
    with pytest.raises(ValueError, match="equally"):
        make().forward(t, out={n: Fake(*outs[n], 0) for n in outs})
    assert not no_calls
