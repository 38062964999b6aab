"""The layer operators' binding refuses tensors of several devices, and tensors
of a device that is not the current one, before any call of the library: a
kernel goes to the current device, and would read the addresses as its own."""
import pytest
import torch

from test_learned_neural_gb300 import runner
from tests.test_layer_pins import lib  # noqa: F401


class Fake:
    """A tensor of a device that this machine need not have."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.index = tuple(shape), dtype, device
        self.device, self.is_cuda = torch.device("cuda", device) if device >= 0 else torch.device("cpu"), device >= 0

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20


def _cases():
    f, h = torch.float32, torch.bfloat16
    return {
        "decay": (lambda: runner.DecayAttention(2, 8, 4),
                  dict(q=((1, 2, 5, 8), h), k=((1, 2, 5, 8), h), v=((1, 2, 5, 4), h), decay=((2,), f),
                       lens=((1,), torch.int32), S0=((1, 2, 8, 4), f)), dict(y=((1, 2, 5, 4), h), S=((1, 2, 8, 4), f))),
        "norm": (lambda: runner.GroupNorm(8, 2), dict(x=((3, 4, 8), h), weight=((8,), f), bias=((8,), f)),
                 dict(y=((3, 4, 8), h))),
        "linear": (lambda: runner.Linear(8, 4), dict(x=((3, 8), h), W=((8, 4), h), bias=((4,), f), residual=((3, 4), h)),
                   dict(y=((3, 4), h))),
    }


@pytest.fixture
def no_calls(monkeypatch):
    """The library's forwards record their calls and launch nothing."""
    calls = []
    for op in ("decay", "norm", "linear"):
        monkeypatch.setattr(runner, f"atlas_{op}_forward", lambda *a, op=op: calls.append((op, a[2])))
    monkeypatch.setattr(runner, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(runner, "_devices", 2, raising=False)
    monkeypatch.setattr(runner, "_raw_stream", lambda index: 100 + index)
    return calls


@pytest.mark.parametrize("op", ["decay", "norm", "linear"])
def test_tensors_of_another_device_are_refused(lib, no_calls, op):  # noqa: F811
    make, ins, outs = _cases()[op]
    h = make()

    def call(at, **kw):
        t = {n: Fake(*ins[n], at.get(n, at["all"])) for n in ins}
        return h.forward(t, out={n: Fake(*outs[n], at.get(n, at["all"])) for n in outs}, **kw)

    call({"all": 0})
    call({"all": 0}, stream=7)
    assert no_calls == [(op, 100), (op, 7)]
    for n in (*ins, *outs):                       # one tensor elsewhere, on the other side or on the host
        for index in (1, -1):
            with pytest.raises(ValueError, match="device"):
                call({"all": 0, n: index})
    with pytest.raises(ValueError, match="current device"):
        call({"all": 1})
    with pytest.raises(ValueError, match="current device"):
        call({"all": 1}, stream=7)
    with pytest.raises(ValueError):
        call({"all": -1})
    assert len(no_calls) == 2


@pytest.mark.parametrize("op", ["decay", "norm", "linear"])
def test_host_tensors_are_refused_where_there_is_one_device(lib, no_calls, monkeypatch, op):  # noqa: F811
    monkeypatch.setattr(runner, "_devices", 1)
    make, ins, outs = _cases()[op]
    h = make()
    for name in (*ins, *outs, None):
        def at(n):
            return -1 if n == name else 0
        t, out = {n: Fake(*ins[n], at(n)) for n in ins}, {n: Fake(*outs[n], at(n)) for n in outs}
        if name is None:
            h.forward(t, out=out)
        else:
            with pytest.raises(ValueError, match="CUDA"):
                h.forward(t, out=out)
    assert no_calls == [(op, 100)]
