"""Cases of the layer operators where they can go wrong: results against the
fp64 oracle at sizes that take each kernel variant, element by element where a
bound on the largest value would hide an error, and the handles' workspaces."""
import numpy as np
import pytest

from oracle import layer
from tests.gpu_common import maxrel
from tests.test_gpu_layer import TOL, TOL_DECAY, _decay_inputs, _decay_ref, _dt, _host

pytestmark = pytest.mark.gpu


def _rms(a):
    return float(np.sqrt(np.mean(np.square(np.asarray(a, np.float64)))))


def _bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16).double().numpy()


# --------------------------------------------------------- decay attention
@pytest.mark.parametrize("dims", [(64, 64), (128, 64), (48, 40), (96, 128)], ids=str)
@pytest.mark.parametrize("B,T", [(2, 600), (160, 140)])
def test_decay_bf16_readouts_carry_only_their_own_rounding(gpu_lib, dims, B, T):
    """Scores and states enter the read-outs' products with 16 bits or more: 2^-16
    of a term, 1/256 of the read-out's rounding of 2^-8.  The two add as squares
    (1 + 2^-16, and a few results rounded to the other side), so the distance
    from the exact read-outs is that of the rounded exact ones to 2 %."""
    import torch
    from test_learned_neural_gb300.runner import DecayAttention
    (dk, dv), H = dims, 2
    t = _decay_inputs(B, H, T, dk, dv, "bf16", 1, "heads", False, True, seed=21, gammas=[0.999, 0.97])
    op = DecayAttention(H, dk, dv)
    out = op.forward(t)
    torch.cuda.synchronize()
    op.status()
    assert op.last_path() == 2
    rows = min(B, 4)
    y, _ = _decay_ref({n: v if n == "decay" else v[:rows] for n, v in t.items()}, "heads", "heads")
    ours, rounding = _rms(_host(out["y"][:rows]) - y), _rms(_bf16(y) - y)
    print(f"{ours:.3e} rounding {rounding:.3e}")
    assert ours <= 1.02 * rounding
