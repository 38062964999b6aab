"""Limits of a call of the layer operators that are refused before any CUDA call."""
import pytest

import test_learned_neural_gb300 as tln
from tests.test_layer_pins import UNS, _refuses, lib  # noqa: F401


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 129, (1 << 31) - 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_refuses_tokens_past_its_index_range(lib, T, dtype):  # noqa: F811
    """A token index plus a segment or a chunk stays below 2^31."""
    h = tln.atlas_decay_create(tln.make_decay_config(H=1, d_k=1, d_v=1, qkv_dtype=dtype))
    io = tln.atlas_decay_io(1, T)
    io.q = io.k = io.v = io.decay = 64            # never dereferenced: validation fails first
    io.y = 128
    _refuses(lib, "decay", h, io, UNS, "2^30")
    assert tln.atlas_decay_workspace_bytes(h, 1, T) == 0
    assert tln.atlas_decay_workspace_bytes(h, 1, 1 << 30) > 0
    tln.atlas_decay_destroy(h)
