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


@pytest.mark.parametrize("d,blocks", [(16, 3), (48, 3), (52, 2), (64, 2), (100, 2), (136, 2), (188, 2)])
def test_decay_fp32_segments_run_at_once(lib, d, blocks):  # noqa: F811
    """Few long fp32 rows: as many segments as run at once, by the shared memory
    that a block of the read-out pass takes (228 KB an SM, 152 SMs): no second
    round of blocks.  (Where an SM holds one block, to d_k = 128, two rounds of half
    the length are as good: the state pass still runs in one.)  The workspace holds
    a state per segment."""
    h = tln.atlas_decay_create(tln.make_decay_config(H=2, d_k=d, d_v=d, qkv_dtype="f32"))
    segments = tln.atlas_decay_workspace_bytes(h, 1, 32768) // (2 * d * d * 4)
    slices = -(-d // 64)
    assert 0.6 * blocks * 152 <= 2 * slices * segments <= blocks * 152
    tln.atlas_decay_destroy(h)
