"""GPU parity of the rotary insert with positions on several axes, through the binding.

The rows are compared bit for bit with the oracle's: the cos and sin of each pair come
from the table row of the pair's own axis, everything behind that is as for one axis.
"""

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import formats, rotary
from test_gpu_rotary import DEV, DT, _cache, _check, _f32, _inputs

pytestmark = pytest.mark.gpu


def _one_axis(table, pos, axes):
    """A table of one row per token that holds what each pair turns by, and positions 0, 1, ..."""
    half = table.shape[1] // 2
    rows = torch.zeros((pos.shape[1], 2 * half), device=DEV)
    for i, a in enumerate(axes.pairs):
        at = pos[a].long().clamp(0, table.shape[0] - 1)
        rows[:, i], rows[:, half + i] = table[at, i], table[at, half + i]
    return rows, torch.arange(pos.shape[1], device=DEV, dtype=torch.int32)


AXES = {
    "blocks": ops.rope_axes([16, 24, 24]),
    "uneven": ops.rope_axes([5, 0, 41, 18]),
    "dealt": ops.rope_axes([24, 20, 20], dealt=True),
    "two": ops.rope_axes([16, 16]),
    "dealt_two": ops.rope_axes([3, 5], dealt=True),
    "last_only": ops.RopeAxes(3, [2] * 24),
    "any": ops.RopeAxes(4, [(7 * i * i + i // 3) % 4 for i in range(64)]),
    "one": ops.rope_axes([64]),
}


@pytest.mark.parametrize("name", AXES)
@pytest.mark.parametrize("n,inter", [(1, False), (130, True), (77, False)])
@pytest.mark.parametrize("dtype,packed", [("bf16", True), ("f16", False), ("f32", True)])
def test_bytes(name, n, inter, dtype, packed):
    axes = AXES[name]
    parts, slots, _, pages, table = _inputs(n, DT[dtype], n, packed, 2 * len(axes.pairs))
    slots[::9] = -1
    pos = torch.randint(0, 5000, (axes.n_axes, n), generator=torch.Generator(DEV).manual_seed(n), device=DEV, dtype=torch.int32)
    cache, before = _cache(pages, 0xA5)
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4], interleaved=inter, axes=axes)
    rows, at = _one_axis(table, pos, axes)
    _check(parts, slots, at, rows, inter, cache, q8, qi8, before)
    assert cache.read_status() == 0


def test_alike_positions_are_one_axis():
    """Text: every axis counts alike, and the bytes are those of the call with one axis."""
    n = 9001
    parts, slots, pos, pages, table = _inputs(n, torch.bfloat16, 5, True, 128)
    a, b = _cache(pages)[0], _cache(pages)[0]
    want = ops.rotary_insert(a, *parts[:4], table, pos, slots, q_idx=parts[4])
    for axes in (AXES["blocks"], AXES["dealt"], AXES["any"]):
        got = ops.rotary_insert(b, *parts[:4], table, pos.repeat(axes.n_axes, 1), slots, q_idx=parts[4], axes=axes)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(a.kv_pool, b.kv_pool) and torch.equal(a.idx_pool, b.idx_pool)


def test_large_calls_of_several_tiles_a_warp():
    n = 13001
    axes = AXES["dealt"]
    parts, slots, _, pages, table = _inputs(n, torch.float32, 6, False, 128)
    pos = torch.randint(0, 5000, (3, n), device=DEV, dtype=torch.int32)
    a, b = _cache(pages)[0], _cache(pages)[0]
    got = ops.rotary_insert(a, *parts[:4], table, pos, slots, q_idx=parts[4], axes=axes)
    rows, at = _one_axis(table, pos, axes)
    want = ops.rotary_insert(b, *parts[:4], rows, at, slots, q_idx=parts[4])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(a.kv_pool, b.kv_pool) and torch.equal(a.idx_pool, b.idx_pool)


def test_a_bad_position_on_any_axis_leaves_the_token_unturned():
    n, axes = 12, AXES["blocks"]
    parts, slots, _, pages, table = _inputs(n, torch.float32, 7, False, 128)
    pos = torch.randint(0, 5000, (3, n), device=DEV, dtype=torch.int32)
    pos[0, 0], pos[1, 1], pos[2, 2] = -1, 5000, 1 << 30
    cache, _ = _cache(pages)
    q8, _ = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4], axes=axes)
    np.testing.assert_array_equal(q8[:3].cpu().numpy(), formats.encode_e4m3(_f32(parts[0][:3]).astype(np.float64)))
    rows, _ = _one_axis(table, pos, axes)
    turned = rotary.turn_fp32(_f32(parts[0]), rows.cpu().numpy(), False)
    np.testing.assert_array_equal(q8[3:].cpu().numpy(), formats.encode_e4m3(turned[3:].astype(np.float64)))
    assert cache.read_status() == ops.STATUS_BAD_SEQ


def test_arguments():
    parts, slots, pos, pages, table = _inputs(5, torch.float32, 7, False, 128)
    cache, _ = _cache(pages)
    with pytest.raises(ValueError, match="pairs"):
        ops.rotary_insert(cache, *parts[:4], table, pos.repeat(2, 1), slots, axes=AXES["two"])
    with pytest.raises(ValueError, match="positions"):
        ops.rotary_insert(cache, *parts[:4], table, pos, slots, axes=AXES["blocks"])
    with pytest.raises(ValueError, match="positions"):
        ops.rotary_insert(cache, *parts[:4], table, pos.repeat(3, 1).t().contiguous().t(), slots, axes=AXES["blocks"])
