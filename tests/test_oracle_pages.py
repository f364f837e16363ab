"""Pins of the page oracle, and the refusals of the page calls and of rotary axes (CPU)."""

import ctypes
import random

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import layout, pages
from test_abi_cpu import _cache, lib  # noqa: F401
from test_oracle_rotary import _row_struct

P = ctypes.c_void_p
FAKE = P(16)


def test_extend_by_hand():
    refs, table, lens = [1, 0, 0, 1, 0], [[0, -1, -1], [3, 2, -1]], [100, 128]
    slots, status = pages.extend(refs, table, lens, [30, 3], 35)
    # sequence 0 fills page 0 and needs one more, the lowest free one; sequence 1 has page 2 in reserve
    assert slots == list(range(100, 128)) + [128, 129] + [256, 257, 258] + [-1, -1]
    assert (refs, table, lens, status) == ([1, 1, 0, 1, 0], [[0, 1, -1], [3, 2, -1]], [130, 131], 0)


def test_extend_runs_dry():
    refs, table, lens = [0, 0, 1], [[-1] * 4, [-1] * 4, [-1] * 4, [2, -1, -1, -1]], [0, 0, 0, 4]
    slots, status = pages.extend(refs, table, lens, [1, 300, 5, 7], 313)
    # the second needs three pages and one is left: neither it nor the third gets any; the fourth needs none
    assert slots == [0] + [-1] * 305 + list(range(2 * 128 + 4, 2 * 128 + 11))
    assert lens == [1, 0, 0, 11] and refs == [1, 0, 1] and status == pages.NO_PAGES


def test_fork_and_release_by_hand():
    refs, table, lens = [1, 1, 0, 0], [[1, 0, -1], [-1] * 3, [-1] * 3, [-1] * 3], [200, 0, 0, 0]
    copies, status = pages.fork(refs, table, lens, [0, 0, 0, 1, 9], [2, 1, 2, 3, 3])
    # the second pair into row 2 and the row outside are left out; row 1 counted as empty when row 3 was made of it
    assert copies == [(0, 2, 72), (0, 3, 72)] and status == pages.BAD_SEQ
    assert table == [[1, 0, -1], [1, 3, -1], [1, 2, -1], [-1] * 3] and lens == [200, 200, 200, 0]
    assert refs == [1, 3, 1, 1]
    assert pages.release(refs, table, lens, [0, 0, 2]) == 0
    assert refs == [0, 1, 0, 1] and table[0] == [-1] * 3 and lens == [0, 200, 0, 0]


def test_counts_add_up():
    rng = random.Random(1)
    refs, table, lens = [0] * 40, [[-1] * 6 for _ in range(8)], [0] * 8
    for _ in range(300):
        op = rng.randrange(3)
        if op == 0:
            new = [rng.choice([0, 0, 1, 100, 200]) for _ in range(8)]
            slots, _ = pages.extend(refs, table, lens, new, sum(new))
            live = [s for s in slots if s >= 0]
            assert len(set(live)) == len(live)
        elif op == 1:
            pages.fork(refs, table, lens, [rng.randrange(8) for _ in range(3)], [rng.randrange(8) for _ in range(3)])
        else:
            pages.release(refs, table, lens, [rng.randrange(8) for _ in range(2)])
        held = [p for r in table for p in r if p >= 0]
        assert refs == [held.count(p) for p in range(40)]
        assert all(sum(p >= 0 for p in r) >= -(-n // 128) for r, n in zip(table, lens))


def test_commit_by_hand():
    rng = np.random.default_rng(2)
    kv = rng.integers(0, 256, (3, layout.KV_PAGE_BYTES), dtype=np.uint8)
    ix = rng.integers(0, 256, (3, layout.IDX_PAGE_BYTES), dtype=np.uint8)
    table, lens = [[2, 0]], [130]
    tokens = [pages.token_bytes(kv, ix, s) for s in [2 * 128 + t for t in range(126, 128)] + [0, 1]]
    keep, keep_ix = kv.copy(), ix.copy()
    new, status = pages.commit(kv, ix, table, lens, [4], [0b1101])  # drafts at 126 .. 129: 1 leaves
    assert (new, status) == ([129], 0)
    for slot, token in ((2 * 128 + 126, tokens[0]), (2 * 128 + 127, tokens[2]), (0, tokens[3])):
        got = pages.token_bytes(kv, ix, slot)
        assert all(np.array_equal(a, b) for a, b in zip(got[0], token[0])) and np.array_equal(got[1], token[1])
    # nothing else changed: 704 bytes of two tokens at most
    assert 0 < np.count_nonzero(kv != keep) <= 2 * 576 and 0 < np.count_nonzero(ix != keep_ix) <= 2 * 128


# ---- refusals -----------------------------------------------------------------------


class _Pool(ctypes.Structure):
    _fields_ = [("refs", P), ("free_mask", P), ("n_pages", ctypes.c_int32), ("status", P)]


def _call(lib, name, *args):  # noqa: F811
    return getattr(lib, name)(*args, None)


def test_page_calls_are_checked_on_the_host(lib):  # noqa: F811
    pool, c = _Pool(16, 16, 4, None), _cache(kv_pool=160, idx_pool=160, n_pages=4)
    layers = ctypes.byref(c)
    ok = ctypes.byref(pool)
    good = {
        "msa_extend_sequences": [ok, FAKE, 4, FAKE, FAKE, 2, 0, FAKE],
        "msa_fork_sequences": [layers, 1, ok, FAKE, 4, FAKE, 2, FAKE, FAKE, 0, FAKE, 1 << 20],
        "msa_release_sequences": [ok, FAKE, 4, FAKE, 2, FAKE, 0],
        "msa_copy_pages": [layers, 1, FAKE, FAKE, None, 0],
        "msa_commit_drafts": [layers, 1, FAKE, 4, FAKE, FAKE, 0, FAKE, P(4096)],
    }
    for name, args in good.items():  # without items nothing is launched
        assert _call(lib, name, *args) == 0, name
    small = ctypes.byref(_Pool(16, 16, 0, None))
    none = ctypes.byref(_Pool(None, 16, 4, None))
    large = ctypes.byref(_Pool(16, 16, 5, None))
    bad = [
        ("msa_extend_sequences", {0: None}, -1), ("msa_extend_sequences", {0: small}, -1), ("msa_extend_sequences", {0: none}, -1),
        ("msa_extend_sequences", {1: None}, -1), ("msa_extend_sequences", {2: 0}, -1), ("msa_extend_sequences", {2: 65537}, -2),
        ("msa_extend_sequences", {5: 4097}, -2), ("msa_extend_sequences", {5: -1}, -1), ("msa_extend_sequences", {6: -1}, -1),
        ("msa_extend_sequences", {6: 262145}, -2), ("msa_extend_sequences", {4: None}, -1), ("msa_extend_sequences", {6: 1, 7: None}, -1),
        ("msa_extend_sequences", {6: 1, 5: 0}, -1),
        ("msa_fork_sequences", {0: None}, -1), ("msa_fork_sequences", {1: 0}, -1), ("msa_fork_sequences", {1: 129}, -2),
        ("msa_fork_sequences", {2: large}, -1), ("msa_fork_sequences", {9: 4097}, -2), ("msa_fork_sequences", {9: 2, 7: None}, -1),
        ("msa_fork_sequences", {9: 2, 11: 31}, -3), ("msa_fork_sequences", {10: P(8)}, -1), ("msa_fork_sequences", {9: -1}, -1),
        ("msa_release_sequences", {3: None}, -1), ("msa_release_sequences", {6: 1, 5: None}, -1), ("msa_release_sequences", {6: 4097}, -2),
        ("msa_copy_pages", {5: -1}, -1), ("msa_copy_pages", {5: 1, 2: None}, -1), ("msa_copy_pages", {1: 129}, -2),
        ("msa_commit_drafts", {5: None}, -1), ("msa_commit_drafts", {6: 1, 7: None}, -1), ("msa_commit_drafts", {6: 1, 8: FAKE}, -1),
        ("msa_commit_drafts", {6: 4, 8: P(28)}, -1), ("msa_commit_drafts", {6: 4097}, -2),
    ]
    for name, change, code in bad:
        args = [change.get(i, a) for i, a in enumerate(good[name])]
        assert _call(lib, name, *args) == code, (name, change)
    off = _cache(kv_pool=168, idx_pool=160, n_pages=4)
    assert _call(lib, "msa_copy_pages", ctypes.byref(off), 1, FAKE, FAKE, None, 0) == -1
    assert lib.msa_fork_workspace_bytes(3) == 48 and lib.msa_fork_workspace_bytes(0) == 16
    assert lib.msa_status_string(0x20) == b"device: no free page was left in the page pool"


def test_axes_are_checked_on_the_host(lib):  # noqa: F811
    c, rows = _cache(kv_pool=160, idx_pool=160, n_pages=4), _row_struct()

    def call(n_axes, pairs, rot=64):
        return lib.msa_rotary_insert_axes(ctypes.byref(c), ctypes.byref(rows), 0, FAKE, 8, rot, 0, FAKE, n_axes, pairs, FAKE, FAKE, FAKE, None)

    assert call(3, bytes([0, 1, 2, 2] * 8)) == 0
    assert call(1, None) == 0 and call(1, bytes([7] * 32)) == 0  # not read for one axis
    assert call(3, bytes([0, 1, 2, 3] * 8)) == -1 and call(2, None) == -1
    assert call(0, bytes(32)) == -2 and call(5, bytes(32)) == -2
    assert call(2, None, rot=0) == 0


def test_rope_axes():
    a = ops.rope_axes([2, 3, 3])
    assert a.n_axes == 3 and list(a.pairs) == [0, 0, 1, 1, 1, 2, 2, 2]
    # dealt: 0 1 2 0 1 2 0 .. while an axis has some left
    assert list(ops.rope_axes([4, 2, 2], dealt=True).pairs) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(ops.rope_axes([0, 1], dealt=True).pairs) == [0]
    for bad in ([], [1, -1], [1] * 5):
        with pytest.raises(ValueError):
            ops.rope_axes(bad)
    with pytest.raises(ValueError):
        ops.RopeAxes(2, [0, 2])


def test_page_pool_needs_a_gpu_tensor():
    with pytest.raises(ValueError, match="CUDA"):
        ops.PagePool.from_refs(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        ops.PagePool.from_refs(torch.zeros(4))


def test_a_fork_leaves_a_row_alone_that_holds_a_page_behind_a_hole():
    for at in (0, 1, 2):
        refs, table, lens = [1, 1, 0, 0], [[0, -1, -1], [-1, -1, -1], [-1, -1, -1]], [5, 0, 0]
        table[1][at] = 1
        copies, status = pages.fork(refs, table, lens, [0, 0], [1, 2])
        assert copies == [(0, 2, 5)] and status == pages.BAD_SEQ and lens == [5, 0, 5]
        assert table[1][at] == 1 and refs == [1, 1, 1, 0]


def test_a_fork_runs_dry():
    refs, table, lens = [1, 1, 0, 1, 1], [[0, 1], [3, -1], [4, -1]] + [[-1, -1] for _ in range(5)], [140, 128, 7, 0, 0, 0, 0, 0]
    # the second pair finds no page any more, nor does the fourth; the third and the fifth need none
    copies, status = pages.fork(refs, table, lens, [0, 2, 1, 0, 7], [3, 4, 5, 6, 6])
    assert copies == [(1, 2, 12)] and status & pages.NO_PAGES
    assert lens == [140, 128, 7, 140, 0, 128, 0, 0] and refs == [2, 1, 1, 2, 1]
    assert table[3:] == [[0, 2], [-1, -1], [3, -1], [-1, -1], [-1, -1]]


def test_extend_grows_none_where_starts_go_back():
    refs, table, lens = [1, 0, 0, 0], [[0, -1], [-1, -1], [-1, -1]], [4, 0, 0]
    slots, status = pages.extend(refs, table, lens, [30, -20, 9], 30)
    assert slots == [-1] * 30 and status == pages.BAD_SEQ
    assert (refs, lens, table) == ([1, 0, 0, 0], [4, 0, 0], [[0, -1], [-1, -1], [-1, -1]])
