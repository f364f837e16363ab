"""Pins of the tree-attention oracle, and the host validation of its entry point (CPU)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from nvfp4_kv_block_gb300 import ops
from oracle import formats, layout, nvfp4, tree
from test_abi_cpu import _cache, lib  # noqa: F401


def test_page_operands_equal_the_slot_reader():
    rng = np.random.default_rng(0)
    pool = rng.integers(0, 256, (1, layout.KV_PAGE_BYTES), dtype=np.uint8)
    for g in range(4):
        for off in (8192, 17408):
            pool[0, g * 18432 + off: g * 18432 + off + 1024] = rng.integers(0, 0x7F, 1024)
    k8, v8 = tree.page_operands(pool[0])
    for t in (0, 1, 2, 63, 100, 127):
        kc, ks, vc, vs = layout.read_kv_slot(pool, 0, t)
        np.testing.assert_array_equal(k8[t], nvfp4.fp8_operand(kc, ks))
        np.testing.assert_array_equal(v8[t], nvfp4.fp8_operand(vc, vs))


def test_visible_by_hand():
    got = tree.visible(3, 3, [0b001, 0b011, 0b101], list(range(7)))
    want = [[1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0], [1, 1, 1, 1, 0, 1, 0]]
    np.testing.assert_array_equal(got, np.array(want, bool))
    got = tree.visible(300, 1, None, [0, 127, 128, 255, 256, 299, 300, 301], sel=[1])
    np.testing.assert_array_equal(got[0], np.array([0, 0, 1, 1, 1, 1, 1, 0], bool))


def test_a_chain_is_the_causal_attention_of_the_decode_oracle():
    rng = np.random.default_rng(1)
    ctx, n = 40, 3
    k8 = formats.encode_e4m3(rng.standard_normal((ctx + n, 4, 128)) * 20)
    v8 = formats.encode_e4m3(rng.standard_normal((ctx + n, 4, 128)) * 20)
    q8 = formats.encode_e4m3(rng.standard_normal((n, 16, 128)))
    out, lse, _, _ = tree.attend(q8, k8, v8, tree.visible(ctx, n, None, range(ctx + n)), 0.09, 30.0, 20.0)
    for j in range(n):
        o, l = oracle.attention.attend(q8[j], k8[: ctx + j + 1], v8[: ctx + j + 1], np.float32(0.09), 30.0, 20.0)
        np.testing.assert_allclose(out[j], o, rtol=0, atol=1e-6)
        np.testing.assert_allclose(lse[j], l, rtol=0, atol=1e-6)


def test_one_key_and_no_key():
    v8 = formats.encode_e4m3(np.arange(3 * 4 * 128).reshape(3, 4, 128) % 97 - 40.0)
    seen = np.array([[0, 1, 0], [0, 0, 0]], bool)
    out, lse, mean, _ = tree.attend(np.zeros((2, 16, 128), np.uint8), v8, v8, seen, 1.0, 1.0, 2.0)
    np.testing.assert_array_equal(out[0, 5], formats.decode_e4m3(v8[1, 1]) / 2)
    assert np.all(lse[0] == 0) and np.all(np.isneginf(lse[1])) and not out[1].any()


def test_validation_needs_no_gpu(lib):  # noqa: F811
    fake, c = ctypes.c_void_p(16), _cache(kv_pool=16)
    big = 1 << 32

    def call(cache=c, q=fake, heads=16, scale=0.1, bt=fake, max_pages=4, lens=fake, qsl=fake, n_seqs=1, T=1, mask=None,
             sel=None, n_sel=None, dtype=1, out=fake, lse=fake, ws=fake, ws_bytes=big):
        return lib.msa_tree_attn(ctypes.byref(cache), q, heads, scale, bt, max_pages, lens, qsl, n_seqs, T, mask, sel,
                                 n_sel, dtype, out, lse, ws, ws_bytes, None)

    assert call(cache=_cache(n_kv_heads=8)) == -2 and call(heads=8) == -2
    assert call(scale=0.0) == -1 and call(scale=float("nan")) == -1
    assert call(dtype=0) == -1 and call(dtype=3) == -1
    assert call(sel=fake) == -1 and call(n_sel=fake) == -1
    assert call(max_pages=0) == -1 and call(n_seqs=0) == -1 and call(T=-1) == -1
    assert call(T=65536) == -2 and call(n_seqs=4097) == -2 and call(max_pages=65537) == -2
    assert call(q=ctypes.c_void_p(8)) == -1 and call(out=ctypes.c_void_p(8)) == -1 and call(ws=ctypes.c_void_p(8)) == -1
    assert call(out=None) == -1 and call(bt=None) == -1
    assert call(ws_bytes=lib.msa_tree_attn_workspace_bytes(1) - 1) == -3
    assert call(scale=3e38) == -1
    # 64 drafts fill two row tiles: more tokens need no more
    a, b = lib.msa_tree_attn_workspace_bytes(64), lib.msa_tree_attn_workspace_bytes(128)
    assert a == b and lib.msa_tree_attn_workspace_bytes(0) == 256


def test_binding_checks():
    with pytest.raises(TypeError):
        ops.TreeBuffers(4, 1, torch.float32, "cpu")
    bufs = ops.TreeBuffers(4, 1, torch.float16, "cpu")
    i32 = torch.int32
    args = [None, torch.zeros(4, 16, 128, dtype=torch.uint8), torch.zeros(1, 4, dtype=i32), torch.zeros(1, dtype=i32),
            torch.zeros(2, dtype=i32), bufs]
    with pytest.raises(ValueError):  # more sequences than the buffers are for
        ops.tree_attn(*args[:2], torch.zeros(2, 4, dtype=i32), *args[3:])
    with pytest.raises(ValueError):
        ops.tree_attn(*args, sel=torch.zeros(1, 17, dtype=i32))
    with pytest.raises(ValueError):
        ops.tree_attn(*args, n_sel=torch.zeros(1, dtype=i32))
