"""Pins of the rotary oracle, and the rotary frequencies and their refusals (CPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from nvfp4_kv_block_gb300 import ops
from test_abi_cpu import _cache, lib  # noqa: F401


@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_turn_is_complex_multiplication(rot, inter):
    rng = np.random.default_rng(rot + inter)
    x = rng.standard_normal((5, 3, 128))
    ang = rng.uniform(-7, 7, (5, rot // 2))
    y = oracle.rotary.turn(x, np.concatenate([np.cos(ang), np.sin(ang)], 1), inter)
    a, b = ((x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot]))
    c, d = ((y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., : rot // 2], y[..., rot // 2: rot]))
    z = (a + 1j * b) * np.exp(1j * ang)[:, None]
    # one product of complex numbers in float64: a few units of 2^-53 of values below 10
    np.testing.assert_allclose(c + 1j * d, z, rtol=0, atol=64 * 2.0**-53)
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])


def test_turn_by_hand():
    x = np.zeros((1, 1, 128))
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 8] = 1.0, 2.0, 3.0
    t = np.zeros((1, 16))
    t[0, 8:] = 1.0  # a quarter turn of every pair: (a, b) -> (-b, a)
    half = oracle.rotary.turn(x, t, False)[0, 0]
    assert (half[0], half[1], half[8], half[9]) == (-3.0, 0.0, 1.0, 2.0)
    inter = oracle.rotary.turn(x, t, True)[0, 0]
    assert (inter[0], inter[1], inter[8], inter[9]) == (-2.0, 1.0, 0.0, 3.0)


def test_half_pairs_of_whole_heads_equal_the_fused_projections_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 128))
    ang = rng.uniform(0, 9, (4, 64))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    want = np.stack([oracle.qkv.rope(x[:, h], cs) for h in range(2)], 1)
    np.testing.assert_allclose(oracle.rotary.turn(x, cs, False), want, rtol=0, atol=32 * 2.0**-53)


def test_fp32_steps_stay_near_the_float64_rotation():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 2, 128)).astype(np.float32)
    ang = rng.uniform(0, 1000, (64, 48))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    a, b = oracle.rotary.turn(x, cs, True), oracle.rotary.turn_fp32(x, cs, True)
    # three roundings, each of at most 2^-24 of a value below |a| + |b|
    bound = 3 * 2.0**-24 * (np.abs(x).reshape(64, 2, 64, 2).sum(-1).repeat(2, -1))
    assert np.all(np.abs(a - b) <= bound)


def test_slot_values_by_hand():
    kv = np.zeros((1, oracle.layout.KV_PAGE_BYTES), np.uint8)
    ix = np.zeros((1, oracle.layout.IDX_PAGE_BYTES), np.uint8)
    codes = np.zeros((4, 128), np.uint8)
    codes[1, 17], codes[1, 18] = 7, 8 | 3   # 6 and -1.5
    scales = np.zeros((4, 8), np.uint8)
    scales[1, 1] = 0x40                     # 2.0
    oracle.layout.write_kv_slot(kv, 0, 77, codes, scales, codes, scales)
    key = np.zeros(128, np.uint8)
    key[100] = 0xB8                          # -1.0
    oracle.layout.write_index_slot(ix, 0, 77, key)
    k, v, i = oracle.rotary.slot_values(kv, ix, 77, 4.0, 8.0)
    assert k[1, 17] == 3.0 and k[1, 18] == -0.75 and v[1, 17] == 1.5 and i[100] == -1.0
    assert np.count_nonzero(k) == 2 and np.count_nonzero(i) == 1


# ---- frequencies ------------------------------------------------------------------


def test_frequencies_unscaled_linear_ntk():
    f, amp = ops.rope_frequencies(64, 10000.0)
    assert amp == 1.0 and f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64), rel_tol=1e-15)
    g, _ = ops.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert all(math.isclose(a, b / 4, rel_tol=1e-15) for a, b in zip(g, f))
    h, _ = ops.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert h[0] == 1.0 and math.isclose(h[31], f[31] / 4, rel_tol=1e-12)  # the slowest pair is stretched by the factor
    assert ops.rope_frequencies(0) == ([], 1.0)


def test_frequencies_by_parts():
    f, _ = ops.rope_frequencies(128, 10000.0)
    g, amp = ops.rope_frequencies(128, 10000.0, "yarn", 8.0, 4096)
    assert math.isclose(amp, 0.1 * math.log(8.0) + 1.0)
    turns = [4096 * x / (2 * math.pi) for x in f]
    for i, (a, b) in enumerate(zip(f, g)):
        if turns[i] > 40:
            assert a == b
        if turns[i] < 0.8:
            assert math.isclose(b, a / 8, rel_tol=1e-15)
        assert a / 8 * (1 - 1e-15) <= b <= a
    ratio = [b / a for a, b in zip(f, g)]
    assert all(x >= y for x, y in zip(ratio, ratio[1:]))


@pytest.mark.parametrize("kw", [dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="cubic"),
                                dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=64, scaling="linear", factor=0.5),
                                dict(rot_dim=64, scaling="yarn", factor=2.0, original_max_pos=10, beta_fast=1.0, beta_slow=2.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        ops.rope_frequencies(**kw)


# ---- host validation of the C entry points ------------------------------------------


def _row_struct(**kw):
    r = ops._Rows(16, 16, 16, 16, 16, 2048, 512, 512, 128, 1024, 1)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_rotary_insert_validation_needs_no_gpu(lib):  # noqa: F811
    fake, c = ctypes.c_void_p(16), _cache()

    def call(r=None, n=1, cs=fake, max_pos=8, rot=64, inter=0, pos=fake, slots=fake, q8=fake, qi8=fake, cache=c):
        return lib.msa_rotary_insert(ctypes.byref(cache), ctypes.byref(r or _row_struct()), n, cs, max_pos, rot, inter,
                                     pos, slots, q8, qi8, None)

    assert call(cache=_cache(head_dim=64)) == -2
    assert call(rot=24) == -2 and call(rot=144) == -2 and call(rot=-16) == -2
    assert call(n=-1) == -1 and call(inter=2) == -1 and call(max_pos=0) == -1
    assert call(r=_row_struct(dtype=3)) == -1 and call(r=_row_struct(k=None)) == -1
    assert call(r=_row_struct(q_stride=2049)) == -1 and call(r=_row_struct(v=24)) == -1 and call(r=_row_struct(k_stride=-8)) == -1
    assert call(q8=None) == -1 and call(qi8=None) == -1 and call(cs=None) == -1 and call(slots=None) == -1
    assert call(q8=ctypes.c_void_p(24)) == -1
    assert lib.msa_rotary_insert(ctypes.byref(c), None, 1, fake, 8, 64, 0, fake, fake, fake, fake, None) == -1


def test_rope_table_freqs_validation_needs_no_gpu(lib):  # noqa: F811
    fake = ctypes.c_void_p(16)
    good = (ctypes.c_double * 8)(*range(8))
    bad = (ctypes.c_double * 8)(*([1.0] * 7 + [float("inf")]))
    assert lib.msa_rope_table_freqs(fake, 4, good, 24, 1.0, None) == -2
    assert lib.msa_rope_table_freqs(fake, 4, bad, 16, 1.0, None) == -1
    assert lib.msa_rope_table_freqs(fake, 4, good, 16, float("nan"), None) == -1
    assert lib.msa_rope_table_freqs(None, 4, good, 16, 1.0, None) == -1
    assert lib.msa_rope_table_freqs(fake, -1, good, 16, 1.0, None) == -1


def test_read_kv_validation_needs_no_gpu(lib):  # noqa: F811
    fake, c = ctypes.c_void_p(16), _cache()
    assert lib.msa_read_kv(ctypes.byref(c), fake, -1, 1, fake, fake, fake, None) == -1
    assert lib.msa_read_kv(ctypes.byref(c), None, 1, 1, fake, fake, fake, None) == -1
    assert lib.msa_read_kv(ctypes.byref(c), fake, 1, 3, fake, fake, fake, None) == -1
    assert lib.msa_read_kv(ctypes.byref(c), fake, 1, 1, ctypes.c_void_p(24), fake, fake, None) == -1
    assert lib.msa_read_kv(ctypes.byref(_cache(idx_dim=64)), fake, 1, 1, fake, fake, fake, None) == -2


def test_row_checks_of_the_binding():
    n, f32, cpu = 3, torch.float32, -1  # (get_device() of a CPU tensor)
    x = torch.zeros(n, 33, 128)
    shape = (n, 4, 128)
    assert ops._rows(x[:, 16:20], "k", shape, f32, cpu) == (x.data_ptr() + 16 * 512, 33 * 128)
    assert ops._rows(x[:, 24], "idx_k", (n, 128), f32, cpu)[1] == 33 * 128
    with pytest.raises(TypeError):
        ops._rows(x[:, :4].half(), "k", shape, f32, cpu)
    with pytest.raises(TypeError):
        ops._rows(x[:, :4].numpy(), "k", shape, f32, cpu)
    with pytest.raises(ValueError):
        ops._rows(x[:, :5], "k", shape, f32, cpu)
    with pytest.raises(ValueError):  # another device
        ops._rows(x[:, :4], "k", shape, f32, 0)
    with pytest.raises(ValueError):  # heads not contiguous
        ops._rows(x[:, :8:2], "k", shape, f32, cpu)
    with pytest.raises(ValueError):  # channels not contiguous
        ops._rows(torch.zeros(n, 4, 256)[:, :, ::2], "k", shape, f32, cpu)
    with pytest.raises(ValueError):  # token stride off 16 bytes
        ops._rows(torch.zeros(n * 514).as_strided((n, 4, 128), (514, 128, 1)), "k", shape, f32, cpu)
    with pytest.raises(ValueError):  # base off 16 bytes
        ops._rows(torch.zeros(n * 512 + 1)[1:].view(n, 4, 128), "k", shape, f32, cpu)


def test_argument_checks_of_the_binding():
    x = torch.zeros(4, 6, dtype=torch.int32)
    for t, dtype, shape, dev, error in ((x, torch.int64, (4, 6), -1, TypeError), ([1, 2], torch.int32, (2,), -1, TypeError),
                                        (x, torch.int32, (4, 6), 0, ValueError), (x, torch.int32, (6, 4), -1, ValueError),
                                        (x.t(), torch.int32, (6, 4), -1, ValueError)):
        with pytest.raises(error):
            ops._arg(t, dtype, shape, dev, "x")
