"""GPU parity of the rotary insert and of the read-back, through the binding.

The rotation's roundings are documented step by step (two products and a sum in
fp32), so FP8 queries and cache bytes are compared bit for bit with the oracle's
quantisers on rows that NumPy turned in the same steps; FP8 queries are also held
to the float64 rotation: half an E4M3 step (2^-4 relative, 2^-10 near zero), and
three fp32 roundings of values up to |a| + |b| before it.  Read-back values have
one documented rounding each and are compared bit for bit.
"""

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import formats, layout, nvfp4, rotary

pytestmark = pytest.mark.gpu

DEV = "cuda"
S_ENC_K, S_ENC_V = 448.0 / 5.0, 448.0 / 6.5
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _inputs(n, dtype, seed, packed, rot, max_pos=5000, n_pages=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows = torch.randn((n, 33, 128), generator=g, device=DEV).to(dtype)
    parts = [rows[:, :16], rows[:, 16:20], rows[:, 20:24], rows[:, 24], rows[:, 25:33]]
    if not packed:
        parts = [p.contiguous() for p in parts]
    pages = n_pages or -(-max(n, 1) // 128) + 1
    slots = torch.randperm(pages * 128, generator=g, device=DEV)[:n]
    pos = torch.randint(0, max_pos, (n,), generator=g, device=DEV, dtype=torch.int32)
    return parts, slots, pos, pages, ops.rope_table_scaled(max_pos, rot, device=DEV)


def _f32(t):
    return t.float().cpu().numpy()


def _check(parts, slots, pos, table, inter, cache, q8, qi8, before):
    q, k, v, ik, qi = (_f32(p) for p in parts)
    cs = table.cpu().numpy()[pos.cpu().numpy()]
    turned = {name: rotary.turn_fp32(x, cs, inter) for name, x in (("q", q), ("k", k), ("ik", ik[:, None]), ("qi", qi))}
    for got, name, x in ((q8, "q", q), (qi8, "qi", qi)):
        got = got.cpu().numpy()
        np.testing.assert_array_equal(got, formats.encode_e4m3(turned[name].astype(np.float64)))
        exact = rotary.turn(x, cs, inter)
        size = np.abs(x).max(-1, keepdims=True) * 2
        err = np.abs(formats.decode_e4m3(got) - np.clip(exact, -448, 448))
        assert np.all(err <= 2.0**-4 * np.abs(exact) + 2.0**-10 + 3 * 2.0**-24 * size)
    kv, ix = before
    kc, ks = nvfp4.quantize(turned["k"], S_ENC_K)
    vc, vs = nvfp4.quantize(v, S_ENC_V)
    i8 = formats.encode_e4m3(turned["ik"][:, 0].astype(np.float64))
    for t, slot in enumerate(slots.cpu().tolist()):
        if 0 <= slot < kv.shape[0] * 128:
            layout.write_kv_slot(kv, slot // 128, slot % 128, kc[t], ks[t], vc[t], vs[t])
            layout.write_index_slot(ix, slot // 128, slot % 128, i8[t])
    np.testing.assert_array_equal(cache.kv_pool.cpu().numpy(), kv)
    np.testing.assert_array_equal(cache.idx_pool.cpu().numpy(), ix)


def _cache(pages, fill=0):
    cache = ops.KVCache(pages, S_ENC_K, S_ENC_V, DEV)
    cache.kv_pool.fill_(fill)
    cache.idx_pool.fill_(fill)
    return cache, (cache.kv_pool.cpu().numpy().copy(), cache.idx_pool.cpu().numpy().copy())


@pytest.mark.parametrize("n", [1, 2, 7, 129])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, True), (48, False), (16, False), (0, False)])
@pytest.mark.parametrize("dtype,packed", [("bf16", True), ("f16", False), ("f32", True)])
def test_bytes(n, rot, inter, dtype, packed):
    parts, slots, pos, pages, table = _inputs(n, DT[dtype], 7 * n + rot, packed, rot)
    cache, before = _cache(pages, 0xA5)  # untouched bytes have to stay
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4], interleaved=inter)
    _check(parts, slots, pos, table, inter, cache, q8, qi8, before)
    assert cache.read_status() == 0


def test_large_call_in_page_order_and_without_index_queries():
    n = 5000
    parts, slots, pos, pages, table = _inputs(n, torch.bfloat16, 3, True, 64)
    slots = torch.arange(n, device=DEV) + 31
    cache, before = _cache(pages)
    q8, none = ops.rotary_insert(cache, *parts[:4], table, pos, slots, interleaved=True)
    assert none is None
    want = ops.rotary_insert(_cache(pages)[0], *parts[:4], table, pos, slots, q_idx=parts[4], interleaved=True)
    assert torch.equal(q8, want[0])
    _check(parts, slots, pos, table, True, cache, q8, want[1], before)


@pytest.mark.parametrize("n", [6500, 13001, 20011])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_large_call_equals_small_ones(n, dtype):
    """Warps with several tiles each, the last ones partly empty, scattered and in runs."""
    parts, slots, pos, pages, table = _inputs(n, DT[dtype], n, True, 64)
    slots[1000:3000] = torch.arange(pages * 128, pages * 128 + 2000, device=DEV)
    pages += 17
    slots[77::501] = -1
    a, b = _cache(pages)[0], _cache(pages)[0]
    q8, qi8 = ops.rotary_insert(a, *parts[:4], table, pos, slots, q_idx=parts[4])
    for lo in range(0, n, 1000):
        c = slice(lo, lo + 1000)
        w8, wi8 = ops.rotary_insert(b, *(p[c] for p in parts[:4]), table, pos[c], slots[c], q_idx=parts[4][c])
        assert torch.equal(q8[c], w8) and torch.equal(qi8[c], wi8)
    assert torch.equal(a.kv_pool, b.kv_pool) and torch.equal(a.idx_pool, b.idx_pool)
    assert a.read_status() == 0


def test_skipped_and_bad_slots_and_positions():
    n = 40
    parts, slots, pos, pages, table = _inputs(n, torch.float32, 11, False, 128)
    slots[::5] = -1
    cache, before = _cache(pages, 0x11)
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4])
    _check(parts, slots, pos, table, False, cache, q8, qi8, before)
    assert cache.read_status() == 0
    # a slot behind the pool is left out and flagged
    slots[3] = pages * 128
    cache, before = _cache(pages, 0x11)
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4])
    _check(parts, slots, pos, table, False, cache, q8, qi8, before)
    assert cache.read_status() == ops.STATUS_BAD_SLOT
    # positions outside the table leave the token unturned and are flagged
    cache, _ = _cache(pages)
    bad = pos.clone()
    bad[0], bad[1] = -1, 5000
    q8, _ = ops.rotary_insert(cache, *parts[:4], table, bad, slots.clamp(max=pages * 128 - 1), q_idx=parts[4])
    np.testing.assert_array_equal(q8[:2].cpu().numpy(), formats.encode_e4m3(_f32(parts[0][:2]).astype(np.float64)))
    assert cache.read_status() == ops.STATUS_BAD_SEQ
    # without a rotation there is no position to be wrong
    cache, _ = _cache(pages)
    ops.rotary_insert(cache, *parts[:4], table[:, :0].contiguous(), bad, slots.clamp(max=pages * 128 - 1), q_idx=parts[4])
    assert cache.read_status() == 0


def test_no_tokens():
    parts, slots, pos, pages, table = _inputs(0, torch.bfloat16, 1, False, 64)
    cache, before = _cache(1, 0x33)
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4])
    assert q8.shape == (0, 16, 128) and qi8.shape == (0, 8, 128)
    k, v, ik = ops.read_kv(cache, slots)
    assert k.shape == (0, 4, 128) and ik.shape == (0, 128)
    np.testing.assert_array_equal(cache.kv_pool.cpu().numpy(), before[0])


def test_large_values_saturate_and_infinities_stay_finite():
    parts, slots, pos, pages, table = _inputs(4, torch.float32, 2, False, 64)
    parts[0][0] *= 1e5
    parts[1][1, 2, 5] = float("inf")
    parts[2][2, 1] = 0.0
    cache, before = _cache(pages)
    zero = torch.zeros_like(pos)  # position 0 turns by nothing: infinities stay alone
    q8, qi8 = ops.rotary_insert(cache, *parts[:4], table[:, :0].contiguous(), zero, slots, q_idx=parts[4])
    _check(parts, slots, zero, table[:, :0], False, cache, q8, qi8, before)
    k, v, _ = ops.read_kv(cache, slots, dtype=torch.float32)
    assert torch.isfinite(k).all() and torch.count_nonzero(v[2, 1]) == 0


def test_codes_at_and_next_to_every_midpoint_and_of_values_that_are_none():
    """Values on, one ulp below and one ulp above each E2M1 midpoint under every scale, of both
    signs, and NaN and infinities: the bytes of quantize_kv_insert."""
    scales = np.arange(1, 127, dtype=np.uint8)
    sb = formats.decode_e4m3(scales).astype(np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    n = len(sb)
    x = np.zeros((n, 4, 8, 16), np.float32)
    # with s_enc = 1 the group's scale is E4M3(max / 6): one value 6 sb sets it
    t = (mids[None] * sb[:, None]).astype(np.float32)
    x[..., 0] = 6 * sb[:, None, None]
    for g, y in enumerate((t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(1e9)), 0.5 * t)):
        x[:, :, g, 1:8], x[:, :, g, 8:15] = y[:, None], -y[:, None]
    x[:, 1, 4, 3], x[:, 1, 5, 4], x[:, 2, 6, 5], x[:, 3, 7, 6] = np.nan, np.inf, -np.inf, 1e38
    k = torch.from_numpy(x.reshape(n, 4, 128)).to(DEV)
    ik = torch.zeros((n, 128), device=DEV)
    slots = torch.arange(n, device=DEV)
    for s_enc in (1.0, 1e3):
        a, b = (ops.KVCache(1, s_enc, 1.0, DEV) for _ in range(2))
        ops.quantize_kv_insert(a, k, k.neg(), ik, slots)
        ops.rotary_insert(b, torch.zeros((n, 16, 128), device=DEV), k, k.neg(), ik, torch.zeros((1, 0), device=DEV),
                          torch.zeros(n, dtype=torch.int32, device=DEV), slots)
        assert torch.equal(a.kv_pool, b.kv_pool)


def test_table_of_given_frequencies():
    for rot, scaling, factor in ((128, None, 1.0), (64, "yarn", 8.0), (96, "ntk", 2.0), (16, "linear", 4.0)):
        t = ops.rope_table_scaled(3000, rot, 500000.0, scaling, factor, 1000, device=DEV).cpu().numpy()
        f, amp = ops.rope_frequencies(rot, 500000.0, scaling, factor, 1000)
        ang = np.arange(3000)[:, None] * np.array(f)
        want = np.concatenate([np.cos(ang), np.sin(ang)], 1) * amp
        # float64 cos and sin of both sides differ by a few units of 2^-53; the fp32 rounding adds half a step
        assert np.all(np.abs(t - want) <= 2.0**-24 * np.abs(want) + 2.0**-50)
    assert torch.equal(ops.rope_table_scaled(300, device=DEV), ops.rope_table(300, device=DEV))


# ---- read-back ------------------------------------------------------------------------


def _filled(pages, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cache = ops.KVCache(pages, S_ENC_K, S_ENC_V, DEV)
    cache.kv_pool.copy_(torch.randint(0, 256, cache.kv_pool.shape, generator=g, device=DEV, dtype=torch.uint8))
    # scale bytes 0x00 .. 0x7E: every finite scale, zero and subnormal ones too
    heads = cache.kv_pool.view(pages, 4, 18432)
    for lo in (8192, 17408):
        heads[:, :, lo: lo + 1024] = torch.randint(0, 127, (pages, 4, 1024), generator=g, device=DEV, dtype=torch.uint8)
    idx = torch.randint(0, 127, cache.idx_pool.shape, generator=g, device=DEV, dtype=torch.uint8)
    sign = torch.randint(0, 2, cache.idx_pool.shape, generator=g, device=DEV, dtype=torch.uint8)
    cache.idx_pool.copy_(idx | (sign << 7))
    return cache, g


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 33, 700])
def test_read_values(n, dtype):
    cache, g = _filled(6, n)
    slots = torch.randint(0, 6 * 128, (n,), generator=g, device=DEV)  # repeats are fine
    got = ops.read_kv(cache, slots, dtype=DT[dtype])
    kv, ix = cache.kv_pool.cpu().numpy(), cache.idx_pool.cpu().numpy()
    want = [np.stack(x) for x in zip(*(rotary.slot_values(kv, ix, s, S_ENC_K, S_ENC_V) for s in slots.cpu().tolist()))]
    for a, b in zip(got, want):
        assert a.dtype == DT[dtype] and torch.equal(a.cpu(), torch.from_numpy(b).to(DT[dtype]))
    assert cache.read_status() == 0


def test_read_into_given_rows_leaves_the_others():
    cache, g = _filled(3, 5)
    n = 50
    slots = torch.randperm(3 * 128, generator=g, device=DEV)[:n]
    slots[7], slots[8], slots[9] = -1, 3 * 128, -(1 << 40)
    k = torch.full((n, 4, 128), 7.0, dtype=torch.float16, device=DEV)
    ret = ops.read_kv(cache, slots, k=k)
    assert ret[0] is k and ret[1] is None and ret[2] is None
    assert torch.all(k[7:10] == 7.0) and cache.read_status() == ops.STATUS_BAD_SLOT
    full = ops.read_kv(cache, slots.clamp(0, 383), dtype=torch.float16)[0]
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[7:10] = False
    assert torch.equal(k[keep], full[keep])
    idx = torch.zeros((n, 128), dtype=torch.float32, device=DEV)
    ops.read_kv(cache, slots.clamp(0, 383), idx_k=idx)
    assert torch.equal(idx, ops.read_kv(cache, slots.clamp(0, 383), dtype=torch.float32)[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_and_outputs_that_begin_at_16_bytes(dtype):
    """Inputs and outputs 16 bytes into their storage (no wider alignment) as from the front."""
    n, t = 300, DT[dtype]
    e = 16 // torch.empty((), dtype=t).element_size()
    parts, slots, pos, pages, table = _inputs(n, t, 41, False, 64)

    def shifted(x):
        y = torch.empty(x.numel() + e, dtype=x.dtype, device=DEV)[e:].view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)

    a, b = _cache(pages)[0], _cache(pages)[0]
    want = ops.rotary_insert(a, *parts[:4], table, pos, slots, q_idx=parts[4])
    got = ops.rotary_insert(b, *(shifted(x) for x in parts[:4]), table, pos, slots, q_idx=shifted(parts[4]))
    assert torch.equal(a.kv_pool, b.kv_pool) and torch.equal(a.idx_pool, b.idx_pool)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    outs = [shifted(torch.zeros(shape, dtype=t, device=DEV)) for shape in ((n, 4, 128), (n, 4, 128), (n, 128))]
    ops.read_kv(a, slots, k=outs[0], v=outs[1], idx_k=outs[2])
    for x, y in zip(outs, ops.read_kv(a, slots, dtype=t)):
        assert torch.equal(x, y)


def test_written_rows_come_back():
    """Insert with this call, read back, and the same bytes through quantize_kv_insert."""
    n = 200
    parts, slots, pos, pages, table = _inputs(n, torch.float32, 21, False, 0)
    cache, _ = _cache(pages)
    ops.rotary_insert(cache, *parts[:4], table, pos, slots)
    other, _ = _cache(pages)
    ops.quantize_kv_insert(other, parts[1], parts[2], parts[3], slots)
    assert torch.equal(cache.kv_pool, other.kv_pool) and torch.equal(cache.idx_pool, other.idx_pool)
    k, v, ik = ops.read_kv(cache, slots, dtype=torch.float32)
    # half the widest E2M1 step (4 to 6) under the group's scale, a scale off by half an E4M3 step
    for got, x in ((k, parts[1]), (v, parts[2])):
        a = x.view(n, 4, 8, 16).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).reshape(n, 4, 128)
        assert torch.all((got - x).abs() <= a * (1 / 6 + 2.0**-4) * 1.01)
    # E4M3 keys: half a step, 2^-10 below the smallest normal value
    assert torch.all((ik - parts[3]).abs() <= parts[3].abs() * 2.0**-4 + 2.0**-10)


def test_refusals():
    parts, slots, pos, pages, table = _inputs(4, torch.bfloat16, 1, False, 64)
    cache, _ = _cache(pages)
    with pytest.raises(ValueError):
        ops.rotary_insert(cache, *parts[:4], table, pos.cpu(), slots)
    with pytest.raises(TypeError):
        ops.rotary_insert(cache, *parts[:4], table, pos.long(), slots)
    with pytest.raises(TypeError):
        ops.rotary_insert(cache, parts[0].double(), *parts[1:4], table, pos, slots)
    with pytest.raises(ValueError):
        ops.rotary_insert(cache, *parts[:4], table, pos[:3], slots)
    with pytest.raises(ops.MsaError):
        ops.rotary_insert(cache, *parts[:4], table[:, :24].contiguous(), pos, slots)
    with pytest.raises(ValueError):
        ops.read_kv(cache, slots, k=torch.empty((3, 4, 128), device=DEV))
    with pytest.raises(TypeError):
        ops.read_kv(cache, slots, k=torch.empty((4, 4, 128), device=DEV), v=torch.empty((4, 4, 128), device=DEV).half())
    with pytest.raises(TypeError):
        ops.read_kv(cache, slots, dtype=torch.float64)
    with pytest.raises(ValueError):
        ops.KVCache.from_pools(cache.kv_pool, cache.idx_pool[:1], 1.0, 1.0)
    assert cache.read_status() == 0


def test_captured_and_replayed_on_another_stream():
    n = 64
    parts, slots, pos, pages, table = _inputs(n, torch.bfloat16, 9, True, 128)
    want_cache, _ = _cache(pages)
    want = ops.rotary_insert(want_cache, *parts[:4], table, pos, slots, q_idx=parts[4])
    want_k = ops.read_kv(want_cache, slots)[0]
    cache, _ = _cache(pages)
    q8, qi8 = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    k = torch.zeros_like(want_k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ops.rotary_insert(cache, *parts[:4], table, pos, slots, q_idx=parts[4], q8=q8, qi8=qi8)
        ops.read_kv(cache, slots, k=k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q8, want[0]) and torch.equal(qi8, want[1]) and torch.equal(k, want_k)
    assert torch.equal(cache.kv_pool, want_cache.kv_pool)
