"""GPU parity of the tree attention where the softmax's reference moves: long runs of pages with
rising scores, references that move with every chunk, scores beyond fp32's steps; and the bytes
that a tree's drafts leave in the cache.  Tolerances are those of test_gpu_tree.py and what the
notes below add.
"""

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import formats, nvfp4, rotary, tree
from test_gpu_tree import BF16, DEV, F16, S_ENC_K, S_ENC_V, SCALE, Batch, tree_words

pytestmark = pytest.mark.gpu


# ---- scores that rise along the context ----------------------------------------------------
#
# A row's reference moves when 32 weights sum to more than 49,152: one of them is then above
# 1,536 = 6 * 2^8, so that a move multiplies what the row has by less than 1/6.  On top of the
# bounds above: the weights of a page's earlier chunks are multiplied and rounded to f16 again
# with each move inside the page, three times at most (in all four roundings: 4 * 2^-11
# relative, or 4 * 2^-25 under the bias of 2^8); what a row had is off by 2^-22 (the
# exponential) and by the reference's own rounding, ten steps of 2^-24 of the scores' size, of
# which the factors below 1/6 leave a sum below twice the last; a move rounds the accumulator once.


def _exact_rows(b, s, words=None):
    """As tree.attend, for all drafts of a head at once."""
    ctx, n = b.seqs[s]
    k8, v8 = zip(*(tree.page_operands(b.pool[b.bt[s, i]]) for i in range(-(-(ctx + n) // 128))))
    k, v = (formats.decode_e4m3(np.concatenate(x))[: ctx + n] for x in (k8, v8))
    rows = slice(b.qsl[s], b.qsl[s + 1])
    q = formats.decode_e4m3(b.q8[rows])
    seen = np.ones((n, ctx + n), bool)
    seen[:, ctx:] = tree.visible(ctx, n, None if words is None else words[rows], range(ctx, ctx + n))
    fac = float(SCALE) / float(np.float32(S_ENC_K))
    out, mean, lse, size = np.zeros((n, 16, 128)), np.zeros((n, 16, 128)), np.zeros((n, 16)), np.zeros((n, 16))
    for h in range(16):
        z = np.where(seen, q[:, h] @ k[:, h // 4].T * fac, -np.inf)
        size[:, h] = np.where(seen, np.abs(q[:, h]) @ np.abs(k[:, h // 4]).T, 0).max(1) * fac
        top = z.max(1)
        p = np.exp(z - top[:, None])
        total = p.sum(1)
        lse[:, h] = top + np.log(total)
        vv = v[:, h // 4] / float(np.float32(S_ENC_V))
        out[:, h], mean[:, h] = (p / total[:, None]) @ vv, (p / total[:, None]) @ np.abs(vv)
    return out, lse, mean, size, seen.sum(1)


def _check_moving(b, out, lse, dtype, which, words=None):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    step = 2.0**-11 if dtype == F16 else 2.0**-8
    for s in which:
        o, l, mean, size, keys = _exact_rows(b, s, words)
        rows, keys = slice(b.qsl[s], b.qsl[s + 1]), keys[:, None]
        e = 140 * 2.0**-24 * size + 2.0**-20
        assert np.all(np.abs(lse[rows] - l) <= e + (keys + 200) * 2.0**-24 + 2.0**-23 * np.abs(l)), s
        tol = (4.01 * 2.0**-11 + 2 * e + 2 * (keys + 200) * 2.0**-24)[..., None] * mean + (keys * 2.0**-31)[..., None] * 448 / S_ENC_V
        tol = tol + step * (np.abs(o) + tol) + 2.0**-25
        off = np.abs(out[rows] - o)
        assert np.all(off <= tol), (s, int((off > tol).sum()), float(off.max()), float(np.abs(o).max()))


@pytest.mark.parametrize("drafts", [[1] * 16, [12] * 16, [24] * 16, [48] * 16, [1, 40, 3, 12, 24, 2, 9, 1] * 2],
                         ids=["1", "12", "24", "48", "mixed"])
def test_scores_that_rise_and_fall_over_long_runs_of_pages(drafts):
    """Some 20 pages of a (sequence, KV head) in a CTA, keys that grow 32-fold along the context:
    rows with rising scores move their reference every few pages and inside pages, among rows
    with falling ones."""
    rng = np.random.default_rng(50)
    b = Batch([(int(rng.integers(5900, 6100)), n) for n in drafts], 51)
    heads = b.pool.reshape(-1, 4, 18432)
    heads[:, :, :8192] &= 0x77  # K codes: every sign positive
    for s, (ctx, n) in enumerate(b.seqs):
        for i in range(-(-(ctx + n) // 128)):
            t = 128 * i + np.arange(128)
            grown = 0x28 + 40 * t // (ctx + n) + rng.integers(0, 3, (4, 8, 128))
            heads[b.bt[s, i], :, 8192:9216] = np.minimum(grown, 0x54).astype(np.uint8).reshape(4, 1024)
    way = rng.choice([40.0, 12.0, -40.0, 3.0], (b.T, 16, 1))
    b.q8 = formats.encode_e4m3(way * (1 + 0.3 * rng.standard_normal((b.T, 16, 128))))
    words = [w for _, n in b.seqs for w in tree_words(b.rng, n)]
    out, lse, cache = b.run(F16, words)
    _check_moving(b, out, lse, F16, range(16), words)
    assert cache.read_status() == 0


@pytest.mark.parametrize("drafts", [1, 12, 20, 64])
def test_the_reference_moves_with_every_chunk(drafts):
    """Keys of 1, 2, 3, ... in the chunks of 32 tokens: scores that rise by 1, 2.9 or 8.7 log2 units
    a chunk, or fall, so that the factors of the moves are from 2^-3 to 2^-9."""
    rng = np.random.default_rng(52)
    b = Batch([(500 + int(rng.integers(0, 60)), drafts) for _ in range(64)], 53)
    heads = b.pool.reshape(-1, 4, 18432)
    heads[:, :, :8192] = 0x22  # K codes: magnitude 2 -> 1.0, positive
    for s, (ctx, n) in enumerate(b.seqs):
        for i in range(-(-(ctx + n) // 128)):
            size = 1.0 + np.minimum((128 * i + np.arange(128)) // 32, 15)  # exact in E4M3
            heads[b.bt[s, i], :, 8192:9216] = np.tile(formats.encode_e4m3(size), (4, 8, 1)).reshape(4, 1024)
    b.q8 = formats.encode_e4m3(np.broadcast_to(rng.choice([5.5, 16.0, 48.0, -16.0], (b.T, 16, 1)), (b.T, 16, 128)))
    out, lse, cache = b.run(F16)
    _check_moving(b, out, lse, F16, range(0, 64, 5))
    assert cache.read_status() == 0


@pytest.mark.parametrize("scale", [1e6, 1e9, 1e25])
def test_log_sums_of_scores_far_beyond_fp32_steps(scale):
    """lse moves by no more than the scores do: 128 products and sums, the scale's three roundings, the
    reference's, its way back to natural logarithms: 140 steps of 2^-24 of the largest sum of |q k|."""
    seqs = [(3000, 1), (700, 9), (500, 40), (6000, 64)]
    b = Batch(seqs, 54)
    cache, q, bt, lens, qsl = b.device()
    bufs = ops.TreeBuffers(b.T, len(seqs), F16)
    ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=scale)
    torch.cuda.synchronize()
    got, up = bufs.lse.double().cpu().numpy(), scale / float(SCALE)
    qv = formats.decode_e4m3(b.q8)
    for s, (ctx, n) in enumerate(seqs):
        k8, _ = zip(*(tree.page_operands(b.pool[b.bt[s, i]]) for i in range(-(-(ctx + n) // 128))))
        k = formats.decode_e4m3(np.concatenate(k8))[: ctx + n]
        seen = np.tril(np.ones((n, ctx + n), bool), ctx)
        rows = slice(b.qsl[s], b.qsl[s + 1])
        fac = float(SCALE) / float(np.float32(S_ENC_K)) * up
        for h in range(16):
            z = np.where(seen, qv[rows, h] @ k[:, h // 4].T * fac, -np.inf)
            size = np.where(seen, np.abs(qv[rows, h]) @ np.abs(k[:, h // 4]).T, 0).max(1) * fac
            want = z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1))
            off = np.abs(got[rows, h] - want)
            assert np.all(off <= 140 * 2.0**-24 * size + (ctx + n) * 2.0**-24 + 2.0**-20 + 2.0**-23 * np.abs(want)), (s, h)
    assert cache.read_status() == 0


@pytest.mark.parametrize("inter,scaling", [(True, "yarn"), (False, "linear")])
def test_the_drafts_of_a_tree_are_turned_by_their_depth(inter, scaling):
    """Queries, keys and index keys of a tree's drafts as the cache holds them (in slot order, turned
    by their depth, part of the head): the bytes of rows that NumPy turned in the documented steps."""
    g = torch.Generator(device=DEV)
    g.manual_seed(55)
    seqs = [(3000, 7), (1111, 12)]
    b = Batch(seqs, 56)
    cache, _, bt, lens, qsl = b.device()
    rows = torch.randn((b.T, 33, 128), generator=g, device=DEV).to(BF16)
    words = [w for _, n in seqs for w in tree_words(b.rng, n)]
    depth = torch.tensor([bin(w).count("1") - 1 for w in words], dtype=torch.int32, device=DEV)
    assert len(set(depth.tolist())) < 12  # (several drafts of one depth)
    pos = torch.cat([torch.arange(c, c + n) for c, n in seqs]).to(DEV)
    seq = torch.tensor([s for s, (_, n) in enumerate(seqs) for _ in range(n)], device=DEV)
    at = torch.tensor([c for c, n in seqs for _ in range(n)], dtype=torch.int32, device=DEV) + depth
    slots = bt[seq, pos // 128].long() * 128 + pos % 128
    table = ops.rope_table_scaled(4096, 64, scaling=scaling, factor=4.0, original_max_pos=1024)
    q8, qi8 = ops.rotary_insert(cache, rows[:, :16], rows[:, 16:20], rows[:, 20:24], rows[:, 24], table, at, slots,
                                q_idx=rows[:, 25:33], interleaved=inter)
    k, v, ik = ops.read_kv(cache, slots, dtype=torch.float32)
    x, cs = rows.float().cpu().numpy(), table.cpu().numpy()[at.cpu().numpy()]
    want = {name: rotary.turn_fp32(x[:, part], cs, inter) for name, part in
            (("q", slice(0, 16)), ("k", slice(16, 20)), ("idx", slice(24, 25)), ("q_idx", slice(25, 33)))}
    for got, name in ((q8, "q"), (qi8, "q_idx")):
        np.testing.assert_array_equal(got.cpu().numpy(), formats.encode_e4m3(want[name].astype(np.float64)))
    for got, y, s_enc in ((k, want["k"], S_ENC_K), (v, x[:, 20:24], S_ENC_V)):
        codes, scales = nvfp4.quantize(y, np.float32(s_enc))
        d = (formats.decode_e4m3(scales).astype(np.float32) * (np.float32(1) / np.float32(s_enc))).astype(np.float32)
        value = formats.decode_e2m1(codes).astype(np.float32).reshape(b.T, 4, 8, 16) * d.reshape(b.T, 4, 8, 1)
        np.testing.assert_array_equal(got.cpu().numpy(), value.reshape(b.T, 4, 128))
    np.testing.assert_array_equal(ik.cpu().numpy(), formats.decode_e4m3(formats.encode_e4m3(want["idx"][:, 0].astype(np.float64))).astype(np.float32))
    assert cache.read_status() == 0


@pytest.mark.parametrize("drafts", [1, 12, 40])
def test_a_scale_whose_quotient_leaves_fp32_is_a_mean(drafts):
    """softmax_scale / s_enc_k below fp32's smallest number: every visible key has the same weight, on
    pages that end inside (whose other tokens are not seen) too."""
    b = Batch([(1000, drafts), (128, drafts), (3, drafts)], 57)
    cache, q, bt, lens, qsl = b.device()
    cache.s_enc_k = 1e8
    bufs = ops.TreeBuffers(b.T, 3, F16)
    ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=1e-38)
    torch.cuda.synchronize()
    got, lse = bufs.out.double().cpu().numpy(), bufs.lse.double().cpu().numpy()
    for s, (ctx, n) in enumerate(b.seqs):
        _, v8 = zip(*(tree.page_operands(b.pool[b.bt[s, i]]) for i in range(-(-(ctx + n) // 128))))
        v = formats.decode_e4m3(np.concatenate(v8)) / float(np.float32(S_ENC_V))
        for j in range(n):
            keys = ctx + j + 1
            m, size = v[:keys].mean(0), np.abs(v[:keys]).mean(0)
            tol = (2.0**-11 + 2 * keys * 2.0**-24) * size + 2.0**-11 * np.abs(m) + 2.0**-24
            assert np.all(np.abs(got[b.qsl[s] + j] - m.repeat(4, 0)) <= tol.repeat(4, 0)), (s, j)
            assert np.all(np.abs(lse[b.qsl[s] + j] - np.log(keys)) <= keys * 2.0**-24 + 2.0**-20), (s, j)
    assert cache.read_status() == 0


@pytest.mark.parametrize("drafts,pad_rows,empty", [(1, 126, 0), (64, 0, 14), (20, 0, 8)])
def test_padded_batches(drafts, pad_rows, empty):
    """Padding rows and empty sequences choose the other kernel than the drafts alone would."""
    b = Batch([(900, drafts), (2500, drafts)] + [(0, 0)] * empty, 58, pad_rows=pad_rows)
    assert (2 * drafts > 16 * 2) != (b.T > 16 * len(b.seqs))
    bufs = ops.TreeBuffers(b.T, len(b.seqs), F16)
    bufs.out.fill_(3.0)
    out, lse, cache = b.run(F16, bufs=bufs)
    b.check(out, lse)
    assert torch.all(out[2 * drafts:] == 3.0) and cache.read_status() == 0


def test_a_query_that_is_no_number_and_sees_nothing_is_zeros():
    b = Batch([(0, 3), (0, 20)], 59)
    b.q8[0, 5, 17] = b.q8[1, 5, 17] = b.q8[4, 0, 0] = 0x7F
    words = [0, 1, 0, 1, 0] + [3] * 18
    out, lse, cache = b.run(F16, words)
    for row in (0, 2, 4):
        assert not out[row].any() and torch.isneginf(lse[row]).all()
    bad = torch.zeros((b.T, 16), dtype=torch.bool, device=DEV)
    bad[1, 5] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(lse.isnan(), bad) and cache.read_status() == 0
