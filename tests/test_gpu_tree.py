"""GPU parity of the tree attention against the float64 oracle, through the binding.

Tolerances.  The operands are exact FP8 values.  A logit is an fp32 sum of 128
products and one fp32 multiply-add: off by at most 130 * 2^-24 of the sum of its
products' sizes (times the scale), as is lse, whose own sum of n terms adds
n 2^-24 (and the exponential 2^-21).  The weights are rounded to f16: 2^-11
relative, or half of f16's smallest step, 2^-25 under the bias of 2^8, for each of n
keys; the fp32 accumulator adds n 2^-24 of the summed sizes.  So an output
element is off by at most (2^-11 + 2 e + 2 n 2^-24) * sum p |v| + n 2^-33 max|v|
with e the logit's bound, and the rounding of the output type.
"""

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import formats, tree

pytestmark = pytest.mark.gpu

DEV = "cuda"
S_ENC_K, S_ENC_V = 448.0 / 5.0, 448.0 / 6.0
SCALE = np.float32(1.0 / np.sqrt(128.0))
BF16, F16 = torch.bfloat16, torch.float16


class Batch:
    """Sequences [(ctx, n_q)] over a random pool: finite scales where tokens are, bytes of
    every value (NaN scales too) behind the sequences and in pages that nobody owns."""

    def __init__(self, seqs, seed, q_scale=1.0, spread=1.0, pad_rows=0, extra_cols=1):
        rng = np.random.default_rng(seed)
        self.seqs = seqs
        pages = [-(-(c + n) // 128) for c, n in seqs]
        total = sum(pages) + 2
        pool = rng.integers(0, 256, (total, 4, 18432), dtype=np.uint8)
        perm = rng.permutation(total)
        bt = np.full((len(seqs), max(pages + [1]) + extra_cols), -7, np.int32)
        at = 0
        for b, n in enumerate(pages):
            bt[b, :n] = perm[at: at + n]
            at += n
            for i in range(n):
                live = min(128, sum(seqs[b]) - 128 * i)
                for lo in (8192, 17408):
                    s = pool[bt[b, i], :, lo: lo + 1024].reshape(4, 8, 128)
                    # E4M3 scales of 2 to 16, times 2^(0 .. 2 spread)
                    s[:, :, :live] = rng.integers(0x40, 0x58, (4, 8, live)) + 8 * rng.integers(0, max(1, int(2 * spread)), (4, 8, live))
                    pool[bt[b, i], :, lo: lo + 1024] = s.reshape(4, 1024)
        self.pool = pool.reshape(total, -1)
        self.bt = bt
        self.lens = np.array([c + n for c, n in seqs], np.int32)
        self.qsl = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        self.T = int(self.qsl[-1]) + pad_rows
        self.q8 = formats.encode_e4m3(rng.standard_normal((self.T, 16, 128)) * q_scale)
        self.rng = rng

    def device(self):
        cache = ops.KVCache(self.pool.shape[0], S_ENC_K, S_ENC_V, DEV)
        cache.kv_pool.copy_(torch.from_numpy(self.pool))
        put = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return cache, put(self.q8), put(self.bt), put(self.lens), put(self.qsl)

    def oracle(self, b, words=None, sel=None):
        ctx, n = self.seqs[b]
        k8, v8 = zip(*(tree.page_operands(self.pool[self.bt[b, i]]) for i in range(-(-(ctx + n) // 128))))
        k8, v8 = np.concatenate(k8)[: ctx + n], np.concatenate(v8)[: ctx + n]
        rows = slice(self.qsl[b], self.qsl[b + 1])
        # context positions are alike for every draft: build the mask from a few
        seen = np.ones((n, ctx + n), bool)
        seen[:, ctx:] = tree.visible(ctx, n, None if words is None else words[rows], range(ctx, ctx + n))
        if sel is not None:
            blk = np.arange(ctx + n) // 128
            seen[:, (blk < ctx // 128) & ~np.isin(blk, sel)] = False
        return tree.attend(self.q8[rows], k8, v8, seen, SCALE, S_ENC_K, S_ENC_V), seen

    def check(self, out, lse, words=None, sels=None, only=None):
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy()
        eps = 2.0**-11 if self.dtype == F16 else 2.0**-8
        for b, (ctx, n) in enumerate(self.seqs):
            if n == 0 or (only is not None and b not in only):
                continue
            (o, l, mean, size), seen = self.oracle(b, words, None if sels is None else sels[b])
            rows = slice(self.qsl[b], self.qsl[b + 1])
            keys = seen.sum(1)[:, None]
            e = 130 * 2.0**-24 * size
            fin = np.isfinite(l)
            np.testing.assert_array_equal(np.isneginf(lse[rows]), ~fin)
            assert np.all(np.abs(np.where(fin, lse[rows], 0) - np.where(fin, l, 0))[fin] <= (e + keys * 2.0**-24 + 2.0**-21 + 2.0**-23 * np.abs(np.where(fin, l, 0)))[fin])
            rel = (2.0**-11 + 2 * e + 2 * keys * 2.0**-24)[..., None]
            tol = rel * mean + (keys * 2.0**-33)[..., None] * 448 / S_ENC_V
            tol = tol + eps * (np.abs(o) + tol) + 2.0**-25
            bad = np.abs(out[rows] - o) > tol
            assert not bad.any(), (b, ctx, n, int(bad.sum()), float(np.abs(out[rows] - o).max()), float(np.abs(o).max()))

    def run(self, dtype=BF16, words=None, sels=None, cache_dev=None, bufs=None):
        self.dtype = dtype
        cache, q, bt, lens, qsl = cache_dev or self.device()
        bufs = bufs or ops.TreeBuffers(self.T, len(self.seqs), dtype)
        kw = {}
        if words is not None:
            kw["tree_mask"] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=DEV)
        if sels is not None:
            sel = np.full((len(sels), 17), -1, np.int32)
            for b, s in enumerate(sels):
                sel[b, : len(s)] = s
            kw["sel"] = torch.from_numpy(sel).to(DEV)
            kw["n_sel"] = torch.tensor([len(s) for s in sels], dtype=torch.int32, device=DEV)
        out = ops.tree_attn(cache, q, bt, lens, qsl, bufs, **kw)
        torch.cuda.synchronize()
        return out, bufs.lse, cache


def tree_words(rng, n):
    words = []
    for j in range(n):
        parent = int(rng.integers(max(0, j - 5), j)) if j else -1
        words.append((words[parent] if j else 0) | (1 << j))
    return words


CASES = {
    "one_token": [(0, 1)],
    "first_page": [(100, 1)],
    "edge_127": [(127, 1)],
    "edge_128": [(128, 1)],
    "edge_126_3": [(126, 3)],
    "no_context_64": [(0, 64)],
    "tile_32": [(500, 32)],
    "tiles_33": [(500, 33)],
    "straddle_64": [(1000, 64)],
    "long_one": [(9000, 1)],
    "long_20": [(7000, 20)],
    "mostly_wide": [(700, 33), (0, 5), (64, 64), (129, 1), (2000, 60), (1, 12)],
    "mostly_small": [(500, 20), (300, 1), (200, 2), (1300, 4), (90, 40), (260, 1), (5, 1)],
    "mixed": [(700, 33), (0, 5), (300, 0), (64, 64), (129, 1), (2500, 8), (1, 1), (383, 2)],
}


@pytest.mark.parametrize("name", CASES)
def test_chain(name):
    b = Batch(CASES[name], 1)
    out, lse, cache = b.run()
    b.check(out, lse)
    assert cache.read_status() == 0


@pytest.mark.parametrize("name", ["no_context_64", "tile_32", "tiles_33", "straddle_64", "mostly_wide", "mostly_small", "mixed", "edge_126_3"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_tree(name, dtype):
    b = Batch(CASES[name], 2)
    words = [w for _, n in b.seqs for w in tree_words(b.rng, n)]
    out, lse, cache = b.run(dtype, words)
    b.check(out, lse, words)
    assert cache.read_status() == 0


def test_arbitrary_masks_and_rows_that_see_nothing():
    b = Batch([(0, 64), (200, 40), (0, 3), (60, 64)], 3)
    words = [int(w) for w in b.rng.integers(0, 1 << 63, b.T, dtype=np.uint64) * 2 + 1]
    words[5] = words[64 + 7] = words[105] = 0   # no draft at all: the context alone, or nothing
    words[106] = 1 << 40                         # a draft that does not exist
    words[9] = (1 << 64) - 1
    out, lse, cache = b.run(F16, words)
    b.check(out, lse, words)
    assert torch.isneginf(lse[5]).all() and not out[5].any() and torch.isneginf(lse[105]).all() and torch.isneginf(lse[106]).all()
    assert cache.read_status() == 0


@pytest.mark.parametrize("nq", [1, 8, 40])
def test_shared_selection(nq):
    b = Batch([(5000, nq), (100, nq), (2047, nq), (2048, nq), (128 * 3, nq)], 4)
    sels = []
    for ctx, n in b.seqs:
        first = ctx // 128
        some = sorted(b.rng.choice(first, min(16, first), replace=False).tolist()) if first else []
        sels.append(some + [first])
    out, lse, cache = b.run(BF16, sels=sels)
    b.check(out, lse, sels=sels)
    # every block listed (and none): the whole context, and the drafts' blocks alone
    full = [list(range(min(17, c // 128 + 1))) for c, _ in b.seqs]
    out, lse, _ = b.run(F16, sels=full)
    b.check(out, lse, sels=full)
    none = [[] for _ in b.seqs]
    out, lse, _ = b.run(F16, sels=none)
    b.check(out, lse, sels=none)
    assert cache.read_status() == 0


def test_bad_selections_are_left_out():
    b = Batch([(1500, 2), (1500, 2), (1500, 2)], 5)
    sels = [[3, 3, 5, 4, 11], [-2, 1, 7], [2, 90]]
    out, lse, cache = b.run(BF16, sels=sels)
    b.check(out, lse, sels=[[3, 5], [1, 7], [2]])
    assert cache.read_status() == ops.STATUS_BAD_SELECTION


@pytest.mark.parametrize("q_scale", [12.0, 60.0])
def test_peaked_and_wide_logits(q_scale):
    """Logits over tens of log2 units: the reference moves, small weights leave."""
    b = Batch([(3000, 9), (900, 64)], 6, q_scale=q_scale, spread=2.0)
    out, lse, cache = b.run(F16)
    b.check(out, lse)
    assert cache.read_status() == 0


def test_one_dominant_key_over_a_long_bulk():
    """A key 14 nats above thousands of equal ones: the bulk still has its share."""
    b = Batch([(12000, 1)], 7)
    ops_k = 0x48  # scale byte 4
    heads = b.pool.reshape(-1, 4, 18432)
    heads[:, :, :8192] = 0x11            # K codes: magnitude 1 -> 0.5 everywhere, positive
    heads[:, :, 8192:9216] = 0x08        # tiny scales: equal keys near zero
    top = b.bt[0, 20]
    for g in range(4):
        heads[top, g, 8192:9216].reshape(8, 128)[:, 77] = ops_k
    q = np.zeros((1, 16, 128))
    q[:] = 14.0 / (0.5 * 4 * 128) / (float(SCALE) / S_ENC_K)
    b.q8 = formats.encode_e4m3(q)
    out, lse, cache = b.run(F16)
    b.check(out, lse)


def test_rows_behind_the_last_sequence_and_skipped_sequences_stay():
    b = Batch([(300, 4), (50, 70), (260, 2), (10, 0), (40, 6)], 8, pad_rows=5)
    b.lens[4] = 5            # fewer cached tokens than query tokens
    b.dtype = BF16
    bufs = ops.TreeBuffers(b.T, 5, BF16)
    bufs.out.fill_(3.0)
    bufs.lse.fill_(4.0)
    out, lse, cache = b.run(BF16, bufs=bufs)
    assert cache.read_status() == ops.STATUS_BAD_SEQ
    b.check(out, lse, only=[0, 2])
    for lo, hi in ((4, 74), (76, b.T)):
        assert torch.all(out[lo:hi] == 3.0) and torch.all(lse[lo:hi] == 4.0)


def test_pages_outside_the_pool_are_not_seen():
    b = Batch([(700, 3), (500, 1)], 9)
    dev = list(b.device())
    bad = b.bt.copy()
    bad[0, 2], bad[1, 0] = b.pool.shape[0], -1
    dev[2] = torch.from_numpy(bad).to(DEV)
    out, lse, cache = b.run(F16, cache_dev=dev)
    assert cache.read_status() == ops.STATUS_BAD_PAGE
    b.dtype = F16
    b.check(out, lse, sels=[[0, 1, 3, 4], [1, 2]])


def test_many_sequences():
    """4,096 sequences of 1 to 300 tokens: several sequences per CTA, most cuts inside a sequence's pages."""
    rng = np.random.default_rng(10)
    seqs = [(int(rng.integers(0, 300)), int(rng.integers(0, 3))) for _ in range(4096)]
    b = Batch(seqs, 11)
    out, lse, cache = b.run(BF16)
    b.check(out, lse, only=set(rng.choice(4096, 300).tolist()) | {0, 1, 4094, 4095})
    assert cache.read_status() == 0


def test_one_page_sequences_over_and_over():
    """Segments of one page, in which one of the softmax sets has nothing to do, among wide ones."""
    rng = np.random.default_rng(30)
    seqs = [(int(rng.integers(0, 90)), int(rng.integers(1, 64)) if i % 9 == 4 else int(rng.integers(1, 3))) for i in range(900)]
    b = Batch(seqs, 31)
    dev = b.device()
    bufs = ops.TreeBuffers(b.T, len(seqs), F16)
    out, lse, cache = b.run(F16, cache_dev=dev, bufs=bufs)
    b.check(out, lse, only=set(range(0, 900, 7)) | set(range(4, 900, 45)))
    first = out.clone(), lse.clone()
    for _ in range(30):
        out, lse, _ = b.run(F16, cache_dev=dev, bufs=bufs)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert cache.read_status() == 0


def test_captured_graph_follows_lengths_and_selections():
    """A captured call replayed on longer sequences and other blocks than it was captured with."""
    b = Batch([(3000, 4), (2000, 4)], 32)
    cache, q, bt, lens, qsl = b.device()
    sel = torch.full((2, 17), -1, dtype=torch.int32, device=DEV)
    n_sel = torch.zeros(2, dtype=torch.int32, device=DEV)
    short = torch.tensor([4, 4], dtype=torch.int32, device=DEV)
    bufs = ops.TreeBuffers(b.T, 2, F16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.tree_attn(cache, q, bt, short, qsl, bufs, sel=sel, n_sel=n_sel)
    graph.replay()
    short.copy_(lens)
    sels = [[0, 3, 9, 22], [1, 2, 14]]
    for i, s in enumerate(sels):
        sel[i, : len(s)] = torch.tensor(s, dtype=torch.int32)
        n_sel[i] = len(s)
    graph.replay()
    torch.cuda.synchronize()
    b.dtype = F16
    b.check(bufs.out, bufs.lse, sels=sels)
    assert cache.read_status() == 0


def test_pages_whose_offsets_pass_32_bits():
    """The last pages of pools of 19.9 and 4.4 GB, written, attended and read as in a small pool."""
    b = Batch([(900, 5), (260, 1)], 33)
    small, q, bt, lens, qsl = b.device()
    n, far = small.n_pages, 270_000
    kv = torch.empty((far, ops.KV_PAGE_BYTES), dtype=torch.uint8, device=DEV)
    ix = torch.empty((far, ops.IDX_PAGE_BYTES), dtype=torch.uint8, device=DEV)
    kv[far - n:] = small.kv_pool
    ix[far - n:] = small.idx_pool
    big = ops.KVCache.from_pools(kv, ix, S_ENC_K, S_ENC_V)
    g = torch.Generator(device=DEV)
    g.manual_seed(34)
    rows = torch.randn((6, 33, 128), generator=g, device=DEV).to(F16)
    pos = torch.tensor([900, 901, 902, 903, 904, 260], dtype=torch.int32, device=DEV)
    seq = torch.tensor([0, 0, 0, 0, 0, 1], device=DEV)
    slots = bt[seq, pos.long() // 128].long() * 128 + pos % 128
    table = ops.rope_table_scaled(1024, 128)
    got = []
    for cache, up in ((small, 0), (big, far - n)):
        q8, _ = ops.rotary_insert(cache, rows[:, :16], rows[:, 16:20], rows[:, 20:24], rows[:, 24], table, pos,
                                  slots + 128 * up)
        bufs = ops.TreeBuffers(6, 2, F16)
        pages = torch.where(bt >= 0, bt + up, bt)
        got.append([q8, ops.tree_attn(cache, q8, pages, lens, qsl, bufs), bufs.lse, *ops.read_kv(cache, slots + 128 * up)])
        assert cache.read_status() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.equal(big.kv_pool[far - n:], small.kv_pool) and torch.equal(big.idx_pool[far - n:], small.idx_pool)
    b.q8, b.pool, b.dtype = got[1][0].cpu().numpy(), small.kv_pool.cpu().numpy(), F16
    b.check(got[1][1], got[1][2])


def test_repeats_are_bit_equal_and_workspaces_come_to_rest():
    b = Batch([(4000, 40), (6000, 3)], 12)
    dev = b.device()
    bufs = ops.TreeBuffers(b.T, 2, BF16)
    first = [x.clone() for x in b.run(cache_dev=dev, bufs=bufs)[:2]]
    for _ in range(3):
        out, lse, _ = b.run(cache_dev=dev, bufs=bufs)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert torch.count_nonzero(bufs.ws[: b.T * 16]) == 0


def test_captured_graph_with_new_inputs():
    b = Batch([(1000, 8), (300, 64)], 13)
    cache, q, bt, lens, qsl = b.device()
    bufs = ops.TreeBuffers(b.T, 2, BF16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs)
    b.q8 = b.q8[::-1].copy()
    q.copy_(torch.from_numpy(b.q8))
    graph.replay()
    torch.cuda.synchronize()
    b.dtype = BF16
    b.check(bufs.out, bufs.lse)


def test_a_chain_agrees_with_the_sparse_decode_where_it_selects_everything():
    b = Batch([(1800, 8), (700, 2)], 14)
    cache, q, bt, lens, qsl = b.device()
    out, lse, _ = b.run(F16, cache_dev=(cache, q, bt, lens, qsl))
    sel = torch.full((b.T, 17), -1, dtype=torch.int32, device=DEV)
    n_sel = torch.zeros(b.T, dtype=torch.int32, device=DEV)
    for s, (ctx, n) in enumerate(b.seqs):
        for j in range(n):
            r = (ctx + j) // 128
            sel[b.qsl[s] + j, : r + 1] = torch.arange(r + 1)
            n_sel[b.qsl[s] + j] = r + 1
    o, l = ops.sparse_attn_decode(cache, q, sel, n_sel, bt, lens, qsl, 1)
    # the sparse path's bound of 2e-3 max|v| and this one's, far below it
    assert (out.float() - o[:, 0]).abs().max() <= 2.1e-3 * 448 / S_ENC_V
    assert (lse - l[:, 0]).abs().max() <= 1e-3


def test_drafts_written_selected_attended_and_read_back():
    """The whole round of a drafted tree: write its keys, select blocks with the root's index
    query, attend, read the accepted drafts' values."""
    g = torch.Generator(device=DEV)
    g.manual_seed(15)
    seqs = [(3000, 7), (1111, 7)]
    b = Batch(seqs, 16)
    cache, _, bt, lens, qsl = b.device()
    cache.idx_pool.copy_(torch.randn(cache.idx_pool.shape, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8))
    rows = torch.randn((14, 33, 128), generator=g, device=DEV).to(BF16)
    words = [w for _ in seqs for w in tree_words(b.rng, 7)]
    depth = torch.tensor([bin(w).count("1") - 1 for w in words], dtype=torch.int32, device=DEV)
    ctx = torch.tensor([c for c, n in seqs for _ in range(n)], dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(c, c + n) for c, n in seqs]).to(DEV)
    seq = torch.tensor([s for s, (_, n) in enumerate(seqs) for _ in range(n)], device=DEV)
    slots = bt[seq, pos // 128].long() * 128 + pos % 128
    q8, qi8 = ops.rotary_insert(cache, rows[:, :16], rows[:, 16:20], rows[:, 20:24], rows[:, 24],
                                ops.rope_table_scaled(4096, 64, scaling="yarn", factor=4.0, original_max_pos=1024),
                                ctx + depth, slots, q_idx=rows[:, 25:33], interleaved=True)
    b.pool = cache.kv_pool.cpu().numpy()
    b.q8 = q8.cpu().numpy()
    roots = torch.tensor([0, 7], device=DEV)
    w = torch.rand((2, 8), generator=g, device=DEV)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    sel, n_sel, _ = ops.indexer_topk(cache, qi8[roots].contiguous(), w, bt, lens - 6, one)
    bufs = ops.TreeBuffers(14, 2, BF16)
    out = ops.tree_attn(cache, q8, bt, lens, qsl, bufs, tree_mask=torch.tensor(words, device=DEV), sel=sel, n_sel=n_sel)
    k, v, _ = ops.read_kv(cache, slots)
    torch.cuda.synchronize()
    sels = [sel[s, : int(n_sel[s])].tolist() for s in range(2)]
    assert all(len(s) >= 9 for s in sels)
    b.dtype = BF16
    b.check(out, bufs.lse, words, sels)
    # half the widest E2M1 step under the group's scale, which is itself half an E4M3 step off; then bf16
    for got, x in ((v, rows[:, 20:24].float()),):
        a = x.reshape(14, 4, 8, 16).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).reshape(14, 4, 128)
        live = (a * S_ENC_V / 6 < 448)
        assert torch.all(((got.float() - x).abs() <= a * (1 / 6 + 2.0**-4) * 1.02)[live])
    assert cache.read_status() == 0


@pytest.mark.parametrize("scale", [1e6, 1e9, 1e25])
def test_scores_far_beyond_fp32_steps(scale):
    """Scores whose rounding alone exceeds f16's range of weights: the largest key takes all."""
    seqs = [(3000, 1), (700, 9), (500, 40)]
    b = Batch(seqs, 18)
    cache, q, bt, lens, qsl = b.device()
    bufs = ops.TreeBuffers(b.T, len(seqs), F16)
    ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=scale)
    torch.cuda.synchronize()
    out, sure = bufs.out.double().cpu().numpy(), 0
    qv = formats.decode_e4m3(b.q8)
    for s, (ctx, n) in enumerate(seqs):
        k8, v8 = zip(*(tree.page_operands(b.pool[b.bt[s, i]]) for i in range(-(-(ctx + n) // 128))))
        k, v = (formats.decode_e4m3(np.concatenate(x)) for x in (k8, v8))
        for j in range(n):
            for h in range(16):
                row, keys = qv[b.qsl[s] + j, h], k[: ctx + j + 1, h // 4]
                z = keys @ row
                first, second = np.sort(z)[[-1, -2]]
                # the scores' own rounding, and then the gap has to leave the second nothing (2^-30)
                if (first - second - 260 * 2.0**-24 * (np.abs(keys) @ np.abs(row)).max()) * scale / S_ENC_K < 21:
                    continue
                sure += 1
                want = v[np.argmax(z), h // 4] / float(np.float32(S_ENC_V))
                got = out[b.qsl[s] + j, h]
                # the weight 2^8 is exact; its sum and the scale 256 / s_enc round once each, then the type
                assert np.all(np.abs(got - want) <= np.abs(want) * (2.0**-11 + 2.0**-21) + 2.0**-24), (s, j, h)
    assert sure > 100 and torch.isfinite(bufs.lse).all() and cache.read_status() == 0


def test_scores_near_zero_are_a_mean():
    b = Batch([(1000, 3)], 19)
    cache, q, bt, lens, qsl = b.device()
    bufs = ops.TreeBuffers(3, 1, F16)
    ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=1e-30)
    torch.cuda.synchronize()
    _, v8 = zip(*(tree.page_operands(b.pool[b.bt[0, i]]) for i in range(8)))
    v = formats.decode_e4m3(np.concatenate(v8)) / float(np.float32(S_ENC_V))
    for j in range(3):
        m, size = v[: 1001 + j].mean(0), np.abs(v[: 1001 + j]).mean(0)
        tol = (2.0**-11 + 2004 * 2.0**-24) * size + 2.0**-11 * np.abs(m) + 2.0**-24
        assert np.all(np.abs(bufs.out[j].double().cpu().numpy() - m.repeat(4, 0)) <= tol.repeat(4, 0))


def test_a_query_that_is_no_number_stays_so():
    b = Batch([(2500, 3), (90, 2), (400, 40)], 20)
    b.q8[1, 5, 17] = 0x7F
    b.q8[4, 0, 0] = 0xFF
    b.q8[20, 15, 127] = 0x7F
    dev = b.device()
    out, lse, cache = b.run(F16, cache_dev=dev)
    bad = torch.zeros((b.T, 16), dtype=torch.bool, device=DEV)
    bad[1, 5] = bad[4, 0] = bad[20, 15] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad) and cache.read_status() == 0


def test_calls_of_different_sizes_share_a_workspace():
    small, large = Batch([(5000, 2)], 21), Batch([(4000, 40), (3000, 30)], 22)
    bufs = [ops.TreeBuffers(x.T, len(x.seqs), F16) for x in (small, large)]
    bufs[0].ws = bufs[1].ws
    for x, y in ((small, bufs[0]), (large, bufs[1]), (small, bufs[0]), (large, bufs[1])):
        out, lse, _ = x.run(F16, bufs=y)
        x.check(out, lse)


def test_two_captured_graphs_share_a_workspace():
    small, large = Batch([(5000, 2), (30, 1)], 36), Batch([(4000, 40), (3000, 30)], 37)
    bufs = [ops.TreeBuffers(x.T, len(x.seqs), F16) for x in (small, large)]
    bufs[0].ws = bufs[1].ws
    devs, graphs = [x.device() for x in (small, large)], []
    torch.cuda.synchronize()
    for d, u in zip(devs, bufs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ops.tree_attn(*d, u)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for x, d, u in zip((small, large), devs, bufs):
        x.dtype = F16
        x.check(u.out, u.lse)
        assert d[0].read_status() == 0


def test_another_stream_than_the_tensors_own():
    b = Batch([(2000, 4), (100, 60)], 23)
    dev = b.device()
    bufs = ops.TreeBuffers(b.T, 2, F16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.tree_attn(*dev, bufs)
    torch.cuda.current_stream().wait_stream(side)
    b.dtype = F16
    b.check(bufs.out, bufs.lse)


def test_two_calls_at_once_with_a_workspace_each():
    """Both kernels want every SM: their CTAs take turns, and neither waits for the other's."""
    batches = [Batch([(9000, 20), (50, 3)], 24), Batch([(7000, 1), (300, 64), (2000, 10)], 25)]
    devs = [b.device() for b in batches]
    bufs = [ops.TreeBuffers(b.T, len(b.seqs), F16) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(4):
        for d, u, s in zip(devs, bufs, streams):
            with torch.cuda.stream(s):
                ops.tree_attn(*d, u)
    torch.cuda.synchronize()
    for b, d, u in zip(batches, devs, bufs):
        b.dtype = F16
        b.check(u.out, u.lse)
        assert d[0].read_status() == 0


def test_a_wait_that_runs_out_is_reported_and_the_next_call_recovers():
    """Every CTA leaves out the copy of its first page: its waits end after their limit, the CTA
    waits for what it has in flight and returns; the workspace is at rest again."""
    b = Batch([(4000, 3), (900, 40), (20, 1)], 35)
    dev = b.device()
    bufs = ops.TreeBuffers(b.T, 3, F16)
    want = [x.clone() for x in b.run(F16, cache_dev=dev, bufs=bufs)[:2]]
    try:
        ops.set_fault_injection(ops.INJECT_ATTENTION_TIMEOUT, 5_000_000)
        b.run(F16, cache_dev=dev, bufs=bufs)
        assert dev[0].read_status() == ops.STATUS_TIMEOUT
    finally:
        ops.set_fault_injection(0, 0)
    dev[0].status.zero_()
    assert torch.count_nonzero(bufs.ws[: b.T * 16]) == 0
    for _ in range(2):
        out, lse, cache = b.run(F16, cache_dev=dev, bufs=bufs)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and cache.read_status() == 0


def test_refusals():
    b = Batch([(300, 2)], 17)
    cache, q, bt, lens, qsl = b.device()
    bufs = ops.TreeBuffers(2, 1)
    with pytest.raises(ValueError):
        ops.tree_attn(cache, q.cpu(), bt, lens, qsl, bufs)
    with pytest.raises(TypeError):
        ops.tree_attn(cache, q, bt.long(), lens, qsl, bufs)
    with pytest.raises(TypeError):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs, tree_mask=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ops.tree_attn(cache, q, bt, lens, qsl, ops.TreeBuffers(3, 1))
    with pytest.raises(ops.MsaError):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=-1.0)
    with pytest.raises(ops.MsaError):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs, softmax_scale=3e38)
    i32 = torch.int32
    for at, bad in ((1, q[:1]), (1, q[:, :8]), (3, lens.repeat(2)), (4, qsl[:1]), (2, bt.t())):
        args = [cache, q, bt, lens, qsl, bufs]
        args[at] = bad
        with pytest.raises(ValueError):
            ops.tree_attn(*args)
    with pytest.raises(ValueError):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs, tree_mask=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ops.tree_attn(cache, q, bt, lens, qsl, bufs, sel=torch.zeros((1, 16), dtype=i32, device=DEV),
                      n_sel=torch.zeros(1, dtype=i32, device=DEV))
    assert cache.read_status() == 0
