"""GPU parity of the prompt attention against the float64 oracle, through the binding.

Tolerances are those of test_gpu_tree.py, with an exponential that is off by 2^-22 and, where a
row's reference moves (by a factor below 2^-7.5, so that what earlier moves left sums to less
than twice the last one's), by the reference's own rounding, ten steps of 2^-24 of the scores'
size: a logit is off by e = 140 * 2^-24 of the sum of its products' sizes and 2^-20; the weights
are rounded to f16, 2^-11 relative or 2^-25 under the bias of 2^8, and those of a page's first 64
tokens once more when the reference moves for its others (together below 2.001 * 2^-11, or two
steps of 2^-25); a sum of n terms in fp32 adds n 2^-24, a move a rounding of the accumulator
(there are fewer than 200).
"""

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import formats, tree
from test_gpu_tree import BF16, DEV, F16, S_ENC_K, S_ENC_V, SCALE, Batch

pytestmark = pytest.mark.gpu


def _put(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device=DEV)


class Prompts(Batch):
    def pages(self):
        return sum(-(-(c + n) // 128) for c, n in self.seqs)

    def buffers(self, dtype, n_pages=None):
        bufs = ops.PrefillBuffers(self.T, len(self.seqs), self.pages() if n_pages is None else n_pages, dtype)
        bufs.ws.fill_(0xFF)  # nothing of it may be taken for something
        return bufs

    def go(self, dtype=BF16, window=0, ends=None, dev=None, bufs=None, **kw):
        cache, q, bt, lens, qsl = dev or self.device()
        bufs = bufs or self.buffers(dtype)
        ops.prefill_attn(cache, q, bt, lens, qsl, bufs, window=window, ends=None if ends is None else _put(ends), **kw)
        torch.cuda.synchronize()
        return bufs.out, bufs.lse, cache

    def seen(self, s, window, ends, hidden_pages=()):
        ctx, n = self.seqs[s]
        pos = ctx + np.arange(n)
        t = np.arange(ctx + n)
        end = pos + 1 if ends is None else np.clip(ends[self.qsl[s]: self.qsl[s + 1]], 0, ctx + n)
        out = t[None] < end[:, None]
        if window:
            out &= t[None] > pos[:, None] - window
        return out & ~np.isin(t // 128, list(hidden_pages))[None]

    def exact(self, s, seen, scale=SCALE):
        """tree.attend for all rows of a head at once."""
        ctx, n = self.seqs[s]
        k8, v8 = zip(*(tree.page_operands(self.pool[self.bt[s, i] % self.pool.shape[0]]) for i in range(-(-(ctx + n) // 128))))
        k, v = (formats.decode_e4m3(np.concatenate(x))[: ctx + n] for x in (k8, v8))
        q = formats.decode_e4m3(self.q8[self.qsl[s]: self.qsl[s + 1]])
        fac = float(scale) / float(np.float32(S_ENC_K))
        out, mean, lse, size = np.zeros((n, 16, 128)), np.zeros((n, 16, 128)), np.full((n, 16), -np.inf), np.zeros((n, 16))
        some = seen.any(1)
        for h in range(16):
            z = np.where(seen, q[:, h] @ k[:, h // 4].T * fac, -np.inf)[some]
            size[some, h] = np.where(seen, np.abs(q[:, h]) @ np.abs(k[:, h // 4]).T, 0).max(1)[some] * fac
            top = z.max(1, initial=-np.inf)
            p = np.exp(z - top[:, None])
            total = p.sum(1)
            lse[some, h] = top + np.log(total)
            vv = v[:, h // 4] / float(np.float32(S_ENC_V))
            out[some, h], mean[some, h] = (p / total[:, None]) @ vv, (p / total[:, None]) @ np.abs(vv)
        return out, lse, mean, size

    def same(self, out, lse, dtype, window=0, ends=None, only=None, hidden=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        step = 2.0**-11 if dtype == F16 else 2.0**-8
        for s, (ctx, n) in enumerate(self.seqs):
            if n == 0 or (only is not None and s not in only):
                continue
            seen = self.seen(s, window, ends, (hidden or {}).get(s, ()))
            o, l, mean, size = self.exact(s, seen)
            rows, keys, fin = slice(self.qsl[s], self.qsl[s + 1]), seen.sum(1)[:, None], np.isfinite(l)
            e = 140 * 2.0**-24 * size + 2.0**-20
            np.testing.assert_array_equal(np.isneginf(lse[rows]), ~fin)
            l0, g0 = np.where(fin, l, 0), np.where(fin, lse[rows], 0)
            assert np.all(np.abs(g0 - l0) <= e + (keys + 200) * 2.0**-24 + 2.0**-23 * np.abs(l0)), (s, ctx, n)
            tol = (2.001 * 2.0**-11 + 2 * e + 2 * (keys + 200) * 2.0**-24)[..., None] * mean + (keys * 2.0**-32)[..., None] * 448 / S_ENC_V
            tol = tol + step * (np.abs(o) + tol) + 2.0**-25
            off = np.abs(out[rows] - o)
            assert np.all(off <= tol), (s, ctx, n, int((off > tol).sum()), float(off.max()), float(np.abs(o).max()))


CASES = {
    "one_token": [(0, 1)],
    "one_behind_100": [(100, 1)],
    "edge_127": [(127, 1)],
    "edge_128": [(128, 1)],
    "first_32": [(0, 32)],
    "first_33": [(0, 33)],
    "first_64": [(0, 64)],
    "first_65": [(0, 65)],
    "page_and_more": [(0, 129)],
    "whole_300": [(0, 300)],
    "from_63": [(63, 65)],
    "from_128": [(128, 128)],
    "straddles": [(700, 200)],
    "one_long": [(9000, 1)],
    "few_long": [(12000, 40)],
    "chunk": [(2000, 150)],
    "mixed": [(700, 133), (0, 5), (300, 0), (64, 64), (129, 1), (1500, 70), (1, 1), (383, 33)],
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_causal(name, dtype):
    b = Prompts(CASES[name], 1)
    out, lse, cache = b.go(dtype)
    b.same(out, lse, dtype)
    assert cache.read_status() == 0


@pytest.mark.parametrize("window", [1, 2, 63, 64, 127, 128, 129, 300, 1000, 1 << 30])
def test_window(window):
    b = Prompts([(700, 133), (0, 200), (130, 1), (1000, 40), (5, 0)], 2)
    out, lse, cache = b.go(F16, window)
    b.same(out, lse, F16, window)
    assert cache.read_status() == 0


def test_a_window_needs_room_for_its_pages_only():
    b = Prompts([(3000, 100)], 3)
    # tokens 3,000 .. 3,099 see 200 positions: from 2,801 to 3,099, pages 21 .. 24
    out, lse, cache = b.go(F16, 200, bufs=b.buffers(F16, 4))
    b.same(out, lse, F16, 200)
    assert cache.read_status() == 0
    bufs = b.buffers(F16, 3)
    bufs.out.fill_(3.0)
    out, lse, cache = b.go(F16, 200, bufs=bufs)
    assert cache.read_status() == ops.STATUS_BAD_SEQ and torch.all(out == 3.0)


@pytest.mark.parametrize("window", [0, 90])
def test_ends_of_each_token(window):
    """Ends at random: nothing, everything, negative, behind the sequence, before the window."""
    b = Prompts([(300, 150), (0, 70), (1000, 33), (129, 1), (40, 64)], 4)
    rng = np.random.default_rng(5)
    ends = np.concatenate([rng.integers(-5, c + n + 20, n) for c, n in b.seqs])
    ends[3:9], ends[20], ends[150:220] = 0, 1 << 30, 70  # (rows 150 ..: the second prompt sees all of itself)
    out, lse, cache = b.go(F16, window, ends)
    b.same(out, lse, F16, window, ends)
    assert torch.isneginf(lse[3:9]).all() and not out[3:9].any()
    assert cache.read_status() == 0
    # tiles in which no token sees anything
    none = np.zeros(b.T, np.int64)
    out, lse, cache = b.go(BF16, window, none)
    assert torch.isneginf(lse).all() and not out.any() and cache.read_status() == 0


@pytest.mark.parametrize("q_scale,spread", [(12.0, 2.0), (60.0, 2.0), (3.0, 3.0)])
def test_peaked_and_wide_scores(q_scale, spread):
    b = Prompts([(2500, 90), (0, 300)], 6, q_scale=q_scale, spread=spread)
    out, lse, cache = b.go(F16)
    b.same(out, lse, F16)
    assert cache.read_status() == 0


def test_scores_that_rise_and_fall_over_long_runs_of_pages():
    """Keys that grow 32-fold along the context: rows with rising scores move their reference
    every few pages, among rows with falling ones."""
    rng = np.random.default_rng(50)
    b = Prompts([(5990, 64), (6010, 40), (5900, 130)], 51)
    heads = b.pool.reshape(-1, 4, 18432)
    heads[:, :, :8192] &= 0x77  # K codes: every sign positive
    for s, (ctx, n) in enumerate(b.seqs):
        for i in range(-(-(ctx + n) // 128)):
            t = 128 * i + np.arange(128)
            grown = 0x28 + 40 * t // (ctx + n) + rng.integers(0, 3, (4, 8, 128))
            heads[b.bt[s, i], :, 8192:9216] = np.minimum(grown, 0x54).astype(np.uint8).reshape(4, 1024)
    way = rng.choice([40.0, 12.0, -40.0, 3.0], (b.T, 16, 1))
    b.q8 = formats.encode_e4m3(way * (1 + 0.3 * rng.standard_normal((b.T, 16, 128))))
    out, lse, cache = b.go(F16)
    b.same(out, lse, F16)
    assert cache.read_status() == 0


def test_many_prompts():
    """4,096 sequences: more than one a thread, tiles of a few tokens, most of one page."""
    rng = np.random.default_rng(10)
    b = Prompts([(int(rng.integers(0, 300)), int(rng.choice([0, 1, 2, 40]))) for _ in range(4096)], 11)
    out, lse, cache = b.go(BF16)
    b.same(out, lse, BF16, only=set(rng.choice(4096, 200).tolist()) | {0, 1, 4094, 4095})
    assert cache.read_status() == 0


BATCHES = {  # jobs of 64 tokens x a KV head: fewer or more than SMs, alike or one far longer than the others
    "short_alike": [(90, 64)] * 70,
    "one_to_each": [(500, 60)] * 30,
    "some_twice": [(1000, 64)] * 40,
    "cut_behind_whole_ones": [(1500, 64)] * 45,
    "one_far_longer": [(50, 64)] * 45 + [(9000, 64)],
    "a_few_long": [(6000, 50), (3000, 64)],
}


@pytest.mark.parametrize("name", BATCHES)
def test_batches_that_share_out_differently(name):
    b = Prompts(BATCHES[name], 50)
    out, lse, cache = b.go(BF16)
    n = len(b.seqs)
    b.same(out, lse, BF16, only={0, 1, n // 2, n - 1})
    assert cache.read_status() == 0 and torch.isfinite(out).all()


@pytest.mark.parametrize("ctx,n,window", [(0, 5000, 0), (20000, 1500, 0), (9000, 2000, 3000)])
def test_large_prompts_by_samples_of_rows(ctx, n, window):
    b = Prompts([(ctx, n)], 12)
    out, lse, cache = b.go(F16, window)
    assert cache.read_status() == 0
    for lo in (0, n // 2 - 7, n - 20):  # prompts that end there, over the same cache
        part = Prompts.__new__(Prompts)
        part.seqs, part.pool, part.bt = [(ctx + lo, 20)], b.pool, b.bt
        part.qsl, part.q8 = np.array([0, 20]), b.q8[lo: lo + 20]
        part.same(out[lo: lo + 20], lse[lo: lo + 20], F16, window)


def test_sequences_behind_the_workspaces_pages_keep_their_rows_in_a_long_queue():
    b = Prompts([(90, 64)] * 70, 51)  # two pages each: the last five do not fit
    bufs = b.buffers(BF16, 130)
    bufs.out.fill_(3.0)
    bufs.lse.fill_(5.0)
    out, lse, cache = b.go(BF16, bufs=bufs)
    assert cache.read_status() == ops.STATUS_BAD_SEQ
    b.same(out, lse, BF16, only={0, 1, 33, 63, 64})
    assert (out[65 * 64:] == 3.0).all() and (lse[65 * 64:] == 5.0).all()


def test_parts_of_a_prompt_agree_with_the_whole():
    """A chunk's rows do not depend on what else the call holds, but for the order of their sums."""
    b = Prompts([(0, 1000)], 13)
    dev = b.device()
    whole, lse, _ = b.go(F16, dev=dev)
    for lo, n in ((0, 100), (100, 333), (433, 567)):
        part = Prompts([(lo, n)], 13)
        part.q8, part.pool, part.bt = b.q8[lo: lo + n], b.pool, b.bt
        got, l, _ = part.go(F16)
        # both are within the bound of the same values: f16 weights and an f16 output each
        scale = np.abs(whole[lo: lo + n].float().cpu().numpy()).max()
        assert (got.float() - whole[lo: lo + n].float()).abs().max() <= 4 * 2.0**-11 * max(scale, 448 / S_ENC_V)
        assert (l - lse[lo: lo + n]).abs().max() <= 1e-4


def test_a_chain_of_drafts_agrees_with_the_tree_attention():
    b = Prompts([(3000, 40), (700, 64), (100, 3)], 14)
    dev = b.device()
    out, lse, _ = b.go(F16, dev=dev)
    bufs = ops.TreeBuffers(b.T, 3, F16)
    want = ops.tree_attn(*dev, bufs)
    assert (out.float() - want.float()).abs().max() <= 4 * 2.0**-11 * 448 / S_ENC_V
    assert (lse - bufs.lse).abs().max() <= 1e-4


def test_rows_of_nobody_and_bad_sequences_stay():
    b = Prompts([(300, 100), (50, 70), (260, 2), (10, 0), (40, 66)], 8, pad_rows=5)
    b.lens[4] = 65            # fewer cached tokens than query tokens
    bufs = b.buffers(BF16)
    bufs.out.fill_(3.0)
    bufs.lse.fill_(4.0)
    out, lse, cache = b.go(BF16, bufs=bufs)
    assert cache.read_status() == ops.STATUS_BAD_SEQ
    b.same(out, lse, BF16, only=[0, 1, 2])
    assert torch.all(out[172:] == 3.0) and torch.all(lse[172:] == 4.0)


def test_rows_that_several_sequences_claim():
    """q_start_loc that goes back: more tiles than rows can have; the call ends and flags it."""
    b = Prompts([(0, 200)] * 8, 15)
    cache, q, bt, lens, _ = b.device()
    qsl = _put([0, 200, 0, 200, 0, 200, 0, 200, 0])
    for t in (200, 400):
        bufs = ops.PrefillBuffers(t, 8, 16, BF16)
        ops.prefill_attn(cache, q[:t], bt, lens, qsl, bufs)
        assert cache.read_status() == ops.STATUS_BAD_SEQ
    ok = b.go(BF16)
    b.same(*ok[:2], BF16)


def test_pages_outside_the_pool_are_not_seen():
    b = Prompts([(700, 133), (500, 1)], 9)
    dev = list(b.device())
    bad = b.bt.copy()
    bad[0, 2], bad[1, 0] = b.pool.shape[0], -1
    dev[2] = torch.from_numpy(bad).to(DEV)
    out, lse, cache = b.go(F16, dev=dev)
    assert cache.read_status() == ops.STATUS_BAD_PAGE
    b.same(out, lse, F16, hidden={0: [2], 1: [0]})


def test_a_query_that_is_no_number_stays_so():
    b = Prompts([(2500, 90), (0, 40)], 20)
    b.q8[1, 5, 17] = 0x7F
    b.q8[70, 0, 0] = 0xFF
    b.q8[120, 15, 127] = 0x7F
    ends = np.concatenate([2500 + 1 + np.arange(90), 1 + np.arange(40)])
    b.q8[100, 3, 3] = 0x7F
    ends[100] = 0                 # sees nothing
    out, lse, cache = b.go(F16, ends=ends)
    bad = torch.zeros((b.T, 16), dtype=torch.bool, device=DEV)
    bad[1, 5] = bad[70, 0] = bad[120, 15] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad) and cache.read_status() == 0
    assert not out[100].any() and torch.isneginf(lse[100]).all()


def test_scores_near_zero_are_a_mean_and_scales_have_an_end():
    b = Prompts([(900, 70)], 19)
    out, lse, cache = b.go(F16, softmax_scale=1e-30)
    _, v8 = zip(*(tree.page_operands(b.pool[b.bt[0, i]]) for i in range(8)))
    v = formats.decode_e4m3(np.concatenate(v8)) / float(np.float32(S_ENC_V))
    for j in (0, 33, 69):
        m, size = v[: 901 + j].mean(0), np.abs(v[: 901 + j]).mean(0)
        tol = (2.0**-11 + 2004 * 2.0**-24) * size + 2.0**-11 * np.abs(m) + 2.0**-24
        assert np.all(np.abs(out[j].double().cpu().numpy() - m.repeat(4, 0)) <= tol.repeat(4, 0))
    # the largest scale: scores of 2^26; the largest key takes all where it leads by enough
    top = 2.0**26 / (128 * 448 * 448 * 1.4426951) * S_ENC_K * (1 - 1e-6)
    out, lse, cache = b.go(F16, softmax_scale=top)
    assert torch.isfinite(lse).all() and cache.read_status() == 0
    q, sure = formats.decode_e4m3(b.q8), 0
    k8, _ = zip(*(tree.page_operands(b.pool[b.bt[0, i]]) for i in range(8)))
    k = formats.decode_e4m3(np.concatenate(k8))
    for j in range(70):
        for h in range(16):
            keys, vals = k[: 901 + j, h // 4], v[: 901 + j, h // 4]
            z = keys @ q[j, h]
            first, second = np.sort(z)[[-1, -2]]
            if (first - second - 260 * 2.0**-24 * (np.abs(keys) @ np.abs(q[j, h])).max()) * top / S_ENC_K < 26:
                continue
            sure += 1
            want = vals[np.argmax(z)]
            # a weight of up to 2^12, rounded to f16; its sum and the scale round once each, then the type
            assert np.all(np.abs(out[j, h].double().cpu().numpy() - want) <= np.abs(want) * (2.0**-10 + 2.0**-20) + 2.0**-24), (j, h)
    assert sure > 100
    with pytest.raises(ops.MsaError):
        b.go(F16, softmax_scale=top * 1.01)


def test_repeats_are_bit_equal_and_calls_share_a_workspace():
    small, large = Prompts([(5000, 2), (30, 100)], 21), Prompts([(4000, 140), (3000, 330)], 22)
    bufs = [x.buffers(F16) for x in (small, large)]
    bufs[0].ws = bufs[1].ws
    first = {}
    for turn in range(4):
        for i, x in enumerate((small, large)):
            out, lse, _ = x.go(F16, bufs=bufs[i])
            if turn == 0:
                x.same(out, lse, F16)
                first[i] = out.clone(), lse.clone()
            assert torch.equal(out, first[i][0]) and torch.equal(lse, first[i][1])


def test_captured_graphs_follow_their_inputs_and_share_a_workspace():
    a, b = Prompts([(1000, 80), (300, 64)], 23), Prompts([(2000, 144)], 24)
    bufs = [x.buffers(BF16) for x in (a, b)]
    bufs[1].ws = bufs[0].ws if bufs[0].ws.numel() > bufs[1].ws.numel() else bufs[1].ws
    bufs[0].ws = bufs[1].ws
    devs, graphs = [x.device() for x in (a, b)], []
    torch.cuda.synchronize()
    for x, dev, buf in zip((a, b), devs, bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.prefill_attn(*dev, buf)
        graphs.append(g)
    for x, dev in zip((a, b), devs):
        x.q8 = x.q8[::-1].copy()
        dev[1].copy_(torch.from_numpy(x.q8))
    a.seqs, a.lens = [(900, 80), (190, 64)], np.array([980, 254], np.int32)  # shorter than captured
    devs[0][3].copy_(torch.from_numpy(a.lens))
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for x, buf, dev in zip((a, b), bufs, devs):
        x.same(buf.out, buf.lse, BF16)
        assert dev[0].read_status() == 0


def test_on_another_stream_without_lse_and_with_slices():
    b = Prompts([(500, 100)], 25)
    cache, q, bt, lens, qsl = b.device()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    bufs = b.buffers(F16)
    with torch.cuda.stream(other):
        ops.prefill_attn(cache, q, bt, lens, qsl, bufs)
    other.synchronize()
    b.same(bufs.out, bufs.lse, F16)
    keep = bufs.lse.clone()
    stream = torch.cuda.current_stream().cuda_stream
    out = torch.zeros_like(bufs.out)
    rc = ops.lib().msa_prefill_attn(cache.packed(), q.data_ptr(), 16, float(SCALE), bt.data_ptr(), bt.shape[1], lens.data_ptr(),
                                    qsl.data_ptr(), 1, b.T, 0, None, bufs.n_pages, 2, out.data_ptr(), None, bufs.ws.data_ptr(),
                                    bufs.ws.numel(), stream)
    assert rc == 0 and torch.equal(out, bufs.out) and torch.equal(keep, bufs.lse)
    with pytest.raises(ValueError):
        ops.prefill_attn(cache, q, bt.repeat(2, 1), lens, qsl, bufs)
    with pytest.raises(ValueError):
        ops.prefill_attn(cache, q[:50], bt, lens, qsl, bufs)
    with pytest.raises(TypeError):
        ops.prefill_attn(cache, q, bt, lens, qsl, bufs, ends=torch.zeros(100, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        ops.PrefillBuffers(1, 1, 1, torch.float32)


def test_a_missing_page_ends_the_call_and_the_next_one_is_right():
    """Every CTA leaves out its first page (the library's test hook): the waits run out after 20 ms,
    the call reports it, and the next one on the same workspace is right."""
    b = Prompts([(3000, 300)], 26)
    dev = b.device()
    bufs = b.buffers(F16)
    want, lse, cache = b.go(F16, dev=dev, bufs=bufs)
    want = want.clone()
    try:
        ops.set_fault_injection(ops.INJECT_ATTENTION_TIMEOUT, 20_000_000)
        b.go(F16, dev=dev, bufs=bufs)
    finally:
        ops.set_fault_injection(0, 0)
    assert cache.read_status() == ops.STATUS_TIMEOUT
    cache.status.zero_()
    for _ in range(2):
        out, lse, _ = b.go(F16, dev=dev, bufs=bufs)
        assert torch.equal(out, want) and cache.read_status() == 0


def test_pages_whose_offsets_pass_32_bits():
    b = Prompts([(900, 95), (260, 1)], 33)
    small, q, bt, lens, qsl = b.device()
    n, far = small.n_pages, 270_000
    kv = torch.empty((far, ops.KV_PAGE_BYTES), dtype=torch.uint8, device=DEV)
    ix = torch.zeros((far, ops.IDX_PAGE_BYTES), dtype=torch.uint8, device=DEV)
    kv[far - n:] = small.kv_pool
    big = ops.KVCache.from_pools(kv, ix, S_ENC_K, S_ENC_V)
    pages = torch.where(bt >= 0, bt + (far - n), bt)
    a, b2 = b.buffers(F16), b.buffers(F16, 30_000)  # (a workspace of 5.9 GB, too)
    ops.prefill_attn(small, q, bt, lens, qsl, a)
    ops.prefill_attn(big, q, pages, lens, qsl, b2)
    assert torch.equal(a.out, b2.out) and torch.equal(a.lse, b2.lse)
    b.same(a.out, a.lse, F16)


def test_a_prompt_with_an_image_is_written_attended_forked_and_continued():
    """The whole way: pages for the prompt, rotary positions on three axes, attention in which the
    image's tokens see all of it, two forks, a tree of drafts on each, the accepted ones committed,
    and one more token over what is left."""
    g = torch.Generator(device=DEV)
    g.manual_seed(40)
    n, first, span = 300, 40, 144
    caches = [ops.KVCache(24, S_ENC_K, S_ENC_V, DEV) for _ in range(2)]
    layers, pool = ops.CacheLayers(caches), ops.PagePool(24)
    table, lens = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    rope, axes = ops.rope_table_scaled(2048, 128), ops.rope_axes([16, 24, 24])

    def rows(m):
        x = torch.randn((m, 33, 128), generator=g, device=DEV).to(BF16)
        return x[:, :16], x[:, 16:20], x[:, 20:24], x[:, 24]

    def write(slots, pos, x):
        return [ops.rotary_insert(c, *x, rope, pos, slots, axes=axes)[0] for c in caches]

    starts = _put([0, n, n, n])
    slots = ops.extend_sequences(pool, table, lens, starts, torch.empty(n, dtype=torch.int64, device=DEV))
    at = np.arange(n)
    image = (at >= first) & (at < first + span)
    pos = np.stack([np.where(image, first, at), np.where(image, first + (at - first) // 12, at), np.where(image, first + (at - first) % 12, at)])
    q8 = write(slots, _put(pos), rows(n))
    ends = np.where(image, first + span, at + 1)
    b = Prompts.__new__(Prompts)
    b.seqs, b.T = [(0, n), (0, 0), (0, 0)], n
    b.pool, b.bt, b.qsl, b.q8 = caches[0].kv_pool.cpu().numpy(), table.cpu().numpy(), np.array([0, n, n, n]), q8[0].cpu().numpy()
    bufs = ops.PrefillBuffers(n, 3, 3, BF16)
    ops.prefill_attn(caches[0], q8[0], table, lens, starts, bufs, ends=_put(ends))
    b.same(bufs.out, bufs.lse, BF16, ends=ends)

    ops.fork_sequences(layers, pool, table, lens, _put([0, 0]), _put([1, 2]))
    starts = _put([0, 0, 8, 16])
    slots = ops.extend_sequences(pool, table, lens, starts, torch.empty(16, dtype=torch.int64, device=DEV))
    words = [1, 3, 5, 9, 19, 37, 83, 16 + 3 + 128]  # ancestors and itself
    depth = [bin(w).count("1") - 1 for w in words]
    q8 = write(slots, _put(np.tile([n + d for d in depth] * 2, (3, 1))), rows(16))
    tree_bufs = ops.TreeBuffers(16, 3, BF16)
    ops.tree_attn(caches[0], q8[0], table, lens, starts, tree_bufs, tree_mask=_put(words * 2, torch.int64))
    kept = ops.read_kv(caches[1], slots[[0, 1, 4, 6]], torch.float32)
    accepted = _put([0, 0b1010011, 0b1], torch.int64)  # a path of four, and the root alone
    new = ops.commit_drafts(layers, table, lens, starts, accepted)
    assert new.tolist() == [300, 304, 301]
    lens.copy_(new)
    row = table[1].long()
    moved = ops.read_kv(caches[1], torch.stack([row[p // 128] * 128 + p % 128 for p in range(300, 304)]), torch.float32)
    assert all(torch.equal(x, y) for x, y in zip(kept, moved))

    starts = _put([0, 0, 1, 2])
    slots = ops.extend_sequences(pool, table, lens, starts, torch.empty(2, dtype=torch.int64, device=DEV))
    q8 = write(slots, _put(np.tile([304, 301], (3, 1))), rows(2))
    bufs = ops.PrefillBuffers(2, 3, 6, BF16)
    ops.prefill_attn(caches[0], q8[0], table, lens, starts, bufs)
    b.seqs, b.T, b.qsl = [(300, 0), (304, 1), (301, 1)], 2, np.array([0, 0, 1, 2])
    b.pool, b.bt, b.q8 = caches[0].kv_pool.cpu().numpy(), table.cpu().numpy(), q8[0].cpu().numpy()
    b.same(bufs.out, bufs.lse, BF16)
    ops.release_sequences(pool, table, lens, _put([0, 1, 2]))
    assert not pool.refs.any() and not lens.any() and (table == -1).all()
    assert pool.status.item() == 0 and caches[0].read_status() == 0 and caches[1].read_status() == 0
