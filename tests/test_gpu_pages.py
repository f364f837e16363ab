"""GPU parity of the page calls against the oracle: tables, lengths, counts, slots and
every byte of the pools are compared exactly.
"""

import random

import numpy as np
import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from oracle import pages
from test_gpu_transfer import _random_caches

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


class State:
    """A pool, a table and lengths, here and in the oracle."""

    def __init__(self, n_pages, rows, cols, status=None):
        self.refs, self.table, self.lens = [0] * n_pages, [[-1] * cols for _ in range(rows)], [0] * rows
        self.pool = ops.PagePool(n_pages, status)
        self.d_table, self.d_lens = _dev(self.table), _dev(self.lens)

    def starts(self, new):
        return _dev(np.concatenate([[0], np.cumsum(new)]).tolist())

    def extend(self, new, pad=0):
        n = sum(max(x, 0) for x in new) + pad
        got = ops.extend_sequences(self.pool, self.d_table, self.d_lens, self.starts(new), torch.full((n,), 77, dtype=torch.int64, device=DEV))
        want, status = pages.extend(self.refs, self.table, self.lens, new, n)
        assert got.tolist() == want
        self.check(status)
        return want

    def fork(self, src, dst, caches, host):
        ops.fork_sequences(caches, self.pool, self.d_table, self.d_lens, _dev(src), _dev(dst))
        copies, status = pages.fork(self.refs, self.table, self.lens, src, dst)
        for kv, ix in host:
            pages.copy(kv, ix, copies)
        self.check(status)

    def release(self, rows):
        ops.release_sequences(self.pool, self.d_table, self.d_lens, _dev(rows))
        self.check(pages.release(self.refs, self.table, self.lens, rows))

    def check(self, status):
        assert self.d_table.tolist() == self.table
        assert self.d_lens.tolist() == self.lens
        assert self.pool.refs.tolist() == self.refs
        words = self.pool.free_mask.tolist()
        assert [words[p // 32] >> (p % 32) & 1 for p in range(len(self.refs))] == [int(n == 0) for n in self.refs]
        assert self.pool.status.item() == status
        self.pool.status.zero_()


def _host(caches):
    return [(c.kv_pool.cpu().numpy().copy(), c.idx_pool.cpu().numpy().copy()) for c in caches]


def _same(caches, host):
    for c, (kv, ix) in zip(caches, host):
        np.testing.assert_array_equal(c.kv_pool.cpu().numpy(), kv)
        np.testing.assert_array_equal(c.idx_pool.cpu().numpy(), ix)


@pytest.mark.parametrize("n_pages,rows,cols,layers", [(5, 3, 2, 1), (32, 6, 5, 1), (100, 17, 6, 2), (700, 70, 9, 3)])
def test_random_lives(n_pages, rows, cols, layers):
    rng = random.Random(n_pages)
    caches = _random_caches(layers, n_pages, n_pages)
    host = _host(caches)
    s = State(n_pages, rows, cols)
    bunch = ops.CacheLayers(caches)
    for _ in range(12):
        s.extend([rng.choice([0, 0, 1, 7, 128, 130, 300]) for _ in range(rows)], pad=rng.choice([0, 3]))
        n = rng.randint(1, rows)
        s.fork([rng.randrange(rows) for _ in range(n)], [rng.randrange(-1, rows + 1) for _ in range(n)], bunch, host)
        s.release([rng.randrange(-1, rows + 1) for _ in range(rng.randint(1, rows))])
    _same(caches, host)


@pytest.mark.parametrize("n_pages,rows", [(1, 1), (31, 31), (33, 40), (4097, 4096), (140001, 5)])
def test_extend_sizes(n_pages, rows):
    """One page, pages that end inside a mask word, more pages than one pass of the scan, more rows than threads."""
    s = State(n_pages, rows, 3)
    rng = random.Random(rows)
    s.extend([rng.choice([0, 1, 129]) if rows > 5 else 200 for _ in range(rows)])
    s.extend([rng.choice([0, 1, 129]) if rows > 5 else 100 for _ in range(rows)], pad=1)
    s.release(list(range(0, rows, 2)))
    s.extend([5] * rows)


def test_lowest_free_pages_far_into_the_pool():
    """Every page below 139,000 is held, and a few beyond."""
    refs = torch.ones(140001, dtype=torch.int32, device=DEV)
    free = [139003, 139999, 140000]
    refs[free] = 0
    pool = ops.PagePool.from_refs(refs)
    table, lens = _dev([[-1, -1], [-1, -1]]), _dev([0, 0])
    slots = ops.extend_sequences(pool, table, lens, _dev([0, 130, 131]), torch.empty(131, dtype=torch.int64, device=DEV))
    assert table.tolist() == [free[:2], [free[2], -1]] and lens.tolist() == [130, 1]
    assert slots.tolist() == [free[0] * 128 + i for i in range(128)] + [free[1] * 128, free[1] * 128 + 1, free[2] * 128]
    assert refs.sum().item() == 140001 and pool.status.item() == 0


def test_extend_a_whole_prompt_and_reserved_pages():
    s = State(600, 3, 520)
    s.table[1][0], s.table[1][2] = 9, 11  # held in reserve, the second behind a hole
    s.refs[9] = s.refs[11] = 1
    s.pool = ops.PagePool.from_refs(_dev(s.refs))
    s.d_table = _dev(s.table)
    s.extend([300, 500, 65536 - 800])
    s.extend([0, 0, 0])
    s.release([1])


@pytest.mark.parametrize("total", [2048, 4096, 4097, 6000])
def test_extend_by_thousands_of_tokens(total):
    """Rows of many pages and of few, one too long, one of nothing, from the middle of a page; then the pool runs dry."""
    s = State(72, 5, 60)
    s.extend([5, 0, 130, 1, 0])
    s.extend([total - 1039, 0, 1000, 0, 30], pad=9)
    s.extend([7, 60 * 128 + 1, 5, 0, 0], pad=9)                   # the second is longer than its row
    s.extend([1, 1, 1, 1, 1])
    s.extend([1500, 0, 40, 7000, 2], pad=1)                       # from the fourth on none finds its pages
    s.release([0, 4])
    s.extend([0, 0, 0, 2500, 900])
    s.release([3, 2])
    rows = State(700, 257, 3)
    rows.extend([20 + i % 9 for i in range(257)])
    rows.extend([130 if i % 31 == 0 else 3 for i in range(257)], pad=2000)


def test_extend_refusals():
    s = State(20, 4, 2)
    s.extend([1, 250, 257, 5])         # the third is longer than its row
    assert s.lens == [1, 250, 0, 5]
    s.table[0][0] = -1                  # a sequence whose last tokens have no page
    s.d_table[0, 0] = -1
    s.extend([2, 1, 0, 1])
    assert s.lens == [1, 251, 0, 6]
    # a row whose end is before its start, and one that ends behind the tokens
    got = ops.extend_sequences(s.pool, s.d_table, s.d_lens, _dev([0, 2, 1, 1, 9]), torch.empty(4, dtype=torch.int64, device=DEV))
    assert s.pool.status.item() == ops.STATUS_BAD_SEQ | ops.STATUS_BAD_PAGE
    assert s.d_lens.tolist() == [1, 251, 0, 6] and got.tolist() == [-1] * 4


def test_fork_shapes():
    """Lengths around a page's end, one source for several rows, sources without tokens, too few pages."""
    caches = _random_caches(2, 40, 3)
    host = _host(caches)
    s = State(40, 24, 4)
    s.extend([0, 1, 127, 128, 129, 15, 16, 17, 255, 257] + [0] * 14)
    s.fork(list(range(10)) + [4, 4], list(range(10, 22)), caches, host)
    _same(caches, host)
    held = sum(n > 0 for n in s.refs)
    # fill the pool but for one page
    s.extend([0] * 22 + [128 * min(4, 39 - held), 128 * max(0, 35 - held)])
    left = sum(n == 0 for n in s.refs)
    s.release([10, 11, 12, 13])
    s.fork([1, 3, 2, 4, 3], [10, 11, 12, 13, 0], caches, host)
    _same(caches, host)
    assert left >= 0


def test_fork_with_a_bad_page():
    caches = _random_caches(1, 6, 4)
    host = _host(caches)
    s = State(6, 4, 3)
    s.extend([200, 300, 0, 0])
    s.table[0][1] = 6
    s.table[1][0] = 99
    s.d_table = _dev(s.table)
    s.fork([0, 1], [2, 3], caches, host)  # a last page outside; a full page outside is taken over
    assert s.lens == [200, 300, 0, 300]
    _same(caches, host)


@pytest.mark.parametrize("tokens", [None, [128, 1, 15, 16, 17, 0, -3, 127, 500, 64]])
def test_copy_pages(tokens):
    caches = _random_caches(3, 30, 5)
    host = _host(caches)
    src, dst = [0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [19, 18, 17, 16, 15, 14, 13, 12, 11, 10]
    src[1], dst[2], dst[3] = -1, -5, 3
    ops.copy_pages(caches, _dev(src), _dev(dst), None if tokens is None else _dev(tokens))
    todo = [(a, b, min(128, (tokens or [128] * 10)[i])) for i, (a, b) in enumerate(zip(src, dst)) if min(a, b) >= 0]
    for kv, ix in host:
        pages.copy(kv, ix, todo)
    _same(caches, host)
    assert caches[0].read_status() == 0
    ops.copy_pages(caches[1], _dev([30, 0]), _dev([0, 30]))
    _same(caches, host)
    assert caches[1].read_status() == ops.STATUS_BAD_PAGE


def _accepted(rng, n):
    return rng.choice([0, (1 << n) - 1 if n else 0, rng.getrandbits(64), rng.getrandbits(64) & rng.getrandbits(64) & rng.getrandbits(64) | 1])


@pytest.mark.parametrize("seed,layers", [(1, 1), (2, 3), (3, 1), (4, 2)])
def test_commit(seed, layers):
    rng = random.Random(seed)
    drafts = [rng.choice([0, 1, 2, 8, 33, 63, 64]) for _ in range(20)]
    lens = [n + rng.choice([0, 1, 64, 100, 127, 128, 200]) for n in drafts]
    counts = [-(-n // 128) for n in lens]
    total = sum(counts)
    perm = rng.sample(range(total), total)
    table, at = [], 0
    for n in counts:
        table.append(perm[at: at + n] + [-1] * (4 - n))
        at += n
    words = [_accepted(rng, n) for n in drafts]
    caches = _random_caches(layers, total, seed)
    host = _host(caches)
    new = ops.commit_drafts(caches, _dev(table), _dev(lens), _dev(np.concatenate([[0], np.cumsum(drafts)]).tolist()),
                            _dev([w - (1 << 64) if w >> 63 else w for w in words], torch.int64))
    for kv, ix in host:
        want, status = pages.commit(kv, ix, table, lens, drafts, words)
    assert new.tolist() == want and status == 0 and caches[0].read_status() == 0
    _same(caches, host)


def test_commit_refusals():
    caches = _random_caches(1, 4, 9)
    host = _host(caches)
    table = [[0, -1], [1, 9], [2, -1], [3, -1]]
    lens, drafts, words = [3, 130, 100, 300], [4, 5, 65, 2], [0b1010, 0b10110, 0b10, 0b10]
    new = ops.commit_drafts(caches, _dev(table), _dev(lens), _dev(np.concatenate([[0], np.cumsum(drafts)]).tolist()), _dev(words, torch.int64))
    want, status = pages.commit(*host[0], table, lens, drafts, words)
    # more drafts than tokens, a page outside the pool under one of the moves, 65 drafts, a row that is too short
    assert new.tolist() == want == [3, 128, 100, 300]
    assert caches[0].read_status() == status == ops.STATUS_BAD_SEQ | ops.STATUS_BAD_PAGE
    _same(caches, host)
    with pytest.raises(ops.MsaError):
        lens = _dev(lens)
        ops.commit_drafts(caches, _dev(table), lens, _dev([0, 1, 2, 3, 4]), _dev(words, torch.int64), lens)
    with pytest.raises(ValueError):
        ops.commit_drafts(caches, _dev(table), lens, _dev([0, 1, 2]), _dev(words, torch.int64))


def test_captured_and_replayed():
    """A graph of release, fork and extend leaves the same state at every replay."""
    caches = _random_caches(2, 64, 11)
    s = State(64, 8, 4)
    s.extend([100, 300, 0, 0, 0, 0, 0, 0])
    bunch = ops.CacheLayers(caches)
    src, dst = _dev([0, 1, 1, 0]), _dev([2, 3, 4, 5])
    starts, slots = s.starts([0, 0, 30, 90, 1, 2, 0, 0]), torch.empty(123, dtype=torch.int64, device=DEV)

    def step():
        ops.release_sequences(s.pool, s.d_table, s.d_lens, dst)
        ops.fork_sequences(bunch, s.pool, s.d_table, s.d_lens, src, dst)
        ops.extend_sequences(s.pool, s.d_table, s.d_lens, starts, slots)

    step()
    want = [t.clone() for t in (s.d_table, s.d_lens, s.pool.refs, s.pool.free_mask, slots, caches[1].kv_pool)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        got = (s.d_table, s.d_lens, s.pool.refs, s.pool.free_mask, slots, caches[1].kv_pool)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert s.pool.status.item() == 0


def test_pages_on_another_stream_and_arguments():
    s = State(8, 2, 2)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        s.extend([3, 130])
    caches = _random_caches(1, 4, 1)  # fewer pages than the pool counts
    with pytest.raises(ops.MsaError):
        ops.fork_sequences(caches, s.pool, s.d_table, s.d_lens, _dev([0]), _dev([1]))
    with pytest.raises(TypeError):
        ops.extend_sequences(s.pool, s.d_table, s.d_lens.long(), _dev([0, 0, 0]), torch.empty(0, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ops.release_sequences(s.pool, s.d_table.t(), s.d_lens, _dev([0]))
    with pytest.raises(ValueError):
        ops.extend_sequences(s.pool, s.d_table, s.d_lens, _dev([0, 0]), torch.empty(0, dtype=torch.int64, device=DEV))


def _held(s, rows):
    """Pages of a caller's own in the rows: ``rows`` maps a row to {column: page}."""
    for b, cells in rows.items():
        for at, page in cells.items():
            s.table[b][at] = page
            s.refs[page] += 1
    s.pool = ops.PagePool.from_refs(_dev(s.refs))
    s.d_table = _dev(s.table)


@pytest.mark.parametrize("rows,cols", [(9, 4), (40, 700)])
def test_fork_leaves_rows_alone_that_hold_a_page_behind_a_hole(rows, cols):
    """Few entries and many, a page in the first, a middle and the last column; afterwards every page is dealt once."""
    caches = _random_caches(1, 64, 21)
    host = _host(caches)
    s = State(64, rows, cols)
    s.extend([200, 128] + [0] * (rows - 2))
    _held(s, {2: {1: 40}, 3: {cols - 1: 41}, 4: {0: 42}, 5: {cols // 2: 63, cols - 1: 62}})
    # (a pair that is left out names a row that a later one may have no more than it)
    src = [0, 0, 1, 0, 0, 1, 0] + [0, 1] * ((rows - 9) // 2)
    dst = [2, 3, 4, 5, 6, 7, 3] + list(range(8, 8 + len(src) - 7))
    before = [list(r) for r in s.table[2:6]]
    s.fork(src, dst, caches, host)
    assert s.table[2:6] == before and s.lens[2:8] == [0, 0, 0, 0, 200, 128]
    _same(caches, host)
    held = [p for r in s.table for p in r if p >= 0]
    assert s.refs == [held.count(p) for p in range(64)]
    s.release(list(range(rows)))
    assert not any(s.refs)


@pytest.mark.parametrize("rows,cols,n", [(4096, 5, 4000), (300, 4, 256), (220, 5, 205), (70, 15, 68), (1040, 17, 1024)])
def test_fork_of_many_rows_some_of_which_hold_pages(rows, cols, n):
    """More pairs than threads, entries at the number that the planning CTA looks at and beyond it."""
    caches = _random_caches(1, 5000, 22)
    host = _host(caches)
    s = State(5000, rows, cols)
    s.extend([129] + [0] * (rows - 1))
    rng = random.Random(cols)
    _held(s, {b: {rng.randrange(cols): 100 + b} for b in rng.sample(range(1, rows), min(60, rows // 3))})
    s.fork([0] * n, [1 + (i * 8 + i // (rows - 1)) % (rows - 1) for i in range(n)], caches, host)
    _same(caches, host)
    s.release(list(range(rows)))
    assert not any(s.refs)


def test_fork_from_a_pool_that_runs_dry():
    """One free page: the first pair that needs one gets it; later ones get none, and those that need none are made."""
    caches = _random_caches(2, 11, 23)
    host = _host(caches)
    s = State(11, 10, 4)
    s.extend([130, 256, 5, 512, 128, 0, 0, 0, 0, 0])
    s.release([4])
    assert sum(n == 0 for n in s.refs) == 2
    s.extend([0, 0, 0, 0, 3, 0, 0, 0, 0, 0])
    assert sum(n == 0 for n in s.refs) == 1
    copies, status = pages.fork(list(s.refs), [list(r) for r in s.table], list(s.lens), [2, 0, 1, 4, 9], [5, 6, 7, 8, 6])
    assert status & pages.NO_PAGES and len(copies) == 1
    s.fork([2, 0, 1, 4, 9], [5, 6, 7, 8, 6], caches, host)
    assert s.lens == [130, 256, 5, 512, 3, 5, 0, 256, 0, 0] and all(s.refs)
    s.fork([0, 3, 2], [6, 8, 9], caches, host)  # none left at all
    assert s.lens[6:] == [0, 256, 512, 0]
    _same(caches, host)


def test_random_lives_of_a_pool_that_is_too_small():
    """Extensions and forks that find too few pages, among those that find them."""
    rng = random.Random(77)
    short = {"extend": 0, "fork": 0}
    copied = 0
    for n_pages, rows, cols in ((9, 5, 3), (40, 20, 4)):
        caches = _random_caches(1, n_pages, n_pages)
        host = _host(caches)
        s = State(n_pages, rows, cols)
        for _ in range(40):
            new = [rng.choice([0, 0, 1, 60, 128]) if n < 300 else 0 for n in s.lens]
            _, status = pages.extend(list(s.refs), [list(r) for r in s.table], list(s.lens), new, sum(new))
            short["extend"] += status & pages.NO_PAGES != 0
            s.extend(new)
            src, dst = [rng.randrange(rows) for _ in range(4)], [rng.randrange(rows) for _ in range(4)]
            copies, status = pages.fork(list(s.refs), [list(r) for r in s.table], list(s.lens), src, dst)
            short["fork"] += status & pages.NO_PAGES != 0
            copied += len(copies)
            s.fork(src, dst, caches, host)
            s.release(rng.sample(range(rows), rng.choice([0, 1, rows // 4])) or [rng.randrange(rows)])
        _same(caches, host)
    assert short["extend"] >= 5 and short["fork"] >= 5 and copied >= 5


@pytest.mark.parametrize("scale", [1, 100])
def test_extend_grows_none_where_starts_go_back(scale):
    """Tokens that two sequences claim: few, and more than the planning CTA writes.  No slot of a token that is there already is
    given out, whatever the threads' order."""
    s = State(400, 4, 130)
    s.extend([60 * scale, 3, 50 * scale, 0])
    before = list(s.lens)
    for new in ([50 * scale, -10 * scale, 50 * scale, 0], [130 * 128, -(130 * 128 - 40 * scale), 50 * scale, 0], [0, 5, -5, 60 * scale]):
        n = 90 * scale
        got = ops.extend_sequences(s.pool, s.d_table, s.d_lens, s.starts(new), torch.full((n,), 77, dtype=torch.int64, device=DEV))
        want, status = pages.extend(s.refs, s.table, s.lens, new, n)
        assert got.tolist() == want == [-1] * n and status == ops.STATUS_BAD_SEQ and s.lens == before
        s.check(status)
    s.extend([50 * scale, 0, 1, 40 * scale])
