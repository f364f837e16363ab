"""Calls in a row: kernels begin launching while the one before still runs, so a chain without waits has
to give the bytes of the same calls one at a time, on one stream, on two at once, and replayed."""

import pytest
import torch

from nvfp4_kv_block_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGES, ROWS, COLS, N = 160, 6, 40, 700


class Server:
    """Two layers, a pool, and a fixed program of calls over inputs of a seed."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.caches = [ops.KVCache(PAGES, 1.5, 0.75, DEV) for _ in range(2)]
        self.layers, self.pool = ops.CacheLayers(self.caches), ops.PagePool(PAGES)
        self.table = torch.full((ROWS, COLS), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        self.new_lens = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        self.rope, self.axes = ops.rope_table_scaled(4096, 128), ops.rope_axes([24, 20, 20], dealt=True)
        self.rows = torch.randn((4, N, 33, 128), generator=g, device=DEV).to(torch.bfloat16)
        self.pos = torch.randint(0, 4096, (4, 3, N), generator=g, device=DEV, dtype=torch.int32)
        self.starts = [self.put(x) for x in ([0, 300, 301, 301, 301, 301, 690], [0, 1, 5, 5, 5, 5, 700],
                                             [0, 100, 164, 170, 234, 298, 298], [0, 8, 16, 24, 32, 40, 41])]
        self.src, self.dst, self.out_rows = self.put([0, 1]), self.put([2, 3]), self.put([3, 2, 3])
        self.accepted = torch.tensor([0b10110101, 0b1, 0xFF, 0b10, 0, 1], dtype=torch.int64, device=DEV)
        self.slots = [torch.full((N,), -1, dtype=torch.int64, device=DEV) for _ in range(4)]
        self.q8 = [[torch.zeros((N, 16, 128), dtype=torch.uint8, device=DEV) for _ in range(2)] for _ in range(4)]
        first = ops.PrefillBuffers(N, ROWS, 120, torch.bfloat16)
        self.bufs = [[first if i == j == 0 else ops.PrefillBuffers(N, ROWS, 120, torch.bfloat16, ws=first.ws) for j in range(2)] for i in range(4)]
        self.seen = [[torch.zeros((N, h, 128), device=DEV) if h > 1 else torch.zeros((N, 128), device=DEV) for h in (4, 4, 1)] for _ in range(8)]

    @staticmethod
    def put(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def step(self, i):
        """Tokens come, are written, attended and read back in both layers."""
        x = self.rows[i]
        yield lambda: ops.extend_sequences(self.pool, self.table, self.lens, self.starts[i], self.slots[i])
        for j, c in enumerate(self.caches):
            yield lambda: ops.rotary_insert(c, x[:, :16], x[:, 16:20], x[:, 20:24], x[:, 24], self.rope, self.pos[i], self.slots[i],
                                            q8=self.q8[i][j], axes=self.axes)
            yield lambda: ops.prefill_attn(c, self.q8[i][j], self.table, self.lens, self.starts[i], self.bufs[i][j], window=200 * (i == 2))
            k, v, idx = self.seen[2 * i + j]
            yield lambda: ops.read_kv(c, self.slots[i], k=k, v=v, idx_k=idx)

    def program(self):
        yield from self.step(0)
        yield lambda: ops.fork_sequences(self.layers, self.pool, self.table, self.lens, self.src, self.dst)
        yield from self.step(1)
        yield from self.step(2)
        yield lambda: ops.release_sequences(self.pool, self.table, self.lens, self.out_rows)
        yield from self.step(3)
        yield lambda: ops.commit_drafts(self.layers, self.table, self.lens, self.starts[3], self.accepted, self.new_lens)
        yield lambda: ops.copy_pages(self.layers, self.put_once, self.put_far)

    def run(self, wait=False):
        for call in self.program():
            call()
            if wait:
                torch.cuda.synchronize()

    def state(self):
        torch.cuda.synchronize()
        out = [self.table, self.lens, self.new_lens, self.pool.refs, self.pool.free_mask, self.pool.status]
        out += [t for c in self.caches for t in (c.kv_pool, c.idx_pool, c.status)]
        out += self.slots + [t for y in self.q8 for t in y] + [t for y in self.bufs for b in y for t in (b.out, b.lse)]
        return [t.clone() for t in out + [t for y in self.seen for t in y]]


def _server(seed):
    s = Server(seed)
    s.put_once, s.put_far = s.put([0, 1]), s.put([PAGES - 1, PAGES - 2])
    return s


def _same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), i


def test_a_chain_without_waits():
    want = _server(1)
    want.run(wait=True)
    want = want.state()
    assert want[5].item() == 0 and want[1].any() and want[8].item() == 0
    for _ in range(3):
        s = _server(1)
        s.run()
        _same(s.state(), want)


def test_two_chains_at_once():
    wants = []
    for seed in (2, 3):
        s = _server(seed)
        s.run(wait=True)
        wants.append(s.state())
    two, streams = [_server(2), _server(3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for pair in zip(*(s.program() for s in two)):
        for call, stream in zip(pair, streams):
            with torch.cuda.stream(stream):
                call()
    for s, want in zip(two, wants):
        _same(s.state(), want)


def test_a_captured_chain():
    want = _server(4)
    want.run(wait=True)
    want = want.state()
    warm = _server(4)
    warm.run()
    s = _server(4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    _same([s.lens], [torch.zeros_like(s.lens)])  # nothing ran
    graph.replay()
    _same(s.state(), want)
