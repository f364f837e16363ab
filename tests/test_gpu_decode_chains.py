"""Decode steps among the calls around a prompt, in a row without waits: the bytes are those of the same calls
one at a time, on the stream and replayed.  (The step's kernels and the calls between them each begin launching
while the one before still runs.)"""

import pytest
import torch

from nvfp4_kv_block_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGES, ROWS, COLS, STEPS = 120, 5, 24, 4


class Server:
    """A prompt a row, then steps of one token each: written, attended over selected blocks, over all of them, by the
    single launch and as a tree of one draft; a fork and a release between the steps."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.cache = ops.KVCache(PAGES, 1.5, 0.75, DEV)
        self.pool = ops.PagePool(PAGES)
        self.table = torch.full((ROWS, COLS), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        self.rope = ops.rope_table_scaled(4096, 128)
        new = [2300, 700, 130, 2, 0]
        self.first = self.put([sum(new[:i]) for i in range(ROWS + 1)])
        self.n = sum(new)
        self.rows = torch.randn((self.n, 33, 128), generator=g, device=DEV).to(torch.bfloat16)
        self.pos = torch.cat([torch.arange(n, device=DEV, dtype=torch.int32) for n in new])
        self.slots = torch.full((self.n,), -1, dtype=torch.int64, device=DEV)
        self.bufs = ops.PrefillBuffers(self.n, ROWS, 40)
        self.step_rows = torch.randn((STEPS, ROWS, 33, 128), generator=g, device=DEV).to(torch.bfloat16)
        self.w = torch.rand((ROWS, 8), generator=g, device=DEV)
        self.step_pos = self.put(list(range(5, 5 + ROWS)))
        self.starts = self.put(list(range(ROWS + 1)))
        self.src, self.dst = self.put([1, 0]), self.put([4, 3])
        self.q8 = torch.zeros((self.n, 16, 128), dtype=torch.uint8, device=DEV)
        self.qi8 = torch.zeros((self.n, 8, 128), dtype=torch.uint8, device=DEV)
        self.seen, self.steps = [], []
        for _ in range(STEPS):
            self.steps.append({
                "slots": torch.full((ROWS,), -1, dtype=torch.int64, device=DEV),
                "q8": torch.zeros((ROWS, 16, 128), dtype=torch.uint8, device=DEV),
                "qi8": torch.zeros((ROWS, 8, 128), dtype=torch.uint8, device=DEV),
                "one": ops.DecodeBuffers(ROWS, COLS, 1, DEV), "cut": ops.DecodeBuffers(ROWS, COLS, 3, DEV), "fused": ops.FusedBuffers(ROWS, COLS, DEV),
                "all": ops.PrefillBuffers(ROWS, ROWS, ROWS * COLS), "tree": ops.TreeBuffers(ROWS, ROWS),
                "kv": [torch.zeros((ROWS, 4, 128), device=DEV), torch.zeros((ROWS, 4, 128), device=DEV), torch.zeros((ROWS, 128), device=DEV)],
            })

    @staticmethod
    def put(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def insert(self, x, pos, slots, q8, qi8):
        ops.rotary_insert(self.cache, x[:, :16], x[:, 16:20], x[:, 20:24], x[:, 24], self.rope, pos, slots, q_idx=x[:, 25:], q8=q8, qi8=qi8)

    def program(self):
        at = (self.table, self.lens)
        yield lambda: ops.extend_sequences(self.pool, *at, self.first, self.slots)
        yield lambda: self.insert(self.rows, self.pos, self.slots, self.q8, self.qi8)
        yield lambda: ops.prefill_attn(self.cache, self.q8, *at, self.first, self.bufs)
        for i, s in enumerate(self.steps):
            if i == 1:
                yield lambda: ops.release_sequences(self.pool, *at, self.dst)
                yield lambda: ops.fork_sequences(self.cache, self.pool, *at, self.src, self.dst)
            yield lambda: ops.extend_sequences(self.pool, *at, self.starts, s["slots"])
            yield lambda: self.insert(self.step_rows[i], self.step_pos, s["slots"], s["q8"], s["qi8"])
            for name in ("one", "cut"):
                yield lambda: ops.decode_step(self.cache, s["q8"], s["qi8"], self.w, *at, self.starts, s[name])
            # (the same selection again, behind a call that is no part of the step)
            yield lambda: ops.read_kv(self.cache, s["slots"], k=s["kv"][0], v=s["kv"][1], idx_k=s["kv"][2])
            yield lambda: ops.sparse_attn_decode(self.cache, s["q8"], s["one"].sel, s["one"].n_sel, *at, self.starts, 1, o_part=s["one"].o_part, lse_part=s["one"].lse_part)
            yield lambda: ops.tree_attn(self.cache, s["q8"], *at, self.starts, s["tree"])
            yield lambda: ops.decode_fused(self.cache, s["q8"], s["qi8"], self.w, *at, self.starts, s["fused"])
            yield lambda: ops.prefill_attn(self.cache, s["q8"], *at, self.starts, s["all"])

    def run(self, wait=False):
        for call in self.program():
            call()
            if wait:
                torch.cuda.synchronize()

    def state(self):
        torch.cuda.synchronize()
        out = [self.table, self.lens, self.pool.refs, self.pool.status, self.cache.kv_pool, self.cache.idx_pool, self.cache.status, self.q8, self.qi8,
               self.bufs.out, self.bufs.lse]
        for s in self.steps:
            out += [s["slots"], s["q8"], s["qi8"], *s["kv"], s["all"].out, s["all"].lse, s["tree"].out, s["tree"].lse]
            for b in (s["one"], s["cut"], s["fused"]):
                out += [b.sel, b.n_sel, b.out]
        return [t.clone() for t in out]


def _same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), i


@pytest.fixture(scope="module")
def want():
    s = Server(5)
    s.run(wait=True)
    state = s.state()
    assert s.cache.read_status() == 0 and s.pool.status.item() == 0 and s.lens.tolist() == [2304, 704, 134, 2304, 704]
    return state


def test_steps_without_waits(want):
    for _ in range(3):
        s = Server(5)
        torch.cuda.synchronize()
        s.run()
        _same(s.state(), want)


def test_captured_steps(want):
    s = Server(5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    graph.replay()
    _same(s.state(), want)
