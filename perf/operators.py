"""Measured cases of the verification operators of the NVFP4 cache.

Three operators that belong together when drafted tokens are verified against a
paged NVFP4 cache, each in a plain form (``own`` false: elementary torch
operations in 32 bits) and through the library (``own`` true):

  * write: rotary positions (half or interleaved pairs, the whole head or its
    first channels) on projected rows, FP8 queries and index queries, NVFP4 K/V
    and FP8 index keys written into their cache slots, and the values that the
    cache now holds read back (a prefill goes on with those values, so that it
    sees what later steps see);
  * read: the values of given cache slots in 16 or 32 bits;
  * tree: attention of a tree of drafted tokens over a sequence's whole cached
    context, or over one block selection shared by the tree.

Page format (128 tokens, 4 KV heads of 128 channels, 16-channel groups): per
head 18,432 bytes: K codes [128][64 B], K scales [8][128], V codes, V scales;
a 32-bit code word holds 8 E2M1 codes (magnitude of channel n at bits 4n..4n+2,
sign of channel n < 4 at bit 8n+7, of channel 4 + n at bit 8n+3), the 16-byte
chunk c of token t at chunk position c ^ ((t >> 1) & 3).  Index pages:
[128][128 B] E4M3, 16-byte chunk c of token t at position c ^ (t & 7).
"""

import math
import random

import numpy as np
import torch

own = False

HEADS, KV, DIM, IDX_HEADS = 16, 4, 128, 8
PAGE, HEAD_BYTES, PAGE_BYTES, IDX_BYTES = 128, 18432, 73728, 16384
OFF = {"k": (0, 8192), "v": (9216, 17408)}
S_ENC_K, S_ENC_V = 89.6, 74.75  # 448 / amax of K and V that reach 5 and about 6
DEC_K, DEC_V = (float(np.float32(1) / np.float32(s)) for s in (S_ENC_K, S_ENC_V))  # the fp32 factors of the way back
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------------


def listed():
    return [
        # one sequence's drafts of one layer: latency
        {"name": "write_draft_8", "op": "write", "n": 8, "dtype": "bf16", "rot": 128, "inter": False, "packed": False, "order": "pages", "skip": 0},
        # a ragged step's rows as slices of one projection, half of each head turned, padding rows
        {"name": "write_mixed_2037", "op": "write", "n": 2037, "dtype": "fp16", "rot": 64, "inter": True, "packed": True, "order": "pages", "skip": 37},
        # a prefill chunk
        {"name": "write_prefill_8192", "op": "write", "n": 8192, "dtype": "bf16", "rot": 128, "inter": False, "packed": True, "order": "pages", "skip": 0},
        # a bulk refill from 32-bit rows at scattered slots
        {"name": "write_bulk_16384", "op": "write", "n": 16384, "dtype": "fp32", "rot": 96, "inter": True, "packed": False, "order": "scatter", "skip": 0},
        # a short prefix at scattered slots
        {"name": "read_short_300", "op": "read", "n": 300, "dtype": "fp16", "order": "scatter", "skip": 0},
        # scattered tokens in 32 bits, some left out
        {"name": "read_scatter_20011", "op": "read", "n": 20011, "dtype": "fp32", "order": "scatter", "skip": 511},
        # a long cached prefix, whole pages anywhere in the pool
        {"name": "read_prefix_131072", "op": "read", "n": 131072, "dtype": "bf16", "order": "pages", "skip": 0},
        # one sequence, one token: latency
        {"name": "tree_one_4096", "op": "tree", "seqs": 1, "ctx": 4096, "least": 1.0, "nq": 1, "nq_least": 1, "dtype": "bf16", "sel": 0, "mask": False},
        # batched single-token steps
        {"name": "tree_step_32x32768", "op": "tree", "seqs": 32, "ctx": 32768, "least": 1.0, "nq": 1, "nq_least": 1, "dtype": "bf16", "sel": 0, "mask": False},
        # ragged sequences with trees of 4 to 24 drafts
        {"name": "tree_ragged_24x30720", "op": "tree", "seqs": 24, "ctx": 30720, "least": 0.2, "nq": 24, "nq_least": 4, "dtype": "fp16", "sel": 0, "mask": True},
        # trees of 8 drafts that share their root's block selection
        {"name": "tree_shared_64x32768", "op": "tree", "seqs": 64, "ctx": 32768, "least": 0.5, "nq": 8, "nq_least": 8, "dtype": "bf16", "sel": 16, "mask": True},
        # wide trees over long contexts
        {"name": "tree_wide_8x131072", "op": "tree", "seqs": 8, "ctx": 131072, "least": 0.9, "nq": 64, "nq_least": 64, "dtype": "bf16", "sel": 0, "mask": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "tree", "tree"])
    if op == "write":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        n = _log_int(rng, 1, 16384)
        return {"op": op, "n": n, "dtype": dtype, "rot": 16 * rng.randint(0, 8), "inter": rng.random() < 0.5, "packed": rng.random() < 0.5,
                "order": rng.choice(["pages", "scatter"]), "skip": rng.choice([0, n // 8])}
    if op == "read":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        n = _log_int(rng, 1, 131072 if dtype != "fp32" else 65536)
        return {"op": op, "n": n, "dtype": dtype, "order": rng.choice(["pages", "scatter"]), "skip": rng.choice([0, n // 8])}
    seqs = _log_int(rng, 1, 64)
    nq = _log_int(rng, 1, 64)
    ctx = _log_int(rng, 1, min(131072, 1048576 // seqs, 67108864 // (seqs * nq)))
    return {"op": op, "seqs": seqs, "ctx": ctx, "least": round(rng.uniform(0.1, 1.0), 3), "nq": nq, "nq_least": rng.randint(1, nq),
            "dtype": rng.choice(["bf16", "fp16"]), "sel": rng.choice([0, 0, 0, 16]), "mask": rng.random() < 0.7}


def _lengths(case):
    """(context tokens before the drafts, drafts) of each sequence of a tree case."""
    r = random.Random(case["seqs"] * 1000003 + case["ctx"] * 31 + case["nq"])
    ctx = [r.randint(max(1, int(case["ctx"] * case["least"])), case["ctx"]) for _ in range(case["seqs"])]
    if case["least"] == 1.0:
        ctx = [case["ctx"]] * case["seqs"]
    # the first sequence has the most drafts
    return ctx, [case["nq"]] + [r.randint(case["nq_least"], case["nq"]) for _ in range(case["seqs"] - 1)]


# ---- inputs ------------------------------------------------------------------------


def _code_table(device):
    """256 E2M1 codes with the frequencies of normal values scaled to their group's maximum."""
    p = (torch.arange(256, dtype=torch.float64, device=device) + 0.5) / 256
    z = torch.special.ndtri(p) * 2.6
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=device)
    m = torch.bucketize(z.abs(), mids)
    return (m | torch.where((z < 0) & (m > 0), 8, 0)).to(torch.int32)


def _pools(n_pages, g, device):
    """A cache that holds tokens everywhere: normal codes, scales from 8 to 30 (a few zero), index keys ~ N(0, 1)."""
    table = _code_table(device)
    kv = torch.empty((n_pages, PAGE_BYTES), dtype=torch.uint8, device=device)
    idx = torch.empty((n_pages, IDX_BYTES), dtype=torch.uint8, device=device)
    for at in range(0, n_pages, 1024):
        n = min(1024, n_pages - at)
        page = kv[at : at + n].view(n, KV, HEAD_BYTES)
        for codes, scales in OFF.values():
            c = table[torch.randint(0, 256, (8, n * KV * PAGE * 16), generator=g, device=device)]
            w = torch.zeros_like(c[0])
            for i in range(8):
                w |= (c[i] & 7) << (4 * i)
                w |= (c[i] >> 3) << (8 * i + 7 if i < 4 else 8 * (i - 4) + 3)
            page[:, :, codes : codes + 8192] = w.view(torch.uint8).view(n, KV, 8192)
            s = torch.randint(0x50, 0x60, (n, KV, 1024), generator=g, device=device, dtype=torch.uint8)
            s[torch.rand((n, KV, 1024), generator=g, device=device) < 0.002] = 0
            page[:, :, scales : scales + 1024] = s
        idx[at : at + n] = torch.randn((n, IDX_BYTES), generator=g, device=device).to(torch.float8_e4m3fn).view(torch.uint8)
    return kv, idx


def _slots(case, g, device):
    n = case["n"]
    pages = -(-n // PAGE) + 1
    if case["order"] == "scatter":
        slots = torch.randperm(pages * PAGE, generator=g, device=device)[:n]
    else:
        perm = torch.randperm(pages, generator=g, device=device)
        at = torch.arange(n, device=device)
        slots = perm[at // PAGE] * PAGE + at % PAGE
    if case["skip"]:
        slots[torch.randperm(n, generator=g, device=device)[: case["skip"]]] = -1
    return slots.to(torch.int64).contiguous(), pages


def _tree_words(rng, n):
    """One word for each draft: a bit for each draft that it sees (its ancestors and itself)."""
    words = []
    for j in range(n):
        parent = rng.randint(max(0, j - 6), j - 1) if j else -1
        words.append((words[parent] if j else 0) | (1 << j))
    return [w - (1 << 64) if w >> 63 else w for w in words]


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=device)}
    if case["op"] == "tree":
        ctx, nq = _lengths(case)
        rng = random.Random(seed)
        lens = [c + n for c, n in zip(ctx, nq)]
        counts = [-(-n // PAGE) for n in lens]
        total = sum(counts)
        s["kv_pool"], s["idx_pool"] = _pools(total, g, device)
        perm = torch.randperm(total, generator=g, device=device).to(torch.int32).cpu().tolist()
        table, at = [], 0
        for n in counts:
            table.append(perm[at : at + n] + [-1] * (max(counts) - n))
            at += n
        s["block_table"] = torch.tensor(table, dtype=torch.int32, device=device)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
        s["q_start_loc"] = torch.tensor([sum(nq[:b]) for b in range(len(nq) + 1)], dtype=torch.int32, device=device)
        s["most"] = max(nq)
        s["q"] = torch.randn((sum(nq), HEADS, DIM), generator=g, device=device).to(torch.float8_e4m3fn).view(torch.uint8)
        if case["mask"]:
            words = [w for n in nq for w in _tree_words(rng, n)]
            s["tree_mask"] = torch.tensor(words, dtype=torch.int64, device=device)
        if case["sel"]:
            sel, n_sel = [], []
            for c in ctx:
                first = c // PAGE
                some = sorted(rng.sample(range(first), min(case["sel"], first))) + [first]
                sel.append(some + [-1] * (case["sel"] + 1 - len(some)))
                n_sel.append(len(some))
            s["sel"] = torch.tensor(sel, dtype=torch.int32, device=device)
            s["n_sel"] = torch.tensor(n_sel, dtype=torch.int32, device=device)
        return s
    n, dtype = case["n"], TYPES[case["dtype"]]
    s["slots"], pages = _slots(case, g, device)
    back = torch.bfloat16 if case["op"] == "write" and case["dtype"] == "fp32" else dtype  # 4-bit values need no 32 bits
    s["out"] = [torch.zeros((n,) + shape, dtype=back, device=device) for shape in ((KV, DIM), (KV, DIM), (DIM,))]
    s["kv_pool"], s["idx_pool"] = _pools(pages, g, device)
    if case["op"] == "read":
        return s
    heads = (HEADS, KV, KV, 1, IDX_HEADS)
    rows = torch.randn((n, sum(heads), DIM), generator=g, device=device)
    rows *= torch.exp(0.5 * torch.randn((1, sum(heads), DIM), generator=g, device=device)).clamp(0.3, 1.2)
    rows = rows.to(dtype)
    parts = torch.split(rows, heads, dim=1)
    if not case["packed"]:
        parts = [p.contiguous() for p in parts]
    s["q"], s["k"], s["v"], s["idx_k"], s["q_idx"] = parts[0], parts[1], parts[2], parts[3][:, 0], parts[4]
    rot, top = case["rot"], 32768
    s["positions"] = torch.randint(0, top - n, (1,), generator=g, device=device, dtype=torch.int32) + torch.arange(n, device=device, dtype=torch.int32)
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
    angle = torch.arange(top, dtype=torch.float64, device=device)[:, None] * freq
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
    s["q8"] = torch.empty((n, HEADS, DIM), dtype=torch.uint8, device=device)
    s["qi8"] = torch.empty((n, IDX_HEADS, DIM), dtype=torch.uint8, device=device)
    return s


# ---- one pass -------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return {"write": _plain_write, "read": _plain_read, "tree": _plain_tree}[s["case"]["op"]](s)


def _run_own(s):
    from nvfp4_kv_block_gb300 import ops

    case = s["case"]
    if "cache" not in s:  # the handle that a program keeps beside its pools
        s["cache"] = ops.KVCache.from_pools(s["kv_pool"], s["idx_pool"], S_ENC_K, S_ENC_V, s["status"])
    cache = s["cache"]
    if case["op"] == "tree":
        if "bufs" not in s:  # outputs and scratch that a program keeps from step to step
            s["bufs"] = ops.TreeBuffers(s["q"].shape[0], s["seq_lens"].shape[0], TYPES[case["dtype"]])
        out = ops.tree_attn(cache, s["q"], s["block_table"], s["seq_lens"], s["q_start_loc"], s["bufs"],
                            tree_mask=s.get("tree_mask"), sel=s.get("sel"), n_sel=s.get("n_sel"))
        return out, s["bufs"].lse
    if case["op"] == "read":
        return ops.read_kv(cache, s["slots"], k=s["out"][0], v=s["out"][1], idx_k=s["out"][2])
    q8, qi8 = ops.rotary_insert(cache, s["q"], s["k"], s["v"], s["idx_k"], s["cos_sin"], s["positions"], s["slots"],
                                q_idx=s["q_idx"], interleaved=case["inter"], q8=s["q8"], qi8=s["qi8"])
    k, v, idx = ops.read_kv(cache, s["slots"], k=s["out"][0], v=s["out"][1], idx_k=s["out"][2])
    return q8.view(torch.float8_e4m3fn), qi8.view(torch.float8_e4m3fn), k, v, idx


def _to_fp8(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _rotate(x, cos_sin, positions, inter):
    """Rotary positions on the first rot channels of fp32 rows [n, heads, 128]; every product and sum rounded to fp32."""
    half = cos_sin.shape[1] // 2
    cs = cos_sin[positions.long()][:, None]
    c, s = cs[..., :half], cs[..., half:]
    turned = x[..., : 2 * half]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if inter else (turned[..., :half], turned[..., half:])
    first, second = a * c - b * s, b * c + a * s
    both = torch.stack((first, second), -1).flatten(-2) if inter else torch.cat((first, second), -1)
    return torch.cat((both, x[..., 2 * half :]), -1)


def _nvfp4_values(x, s_enc, dec):
    """What a cache with encode scale s_enc holds for fp32 rows: E2M1 codes under an E4M3 scale of each 16 channels."""
    g = x.unflatten(-1, (8, 16))
    a = g.abs().amax(-1, keepdim=True)
    sb = _to_fp8(a / torch.full_like(a, 6.0) * s_enc).float()  # a division: one by a number would be a product
    y = g.abs() * s_enc
    up = [y > 0.25 * sb, y >= 0.75 * sb, y > 1.25 * sb, y >= 1.75 * sb, y > 2.5 * sb, y >= 3.5 * sb, y > 5.0 * sb]
    e = 0.5 * (up[0].float() + up[1] + up[2] + up[3]) + up[4].float() + up[5] + 2.0 * up[6]
    e = torch.where(sb > 0, torch.copysign(e, g), 0.0)
    return (e * (sb * dec)).flatten(-2)


def _kept(new, slots, old):
    """Rows of skipped slots stay as they were."""
    return torch.where((slots >= 0).view((-1,) + (1,) * (old.dim() - 1)), new.to(old.dtype), old)


def _plain_write(s):
    inter, cs, pos = s["case"]["inter"], s["cos_sin"], s["positions"]
    q8 = _to_fp8(_rotate(s["q"].float(), cs, pos, inter))
    qi8 = _to_fp8(_rotate(s["q_idx"].float(), cs, pos, inter))
    k = _nvfp4_values(_rotate(s["k"].float(), cs, pos, inter), S_ENC_K, DEC_K)
    v = _nvfp4_values(s["v"].float(), S_ENC_V, DEC_V)
    idx = _to_fp8(_rotate(s["idx_k"].float()[:, None], cs, pos, inter))[:, 0].float()
    k0, v0, i0 = s["out"]
    return q8, qi8, _kept(k, s["slots"], k0), _kept(v, s["slots"], v0), _kept(idx, s["slots"], i0)


def _unpack(words):
    """E2M1 values (fp32) of code words [..., 16] int32 -> [..., 128]."""
    d = words.device
    at = torch.arange(8, device=d, dtype=torch.int32)
    mag = (words[..., None] >> (4 * at)) & 7
    sign = (words[..., None] >> torch.where(at < 4, 8 * at + 7, 8 * (at - 4) + 3)) & 1
    value = torch.where(mag < 4, mag.float() * 0.5, torch.where(mag < 6, mag.float() - 2.0, 2.0 * mag.float() - 8.0))
    return torch.where(sign == 1, -value, value).flatten(-2)


def _plain_read(s):
    slots = s["slots"]
    safe = slots.clamp(min=0)
    page, t = safe // PAGE, safe % PAGE
    kv = s["kv_pool"].view(-1, KV, HEAD_BYTES)
    place = torch.arange(4, device=slots.device)[None, :] ^ ((t[:, None] >> 1) & 3)  # chunk c of token t
    inside = (t[:, None, None] * 64 + place[:, :, None] * 16 + torch.arange(16, device=slots.device)).flatten(1)  # [n, 64]
    group = torch.arange(8, device=slots.device) * PAGE + t[:, None]  # [n, 8]
    head = torch.arange(KV, device=slots.device)[None, :, None]
    got = []
    for (codes, scales), dec, old in ((OFF["k"], DEC_K, s["out"][0]), (OFF["v"], DEC_V, s["out"][1])):
        words = kv[page[:, None, None], head, codes + inside[:, None]].contiguous().view(torch.int32)
        sb = kv[page[:, None, None], head, scales + group[:, None]].view(torch.float8_e4m3fn).float()
        value = _unpack(words).unflatten(-1, (8, 16)) * (sb * dec)[..., None]
        got.append(_kept(value.flatten(-2), slots, old))
    c = torch.arange(8, device=slots.device)[None, :] ^ (t[:, None] & 7)
    at = (t[:, None, None] * DIM + c[:, :, None] * 16 + torch.arange(16, device=slots.device)).flatten(1)
    idx = s["idx_pool"][page[:, None], at].view(torch.float8_e4m3fn).float()
    return got[0], got[1], _kept(idx, slots, s["out"][2])


def _plain_tree(s):
    """Attention of every draft over its sequence's visited blocks, padded to the longest list."""
    table, lens, start = s["block_table"].long(), s["seq_lens"].long(), s["q_start_loc"].long()
    d, seqs = table.device, table.shape[0]
    nq = start[1:] - start[:-1]
    ctx = lens - nq
    first = ctx // PAGE  # the first block that can hold a draft
    if "sel" in s:
        near = first[:, None] + torch.arange(2, device=d)
        blocks = torch.cat((torch.where((s["sel"] >= 0) & (s["sel"] < first[:, None]), s["sel"].long(), -1), near), 1)
    else:
        blocks = torch.arange(table.shape[1], device=d).expand(seqs, -1)
    blocks = torch.where(blocks * PAGE < lens[:, None], blocks, -1)
    place = (blocks[:, :, None] * PAGE + torch.arange(PAGE, device=d)).flatten(1)  # position of each key
    place = torch.where((blocks >= 0).repeat_interleave(PAGE, 1), place, -1)
    pages = torch.gather(table, 1, blocks.clamp(min=0)).clamp(min=0)
    kv = s["kv_pool"].view(-1, KV, HEAD_BYTES)
    tok = torch.arange(PAGE, device=d)[:, None]
    order = tok * 4 + (torch.arange(4, device=d)[None, :] ^ ((tok >> 1) & 3))  # chunk c of token t
    operand = []
    for codes, scales in OFF.values():
        words = kv[:, :, codes : codes + 8192].contiguous().view(torch.int32).view(-1, KV, PAGE * 4, 4)[pages]
        words = words[:, :, :, order.flatten()].view(words.shape[:3] + (PAGE, 16))
        sb = kv[:, :, scales : scales + 1024][pages].view(torch.float8_e4m3fn).float()
        sb = sb.view(sb.shape[:3] + (8, PAGE)).transpose(-1, -2)
        x = _to_fp8(_unpack(words).unflatten(-1, (8, 16)) * sb[..., None]).float()
        operand.append(x.flatten(-2).permute(0, 2, 1, 3, 4).flatten(2, 3))  # [B, 4, keys, 128]
    k, v = operand
    v = torch.where((place >= 0) & (place < lens[:, None]), 1.0, 0.0)[:, None, :, None] * v
    most = s["most"]
    row = start[:-1, None] + torch.arange(most, device=d)  # [B, most] draft rows
    there = torch.arange(most, device=d) < nq[:, None]
    row = torch.where(there, row, 0)
    q = s["q"].view(torch.float8_e4m3fn).float()[row].view(seqs, most, KV, HEADS // KV, DIM).permute(0, 2, 1, 3, 4).flatten(2, 3)
    bit = place[:, None, :] - ctx[:, None, None]  # which draft a key is
    if "tree_mask" in s:
        sees = (s["tree_mask"][row][:, :, None] >> bit.clamp(0, 63)) & 1 == 1
    else:
        sees = bit <= torch.arange(most, device=d)[None, :, None]
    sees = (bit < 0) | (sees & (bit < nq[:, None, None]))
    sees = sees & (place >= 0)[:, None, :]
    logits = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(DIM) / S_ENC_K)
    logits.masked_fill_(~sees[:, None].repeat_interleave(HEADS // KV, 2), -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logits.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0) / S_ENC_V
    lse = (top + total.log()).squeeze(-1)
    o = o.view(seqs, KV, most, HEADS // KV, DIM).permute(0, 2, 1, 3, 4).flatten(2, 3)[there]
    lse = lse.view(seqs, KV, most, HEADS // KV).permute(0, 2, 1, 3).flatten(2, 3)[there]
    return o.to(TYPES[s["case"]["dtype"]]), lse


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    if case["op"] == "tree":
        ctx, nq = _lengths(case)
        size = 0.0
        flops = 0.0
        for c, n in zip(ctx, nq):
            keys = min(c // PAGE, case["sel"]) * PAGE + c % PAGE if case["sel"] else c
            size += 576.0 * (keys + n) + n * HEADS * DIM * 3 + n * HEADS * 4 + 4 * (keys // PAGE + 1)
            flops += 4.0 * HEADS * DIM * (n * keys + n * (n + 1) / 2)
        return {"bytes": size, "flops": flops}
    n, width = case["n"], 4 if case["dtype"] == "fp32" else 2
    live = n - case["skip"]
    back = live * (704 + (2 * KV + 1) * DIM * (2 if case["op"] == "write" else width)) + 8 * n  # cache bytes in, values out
    if case["op"] == "read":
        return {"bytes": float(back), "flops": float(live * (2 * KV + 1) * DIM)}
    rows = HEADS + 2 * KV + 1 + IDX_HEADS
    size = n * (rows * DIM * width + 12 + case["rot"] * 4 + (HEADS + IDX_HEADS) * DIM) + live * 704
    return {"bytes": float(size + back), "flops": float(n * (rows - KV) * case["rot"] * 3 + live * 2 * KV * DIM * 4)}


# ---- the definitions in 64 bits -------------------------------------------------------------


def _fp8_table():
    """Values of the 256 E4M3 bytes, from their bit fields."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0**-6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return torch.from_numpy(np.where(b & 128, -v, v)).cuda()


def _nearest(x, grid):
    """Each value of x >= 0 moved to the nearest of the ascending grid; ties to the even place."""
    mids = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(x, mids), torch.bucketize(x, mids, right=True)
    return grid[torch.where((below != above) & (below % 2 == 1), above, below)]


def _exact_fp8(x):
    return torch.copysign(_nearest(x.abs().contiguous(), _fp8_table()[:127]), x)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_turn(x, table, inter):
    """Pairs as complex numbers times e^(i angle)."""
    half = table.shape[1] // 2
    if not half:
        return x
    z = torch.complex(table[:, :half], table[:, half:])[:, None]
    w = x[..., : 2 * half]
    w = torch.view_as_complex(w.unflatten(-1, (half, 2)).contiguous()) if inter else torch.complex(w[..., :half].contiguous(), w[..., half:].contiguous())
    w = w * z
    w = torch.view_as_real(w).flatten(-2) if inter else torch.cat((w.real, w.imag), -1)
    return torch.cat((w, x[..., 2 * half :]), -1)


def _exact_cached(x, s_enc):
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    blocks = x.reshape(-1, 16)
    scale = _exact_fp8(blocks.abs().max(1).values / 6 * s_enc)[:, None]
    r = torch.where(scale > 0, blocks.abs() * s_enc / torch.where(scale > 0, scale, 1.0), 0.0)
    return (torch.copysign(_nearest(r.contiguous(), grid), blocks) * scale / s_enc).view(x.shape)


def _exact_rows(pool, slots, codes, scales, fp8):
    """e2m1 * scale of the tokens at `slots` for every head [n, 4, 128], byte by byte from the page format."""
    d = pool.device
    page, t = slots // PAGE, slots % PAGE
    ch = torch.arange(DIM, device=d)
    word, n = ch // 8, ch % 8
    row = (t[:, None] * 64 + (((word // 4)[None] ^ ((t[:, None] // 2) % 4)) * 16) + (word % 4)[None] * 4)  # first byte of the word
    flat = pool.view(-1)
    base = (page[:, None] * PAGE_BYTES + torch.arange(KV, device=d) * HEAD_BYTES)[:, :, None]
    mag = flat[base + codes + (row + (n // 2)[None])[:, None]].long() >> (4 * (n % 2)) & 7
    sgn = flat[base + codes + (row + (n % 4)[None])[:, None]].long() >> torch.where(n < 4, 7, 3) & 1
    sb = _fp8_table()[flat[base + scales + ((ch // 16) * PAGE + t[:, None])[:, None]].long()]
    v = torch.tensor(_E2M1, dtype=torch.float64, device=d)[mag] * sb
    if fp8:
        v = _exact_fp8(v)
    return torch.where(sgn == 1, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    f8 = _fp8_table()
    if case["op"] == "tree":
        return _exact_tree(s)
    live = s["slots"] >= 0
    if case["op"] == "read":
        at = s["slots"].clamp(min=0)
        k = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["k"], False) for a in at.split(16384)]) / S_ENC_K
        v = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["v"], False) for a in at.split(16384)]) / S_ENC_V
        t = (at % PAGE)[:, None]
        ch = torch.arange(DIM, device=at.device)
        idx = f8[s["idx_pool"].view(-1)[(at // PAGE)[:, None] * IDX_BYTES + t * DIM + ((ch // 16) ^ (t % 8)) * 16 + ch % 16].long()]
        return k * live[:, None, None], v * live[:, None, None], idx * live[:, None]
    table = s["cos_sin"].double()[s["positions"].long()]
    inter = case["inter"]
    q, qi = (_exact_fp8(_exact_turn(s[name].double(), table, inter)) for name in ("q", "q_idx"))
    k = _exact_cached(_exact_turn(s["k"].double(), table, inter), S_ENC_K) * live[:, None, None]
    v = _exact_cached(s["v"].double(), S_ENC_V) * live[:, None, None]
    idx = _exact_fp8(_exact_turn(s["idx_k"].double()[:, None], table, inter))[:, 0] * live[:, None]
    return q, qi, k, v, idx


def _exact_tree(s):
    """Sequence by sequence, KV head by KV head."""
    f8 = _fp8_table()
    lens, start = s["seq_lens"].tolist(), s["q_start_loc"].tolist()
    out, lse = [], []
    for b, total in enumerate(lens):
        n = start[b + 1] - start[b]
        ctx = total - n
        at = torch.arange(total, device="cuda")
        if "sel" in s:
            chosen = set(s["sel"][b, : int(s["n_sel"][b])].tolist())
            blk = (at // PAGE).tolist()
            at = at[torch.tensor([x in chosen or x >= ctx // PAGE for x in blk], device="cuda")]
        slots = s["block_table"][b].long()[at // PAGE] * PAGE + at % PAGE
        k = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["k"], True) for a in slots.split(16384)]) / S_ENC_K
        v = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["v"], True) for a in slots.split(16384)]) / S_ENC_V
        q = f8[s["q"][start[b] : start[b + 1]].long()]
        hidden = torch.zeros((n, at.numel()), dtype=torch.bool, device="cuda")
        words = s["tree_mask"][start[b] : start[b + 1]].tolist() if "tree_mask" in s else [(2 << j) - 1 for j in range(n)]
        for key, draft in enumerate((at - ctx).tolist()[-n:]):
            assert draft == key
            hidden[:, at.numel() - n + key] = torch.tensor([not (w >> draft) & 1 for w in words], device="cuda")
        o, l = [], []
        for h in range(HEADS):
            z = (q[:, h] @ k[:, h // 4].T) / DIM**0.5
            z[hidden] = -math.inf
            l.append(torch.logsumexp(z, 1))
            o.append(torch.softmax(z, 1) @ v[:, h // 4])
        out.append(torch.stack(o, 1))
        lse.append(torch.stack(l, 1))
    return torch.cat(out), torch.cat(lse)
