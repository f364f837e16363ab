"""Measured cases of the operators around a prompt in the paged NVFP4 cache.

Each in a plain form (``own`` false: elementary torch operations in 32 bits) and
through the library (``own`` true):

  * axes: rotary positions with several axes (time, height, width of images and
    video) on projected rows, FP8 queries and index queries, the cache write, and
    the values that the cache now holds;
  * prefill: attention of a prompt's tokens, any number a sequence, over the whole
    cached context: causal, within a window, or up to an end of each token's own
    (tokens of an image see all of it);
  * branch: sequences released, forked (full pages shared, the last one copied) and
    given pages for new tokens, with reference counts and the lowest free pages first;
  * commit: the accepted drafts of each sequence moved together behind its context,
    in every layer's pools.

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
        # one small image of 16 x 16 patches and a few words: latency
        {"name": "axes_image_267", "op": "axes", "n": 267, "dtype": "bf16", "sections": "16,24,24", "dealt": False, "inter": False, "packed": False, "skip": 0},
        # a chunk of video frames, axes dealt to the pairs in turn, rows as slices of one projection, some not inserted
        {"name": "axes_video_8185", "op": "axes", "n": 8185, "dtype": "fp16", "sections": "24,20,20", "dealt": True, "inter": False, "packed": True, "skip": 25},
        # a short first prompt: latency
        {"name": "prefill_short_100", "op": "prefill", "seqs": 1, "nq": 100, "nq_least": 100, "ctx": 0, "ctx_least": 0, "window": 0, "image": 0, "dtype": "bf16"},
        # a whole prompt from its beginning
        {"name": "prefill_prompt_8192", "op": "prefill", "seqs": 1, "nq": 8192, "nq_least": 8192, "ctx": 0, "ctx_least": 0, "window": 0, "image": 0, "dtype": "bf16"},
        # chunks of several prompts in one step, each at its own place
        {"name": "prefill_ragged_9x30720", "op": "prefill", "seqs": 9, "nq": 1500, "nq_least": 1, "ctx": 30720, "ctx_least": 0, "window": 0, "image": 0, "dtype": "fp16"},
        # a layer with a sliding window
        {"name": "prefill_window_4096", "op": "prefill", "seqs": 1, "nq": 4096, "nq_least": 4096, "ctx": 30720, "ctx_least": 30720, "window": 4096, "image": 0, "dtype": "bf16"},
        # prompts with images whose tokens see all of their image, and padding tokens
        {"name": "prefill_images_4x1777", "op": "prefill", "seqs": 4, "nq": 1777, "nq_least": 900, "ctx": 4096, "ctx_least": 0, "window": 0, "image": 577, "dtype": "bf16"},
        # a chunk at the end of a long context
        {"name": "prefill_long_2048x131072", "op": "prefill", "seqs": 1, "nq": 2048, "nq_least": 2048, "ctx": 131072, "ctx_least": 131072, "window": 0, "image": 0, "dtype": "bf16"},
        # four continuations of one prompt, one layer: latency
        {"name": "branch_4_of_1", "op": "branch", "prompts": 1, "each": 4, "len": 1000, "len_least": 1000, "new": 1, "layers": 1},
        # many continuations of many prompts in several layers
        {"name": "branch_256_of_16", "op": "branch", "prompts": 16, "each": 16, "len": 4096, "len_least": 100, "new": 8, "layers": 12},
        # the accepted drafts of a small batch, one layer: latency
        {"name": "commit_8x8", "op": "commit", "seqs": 8, "drafts": 8, "drafts_least": 8, "ctx": 1000, "layers": 1},
        # wide trees of a large batch in several layers
        {"name": "commit_64x64_12", "op": "commit", "seqs": 64, "drafts": 64, "drafts_least": 20, "ctx": 500, "layers": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "prefill", "prefill", "prefill", "branch", "commit"])
    if op == "axes":
        n = _log_int(rng, 1, 16384)
        half = 8 * rng.randint(1, 8)
        cut = sorted(rng.randint(0, half) for _ in range(rng.randint(1, 3)))
        sections = [b - a for a, b in zip([0] + cut, cut + [half])]
        return {"op": op, "n": n, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "sections": ",".join(map(str, sections)), "dealt": rng.random() < 0.5,
                "inter": rng.random() < 0.5, "packed": rng.random() < 0.5, "skip": rng.choice([0, n // 8])}
    if op == "prefill":
        seqs = _log_int(rng, 1, 16)
        nq = _log_int(rng, 1, 8192 // seqs)
        ctx = _log_int(rng, 1, min(131072 // seqs, 268435456 // (seqs * nq) - nq))
        image = rng.choice([0, 0, rng.randint(2, 700)])
        return {"op": op, "seqs": seqs, "nq": nq, "nq_least": rng.randint(1, nq), "ctx": ctx, "ctx_least": rng.choice([0, ctx, ctx // 2]),
                "window": 0 if image else rng.choice([0, 0, _log_int(rng, 1, 8192)]), "image": image, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "branch":
        prompts, each = _log_int(rng, 1, 16), _log_int(rng, 1, 16)
        size = _log_int(rng, 1, 4096)
        return {"op": op, "prompts": prompts, "each": each, "len": size, "len_least": rng.randint(1, size), "new": _log_int(rng, 1, 64), "layers": rng.randint(1, 12)}
    drafts = rng.randint(1, 64)
    return {"op": op, "seqs": _log_int(rng, 1, 64), "drafts": drafts, "drafts_least": rng.randint(0, drafts), "ctx": _log_int(rng, 1, 1000), "layers": rng.randint(1, 12)}


def _spread(r, least, most, count):
    """`count` numbers from `least` to `most`; the first is the largest."""
    return [most] + [r.randint(least, most) for _ in range(count - 1)]


def _prefill_sizes(case):
    """(context tokens before the new ones, new tokens) of each sequence; of five and more one has no new token and one a single one."""
    r = random.Random(case["seqs"] * 1000003 + case["ctx"] * 31 + case["nq"])
    nq = _spread(r, case["nq_least"], case["nq"], case["seqs"])
    ctx = _spread(r, case["ctx_least"], case["ctx"], case["seqs"])
    if len(nq) >= 5:
        nq[2], nq[4] = 0, 1
    r.shuffle(ctx)
    return ctx, nq


def _branch_sizes(case):
    """Length of each prompt, its branches, and the new tokens of each branch."""
    r = random.Random(case["prompts"] * 1000003 + case["len"] * 31 + case["each"])
    lens = _spread(r, case["len_least"], case["len"], case["prompts"])
    new = [r.randint(1, case["new"]) for _ in range(case["prompts"] * case["each"])]
    return lens, new


def _commit_sizes(case):
    r = random.Random(case["seqs"] * 1000003 + case["ctx"] * 31 + case["drafts"])
    return _spread(r, (case["ctx"] + 1) // 2, case["ctx"], case["seqs"]), _spread(r, case["drafts_least"], case["drafts"], case["seqs"])


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


def _axis_of_pair(case):
    """Axis of each pair: the sections one after another, or dealt in turn while an axis has pairs left (what stays goes to the first)."""
    sections = [int(x) for x in case["sections"].split(",")]
    if not case["dealt"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    m = len(sections)
    return [i % m if i < m * sections[i % m] else 0 for i in range(sum(sections))]


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rng = random.Random(seed)
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=device)}
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=device)  # noqa: E731
    return {"axes": _prepare_axes, "prefill": _prepare_prefill, "branch": _prepare_branch, "commit": _prepare_commit}[case["op"]](case, s, g, rng, device, ints)


def _prepare_axes(case, s, g, rng, device, ints):
    n, dtype = case["n"], TYPES[case["dtype"]]
    pages = -(-n // PAGE) + 1
    perm = torch.randperm(pages, generator=g, device=device)
    at = torch.arange(n, device=device)
    slots = perm[at // PAGE] * PAGE + at % PAGE
    if case["skip"]:
        slots[torch.randperm(n, generator=g, device=device)[: case["skip"]]] = -1
    s["slots"] = slots.to(torch.int64).contiguous()
    heads = (HEADS, KV, KV, 1, IDX_HEADS)
    rows = torch.randn((n, sum(heads), DIM), generator=g, device=device)
    rows *= torch.exp(0.5 * torch.randn((1, sum(heads), DIM), generator=g, device=device)).clamp(0.3, 1.2)
    rows = rows.to(dtype)
    parts = torch.split(rows, heads, dim=1)
    if not case["packed"]:
        parts = [p.contiguous() for p in parts]
    s["q"], s["k"], s["v"], s["idx_k"], s["q_idx"] = parts[0], parts[1], parts[2], parts[3][:, 0], parts[4]
    axes = _axis_of_pair(case)
    m, rot, top = len(case["sections"].split(",")), 2 * len(axes), 65536
    # words count every axis alike; the patches of a frame are a grid at one time
    base = rng.randint(0, top - 2 * n - 2)
    frame, width = 24 * 24, 24
    place = [at // frame] + [(at % frame) // width, at % width, at % 7][: m - 1]
    text = at % (frame + 11) < 11
    s["positions"] = torch.stack([(base + torch.where(text, at, p)).to(torch.int32) for p in place[:m]]).contiguous()
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(top, dtype=torch.float64, device=device)[:, None] * freq
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
    s["axis"] = ints(axes, torch.int64)
    s["kv_pool"], s["idx_pool"] = _pools(pages, g, device)
    back = torch.bfloat16 if case["dtype"] == "fp32" else dtype  # 4-bit values need no 32 bits
    s["out"] = [torch.zeros((n,) + shape, dtype=back, device=device) for shape in ((KV, DIM), (KV, DIM), (DIM,))]
    s["q8"] = torch.empty((n, HEADS, DIM), dtype=torch.uint8, device=device)
    s["qi8"] = torch.empty((n, IDX_HEADS, DIM), dtype=torch.uint8, device=device)
    return s


def _prepare_prefill(case, s, g, rng, device, ints):
    ctx, nq = _prefill_sizes(case)
    lens = [c + n for c, n in zip(ctx, nq)]
    counts = [-(-n // PAGE) for n in lens]
    total = sum(counts)
    s["kv_pool"], s["idx_pool"] = _pools(total, g, device)
    perm = torch.randperm(total, generator=g, device=device).to(torch.int32).cpu().tolist()
    table, at = [], 0
    for n in counts:
        table.append(perm[at : at + n] + [-1] * (max(counts) - n))
        at += n
    s["pages"] = total
    s["block_table"], s["seq_lens"] = ints(table), ints(lens)
    s["starts"] = [sum(nq[:b]) for b in range(len(nq) + 1)]
    s["q_start_loc"] = ints(s["starts"])
    s["q"] = torch.randn((sum(nq), HEADS, DIM), generator=g, device=device).to(torch.float8_e4m3fn).view(torch.uint8)
    if case["image"]:
        ends = []
        for c, n in zip(ctx, nq):
            i = 0
            while i < n:
                words = min(rng.randint(1, 200), n - i)
                ends += [c + i + 1 + j if rng.random() > 0.01 else 0 for j in range(words)]  # 0: padding, sees nothing
                i += words
                span = min(case["image"], n - i)
                ends += [c + i + span] * span
                i += span
        s["ends"] = ints(ends)
    return s


def _layers(case, pages, g, device):
    kv = torch.randint(0, 256, (case["layers"], pages, PAGE_BYTES), generator=g, device=device, dtype=torch.uint8)
    idx = torch.randint(0, 256, (case["layers"], pages, IDX_BYTES), generator=g, device=device, dtype=torch.uint8)
    return kv, idx


def _prepare_branch(case, s, g, rng, device, ints):
    lens, new = _branch_sizes(case)
    counts = [-(-n // PAGE) for n in lens]
    rows = len(lens) + len(new)
    fresh = sum(-(-(lens[i // case["each"]] % PAGE + n) // PAGE) for i, n in enumerate(new))
    pages = sum(counts) + fresh + 16
    wide = max(counts) + 2
    perm = torch.randperm(pages, generator=g, device=device).tolist()
    table, at = [], 0
    for n in counts:
        table.append(perm[at : at + n] + [-1] * (wide - n))
        at += n
    refs = [0] * pages
    for p in perm[:at]:
        refs[p] = 1
    s["block_table"] = ints(table + [[-1] * wide for _ in new])
    s["seq_lens"] = ints(lens + [0] * len(new))
    s["refs"] = ints(refs)
    s["src"] = ints([i // case["each"] for i in range(len(new))])
    s["dst"] = ints([len(lens) + i for i in range(len(new))])
    s["starts"] = [0] * len(lens) + [sum(new[:i]) for i in range(len(new) + 1)]
    s["q_start_loc"] = ints(s["starts"])
    s["new"] = s["starts"][-1]
    s["kv"], s["idx"] = _layers(case, pages, g, device)
    s["rows"] = rows
    return s


def _prepare_commit(case, s, g, rng, device, ints):
    ctx, drafts = _commit_sizes(case)
    lens = [c + n for c, n in zip(ctx, drafts)]
    counts = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(counts), generator=g, device=device).tolist()
    table, at = [], 0
    for n in counts:
        table.append(perm[at : at + n] + [-1] * (max(counts) - n))
        at += n
    s["block_table"], s["seq_lens"] = ints(table), ints(lens)
    s["q_start_loc"] = ints([sum(drafts[:b]) for b in range(len(drafts) + 1)])
    words = []
    for n in drafts:  # a path from the root: each accepted draft's next one is among the following
        w, j = 0, 0
        while j < n and rng.random() < 0.9:
            w |= 1 << j
            j += rng.randint(1, max(1, n // 8))
        words.append(w - (1 << 64) if w >> 63 else w)
    s["accepted"] = ints(words, torch.int64)
    s["new_lens"] = torch.zeros_like(s["seq_lens"])
    s["most"] = max(drafts)
    s["kv"], s["idx"] = _layers(case, sum(counts), g, device)
    return s


# ---- one pass -------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"axes": _own_axes, "prefill": _own_prefill, "branch": _own_branch, "commit": _own_commit}[op](s)
    return {"axes": _plain_axes, "prefill": _plain_prefill, "branch": _plain_branch, "commit": _plain_commit}[op](s)


def _own_axes(s):
    from nvfp4_kv_block_gb300 import ops

    case = s["case"]
    if "cache" not in s:  # the handles that a program keeps beside its pools
        s["cache"] = ops.KVCache.from_pools(s["kv_pool"], s["idx_pool"], S_ENC_K, S_ENC_V, s["status"])
        s["axes"] = ops.rope_axes([int(x) for x in case["sections"].split(",")], dealt=case["dealt"])
    q8, qi8 = ops.rotary_insert(s["cache"], s["q"], s["k"], s["v"], s["idx_k"], s["cos_sin"], s["positions"], s["slots"],
                                q_idx=s["q_idx"], interleaved=case["inter"], q8=s["q8"], qi8=s["qi8"], axes=s["axes"])
    k, v, idx = ops.read_kv(s["cache"], s["slots"], k=s["out"][0], v=s["out"][1], idx_k=s["out"][2])
    return q8.view(torch.float8_e4m3fn), qi8.view(torch.float8_e4m3fn), k, v, idx


def _own_prefill(s):
    from nvfp4_kv_block_gb300 import ops

    case = s["case"]
    if "cache" not in s:
        s["cache"] = ops.KVCache.from_pools(s["kv_pool"], s["idx_pool"], S_ENC_K, S_ENC_V, s["status"])
        s["bufs"] = ops.PrefillBuffers(s["q"].shape[0], s["seq_lens"].shape[0], s["pages"], TYPES[case["dtype"]])
    out = ops.prefill_attn(s["cache"], s["q"], s["block_table"], s["seq_lens"], s["q_start_loc"], s["bufs"],
                           window=case["window"], ends=s.get("ends"))
    return out, s["bufs"].lse


def _caches(s, ops):
    return [ops.KVCache.from_pools(kv, idx, S_ENC_K, S_ENC_V, s["status"]) for kv, idx in zip(s["kv"], s["idx"])]


def _own_branch(s):
    from nvfp4_kv_block_gb300 import ops

    if "pool" not in s:
        s["layers"] = ops.CacheLayers(_caches(s, ops))
        s["pool"] = ops.PagePool.from_refs(s["refs"], s["status"])
        s["slots"] = torch.empty(s["new"], dtype=torch.int64, device="cuda")
    ops.release_sequences(s["pool"], s["block_table"], s["seq_lens"], s["dst"])
    ops.fork_sequences(s["layers"], s["pool"], s["block_table"], s["seq_lens"], s["src"], s["dst"])
    slots = ops.extend_sequences(s["pool"], s["block_table"], s["seq_lens"], s["q_start_loc"], s["slots"])
    return s["block_table"], s["seq_lens"], s["refs"], slots, s["kv"], s["idx"]


def _own_commit(s):
    from nvfp4_kv_block_gb300 import ops

    if "layers" not in s:
        s["layers"] = ops.CacheLayers(_caches(s, ops))
    new_lens = ops.commit_drafts(s["layers"], s["block_table"], s["seq_lens"], s["q_start_loc"], s["accepted"], s["new_lens"])
    return new_lens, s["kv"], s["idx"]


# ---- plain forms ------------------------------------------------------------------------


def _to_fp8(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _rotate(x, c, s, inter):
    """Rotary positions on the first channels of fp32 rows [n, heads, 128] by c and s [n, pairs]; every product and sum rounded to fp32."""
    half = c.shape[1]
    c, s = c[:, None], s[:, None]
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


def _plain_axes(s):
    inter, table = s["case"]["inter"], s["cos_sin"]
    half = table.shape[1] // 2
    pos = s["positions"].long()[s["axis"]].T  # [n, pairs]: each pair's own position
    pair = torch.arange(half, device=table.device)
    c, t = table[pos, pair], table[pos, half + pair]
    q8 = _to_fp8(_rotate(s["q"].float(), c, t, inter))
    qi8 = _to_fp8(_rotate(s["q_idx"].float(), c, t, inter))
    k = _nvfp4_values(_rotate(s["k"].float(), c, t, inter), S_ENC_K, DEC_K)
    v = _nvfp4_values(s["v"].float(), S_ENC_V, DEC_V)
    idx = _to_fp8(_rotate(s["idx_k"].float()[:, None], c, t, inter))[:, 0].float()
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


def _plain_prefill(s):
    """Sequence by sequence: all keys of its pages, all of its rows at once."""
    case, d = s["case"], s["q"].device
    kv = s["kv_pool"].view(-1, KV, HEAD_BYTES)
    tok = torch.arange(PAGE, device=d)[:, None]
    order = (tok * 4 + (torch.arange(4, device=d)[None, :] ^ ((tok >> 1) & 3))).flatten()  # chunk c of token t
    ctx, nq = _prefill_sizes(case)
    q8 = s["q"].view(torch.float8_e4m3fn)
    out, lse = [], []
    for b, (before, n) in enumerate(zip(ctx, nq)):
        if not n:
            continue
        total = before + n
        pages = s["block_table"][b, : -(-total // PAGE)].long()
        operand = []
        for codes, scales in OFF.values():
            words = kv[:, :, codes : codes + 8192].contiguous().view(torch.int32).view(-1, KV, PAGE * 4, 4)[pages]
            words = words[:, :, order].view(-1, KV, PAGE, 16)
            sb = kv[:, :, scales : scales + 1024][pages].view(torch.float8_e4m3fn).float()
            sb = sb.view(-1, KV, 8, PAGE).transpose(-1, -2)
            x = _to_fp8(_unpack(words).unflatten(-1, (8, 16)) * sb[..., None]).float()
            operand.append(x.flatten(-2).transpose(0, 1).flatten(1, 2)[:, :total])  # [4, keys, 128]
        k, v = operand
        rows = slice(s["starts"][b], s["starts"][b + 1])
        q = q8[rows].float().view(n, KV, HEADS // KV, DIM).permute(1, 0, 2, 3).flatten(1, 2)  # [4, 4 n, 128]
        at = torch.arange(total, device=d)
        pos = before + torch.arange(n, device=d)
        end = s["ends"][rows] if "ends" in s else pos + 1
        hidden = at[None, :] >= end[:, None]
        if case["window"]:
            hidden |= at[None, :] <= pos[:, None] - case["window"]
        logits = torch.matmul(q, k.transpose(-1, -2)).view(KV, n, HEADS // KV, total)
        logits *= 1.0 / math.sqrt(DIM) / S_ENC_K
        logits.masked_fill_(hidden[None, :, None], -math.inf)
        top = logits.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = logits.sub_(top).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v).view(KV, n, HEADS // KV, DIM) / torch.where(l > 0, l, 1.0) / S_ENC_V
        out.append(o.permute(1, 0, 2, 3).flatten(1, 2))
        lse.append((top + l.log()).squeeze(-1).permute(1, 0, 2).flatten(1, 2))
    return torch.cat(out).to(TYPES[case["dtype"]]), torch.cat(lse)


def _first_free(refs):
    """Page of each rank among the free ones (the others' entries are none)."""
    free = refs == 0
    rank = torch.where(free, torch.cumsum(free, 0) - 1, refs.numel())
    pages = torch.full((refs.numel() + 1,), -1, dtype=torch.int64, device=refs.device)
    return pages.scatter_(0, rank, torch.arange(refs.numel(), device=refs.device))


def _count(refs, pages, by):
    """by added to the count of every page of the list that is one."""
    there = pages >= 0
    refs.scatter_add_(0, pages.clamp(min=0).long().flatten(), torch.where(there, by, 0).to(refs.dtype).flatten())


def _token_of_byte(device):
    """The token that each byte of a KV page and of an index page belongs to."""
    at = torch.arange(HEAD_BYTES // 2, device=device)
    half = torch.where(at < 8192, at // 64, (at - 8192) % PAGE)
    return half.repeat(2 * KV), torch.arange(IDX_BYTES, device=device) // DIM


def _plain_branch(s):
    table, lens, refs = s["block_table"], s["seq_lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    d, wide = table.device, table.shape[1]
    col = torch.arange(wide, device=d)
    # the branches' pages go back
    _count(refs, table[dst], -1)
    table[dst] = -1
    lens[dst] = 0
    # full pages are shared, the rest of a prompt gets a page of its own
    size = lens[src]
    full, rest = (size // PAGE).long(), size % PAGE
    pages = _first_free(refs)
    rank = torch.cumsum(rest > 0, 0) - 1
    own_page = torch.where(rest > 0, pages[rank.clamp(min=0)], -1).to(torch.int32)
    last = table[src, full.clamp(max=wide - 1)]
    rows = torch.where(col[None, :] < full[:, None], table[src], torch.where(col[None, :] == full[:, None], own_page[:, None], -1))
    _count(refs, rows, 1)
    table[dst] = rows
    lens[dst] = size
    # (a prompt without a rest writes its first page to where it is)
    fro = torch.where(rest > 0, last, table[src, 0]).long()
    to = torch.where(rest > 0, own_page, table[src, 0]).long()
    for pool, of in zip((s["kv"], s["idx"]), _token_of_byte(d)):
        pool[:, to] = torch.where((of[None, :] < rest[:, None])[None], pool[:, fro], pool[:, to])
    # pages and slots of the new tokens
    start = s["q_start_loc"].long()
    n = start[1:] - start[:-1]
    now = lens.long()
    need = (col[None, :] * PAGE < (now + n)[:, None]) & (col[None, :] * PAGE >= now[:, None]) & (table < 0) & (n > 0)[:, None]
    pages = _first_free(refs)
    rank = torch.cumsum(need.flatten(), 0) - 1
    got = torch.where(need.flatten(), pages[rank.clamp(min=0)], -1).view(need.shape)
    _count(refs, got, 1)
    table.copy_(torch.where(need, got.to(torch.int32), table))
    row = torch.repeat_interleave(torch.arange(n.numel(), device=d), n, output_size=s["new"])
    place = now[row] + torch.arange(s["new"], device=d) - start[row]
    slots = table[row, place // PAGE].long() * PAGE + place % PAGE
    lens += n.to(torch.int32)
    return table, lens, refs, slots, s["kv"], s["idx"]


def _token_bytes(slots, device):
    """(page, byte offsets) of the KV bytes of tokens at `slots` [n], channel order: [n, 4 * 144], and of their index keys [n, 128]."""
    page, t = slots // PAGE, slots % PAGE
    chunk = torch.arange(4, device=device)[None, :] ^ ((t[:, None] >> 1) & 3)
    code = (t[:, None, None] * 64 + chunk[:, :, None] * 16 + torch.arange(16, device=device)).flatten(1)
    scale = 8192 + torch.arange(8, device=device) * PAGE + t[:, None]
    half = torch.cat((code, scale), 1)
    head = torch.cat((half, half + HEAD_BYTES // 2), 1)
    kv = (torch.arange(KV, device=device)[None, :, None] * HEAD_BYTES + head[:, None]).flatten(1)
    c = torch.arange(8, device=device)[None, :] ^ (t[:, None] & 7)
    idx = (t[:, None, None] * DIM + c[:, :, None] * 16 + torch.arange(16, device=device)).flatten(1)
    return page, kv, idx


def _plain_commit(s):
    table, lens, start = s["block_table"].long(), s["seq_lens"].long(), s["q_start_loc"].long()
    d, most = table.device, s["most"]
    n = start[1:] - start[:-1]
    j = torch.arange(most, device=d)
    keep = ((s["accepted"][:, None] >> j) & 1 == 1) & (j < n[:, None])
    rank = torch.cumsum(keep, 1) - 1
    ctx = (lens - n)[:, None]
    there = j < n[:, None]
    src = torch.where(there, ctx + j, 0)
    dst = torch.where(keep, ctx + rank, 0)
    slot = lambda p: (torch.gather(table, 1, p // PAGE) * PAGE + p % PAGE).flatten()  # noqa: E731
    a, b = slot(src), slot(dst)
    # the pairs that are none write the sequence's first token to where it is
    a = torch.where(keep.flatten(), a, (table[:, :1] * PAGE).expand(-1, most).flatten())
    b = torch.where(keep.flatten(), b, a)
    pa, ka, ia = _token_bytes(a, d)
    pb, kb, ib = _token_bytes(b, d)
    s["kv"][:, pb[:, None], kb] = s["kv"][:, pa[:, None], ka]
    s["idx"][:, pb[:, None], ib] = s["idx"][:, pa[:, None], ia]
    s["new_lens"].copy_((ctx[:, 0] + keep.sum(1)).to(torch.int32))
    return s["new_lens"], s["kv"], s["idx"]


# ---- what a pass cannot do without -------------------------------------------------------


def _visible(case):
    """Visible keys over all rows (an average where images are drawn), and tokens that some row of their sequence sees."""
    ctx, nq = _prefill_sizes(case)
    pairs = keys = 0.0
    for c, n in zip(ctx, nq):
        if not n:
            continue
        first = max(0, c + 1 - case["window"]) if case["window"] else 0
        keys += c + n - first
        if case["window"]:
            w = case["window"]
            short = max(0, min(n, w - c))  # rows whose window reaches the beginning
            pairs += short * c + short * (short + 1) / 2 + (n - short) * w
        else:
            pairs += n * c + n * (n + 1) / 2
            if case["image"]:  # half a span more for the tokens of images, most of them
                span = min(case["image"], max(0, n - 100))
                pairs += n * span / (span + 100.0) * span / 2
    return pairs, keys, sum(nq)


def work(case):
    if case["op"] == "prefill":
        pairs, keys, rows = _visible(case)
        return {"bytes": 576.0 * keys + rows * HEADS * (DIM * 3 + 4), "flops": 4.0 * HEADS * DIM * pairs}
    if case["op"] == "branch":
        lens, new = _branch_sizes(case)
        size = 0.0
        for i, n in enumerate(new):
            total = lens[i // case["each"]]
            size += 2.0 * 704 * (total % PAGE) * case["layers"]  # the rest of the prompt, read and written
            size += 4.0 * (2 * (total // PAGE) + 2) + 8 * n  # table rows, counts, slots
        return {"bytes": size, "flops": 0.0}
    if case["op"] == "commit":
        _, drafts = _commit_sizes(case)
        kept = sum(min(9.0, 2.0 * n / (1 + max(1, n // 8))) for n in drafts)  # about, of a drawn path
        return {"bytes": 2.0 * 704 * kept * case["layers"] + 16.0 * len(drafts), "flops": 0.0}
    n, width = case["n"], 4 if case["dtype"] == "fp32" else 2
    pairs, m = len(_axis_of_pair(case)), len(case["sections"].split(","))
    live = n - case["skip"]
    rows = HEADS + 2 * KV + 1 + IDX_HEADS
    size = n * (rows * DIM * width + 8 + 4 * m + pairs * 8 + (HEADS + IDX_HEADS) * DIM) + live * 704
    back = live * (704 + (2 * KV + 1) * DIM * 2) + 8 * n  # cache bytes in, values out
    return {"bytes": float(size + back), "flops": float(n * (rows - KV) * pairs * 6 + live * 2 * KV * DIM * 4)}


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


def _exact_turn(x, z, inter):
    """Pairs as complex numbers times z [n, pairs]."""
    half = z.shape[1]
    w = x[..., : 2 * half]
    w = torch.view_as_complex(w.unflatten(-1, (half, 2)).contiguous()) if inter else torch.complex(w[..., :half].contiguous(), w[..., half:].contiguous())
    w = w * z[:, None]
    w = torch.view_as_real(w).flatten(-2) if inter else torch.cat((w.real, w.imag), -1)
    return torch.cat((w, x[..., 2 * half :]), -1)


def _exact_cached(x, s_enc):
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    blocks = x.reshape(-1, 16)
    scale = _exact_fp8(blocks.abs().max(1).values / 6 * s_enc)[:, None]
    r = torch.where(scale > 0, blocks.abs() * s_enc / torch.where(scale > 0, scale, 1.0), 0.0)
    return (torch.copysign(_nearest(r.contiguous(), grid), blocks) * scale / s_enc).view(x.shape)


def _exact_rows(pool, slots, codes, scales):
    """FP8 operands e2m1 * scale of the tokens at `slots` for every head [n, 4, 128], byte by byte from the page format."""
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
    v = _exact_fp8(torch.tensor(_E2M1, dtype=torch.float64, device=d)[mag] * sb)
    return torch.where(sgn == 1, -v, v)


def exact(case, seed):
    if case["op"] in ("branch", "commit"):
        return None  # bytes and whole numbers
    s = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(s)
    live = s["slots"] >= 0
    half = s["cos_sin"].shape[1] // 2
    z = torch.zeros((case["n"], half), dtype=torch.complex128, device="cuda")
    for i, a in enumerate(_axis_of_pair(case)):
        t = s["cos_sin"][s["positions"][a].long()].double()
        z[:, i] = torch.complex(t[:, i], t[:, half + i])
    inter = case["inter"]
    q, qi = (_exact_fp8(_exact_turn(s[name].double(), z, inter)) for name in ("q", "q_idx"))
    k = _exact_cached(_exact_turn(s["k"].double(), z, inter), S_ENC_K) * live[:, None, None]
    v = _exact_cached(s["v"].double(), S_ENC_V) * live[:, None, None]
    idx = _exact_fp8(_exact_turn(s["idx_k"].double()[:, None], z, inter))[:, 0] * live[:, None]
    return q, qi, k, v, idx


def _exact_prefill(s):
    """Sequence by sequence, KV head by KV head, some rows at a time."""
    case, f8 = s["case"], _fp8_table()
    lens, start = s["seq_lens"].tolist(), s["q_start_loc"].tolist()
    out = torch.zeros((start[-1], HEADS, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((start[-1], HEADS), -math.inf, dtype=torch.float64, device="cuda")
    for b, total in enumerate(lens):
        n = start[b + 1] - start[b]
        if not n:
            continue
        at = torch.arange(total, device="cuda")
        slots = s["block_table"][b].long()[at // PAGE] * PAGE + at % PAGE
        k = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["k"]) for a in slots.split(16384)]) / S_ENC_K
        v = torch.cat([_exact_rows(s["kv_pool"], a, *OFF["v"]) for a in slots.split(16384)]) / S_ENC_V
        for i in range(0, n, 512):
            rows = torch.arange(i, min(i + 512, n), device="cuda")
            pos = total - n + rows
            sees = at[None, :] < (s["ends"][start[b] + rows][:, None] if "ends" in s else pos[:, None] + 1)
            if case["window"]:
                sees &= at[None, :] > pos[:, None] - case["window"]
            some = sees.any(1)
            q = f8[s["q"][start[b] + rows].long()]
            for h in range(HEADS):
                z = (q[:, h] @ k[:, h // 4].T) / DIM**0.5
                z = z.masked_fill(~sees, -math.inf)[some]
                lse[start[b] + rows[some], h] = torch.logsumexp(z, 1)
                out[start[b] + rows[some], h] = torch.softmax(z, 1) @ v[:, h // 4]
    return out, lse
