"""Oracle: attention of drafted tokens over a cached context, float64.

Test infrastructure only (see ``oracle/__init__``).  Operands as in the sparse
decode (``oracle.attention``): FP8 queries against NVFP4 keys and values
dequantised to FP8; draft i of a sequence sits behind its ctx committed tokens
and sees them and the drafts whose bits its mask word has.

Parity: pinned (tests/test_oracle_tree.py) by ``oracle.attention.attend`` for
chains, by a per-key Python loop and by hand masks.
"""

import numpy as np

from . import formats, layout, nvfp4


def page_operands(page):
    """E4M3 bytes (k8, v8) [128 tokens, 4 heads, 128] of one KV page's 73,728 bytes.

    Scale bytes that are no number (0x7F, 0xFF) count as zero."""
    heads = np.asarray(page, dtype=np.uint8).reshape(layout.KV_HEADS, layout.HEAD_BYTES)
    t = np.arange(layout.PAGE_TOKENS)
    out = []
    for off_c, off_s in ((layout.OFF_KC, layout.OFF_KS), (layout.OFF_VC, layout.OFF_VS)):
        rows = heads[:, off_c: off_c + 8192].reshape(4, 128, 4, 16)
        chunks = np.stack([rows[:, t, layout.code_chunk_position(c, t)] for c in range(4)], axis=2)
        codes = layout.unpack_codes(chunks.reshape(4, 128, 64))
        scales = heads[:, off_s: off_s + 1024].reshape(4, 8, 128).transpose(0, 2, 1)
        scales = np.where((scales & 0x7F) == 0x7F, 0, scales)
        out.append(nvfp4.fp8_operand(codes, scales).transpose(1, 0, 2))
    return out[0], out[1]


def visible(ctx, n_q, words, positions, sel=None):
    """bool [n_q, len(positions)]: which cached positions each draft sees.  words: one
    int per draft (None: draft j sees 0 .. j); sel: block ids of the context that are
    visited (None: all), beside the blocks from ctx // 128 on."""
    out = np.zeros((n_q, len(positions)), dtype=bool)
    for j in range(n_q):
        word = (2 << j) - 1 if words is None else int(words[j])
        for i, pos in enumerate(positions):
            if sel is not None and pos // 128 < ctx // 128 and pos // 128 not in sel:
                continue
            out[j, i] = pos < ctx or (pos - ctx < n_q and word >> (pos - ctx) & 1)
    return out


def attend(q8, k8, v8, seen, softmax_scale, s_enc_k, s_enc_v):
    """(out [n, 16, 128], lse [n, 16], the mean |v| under the weights [n, 16, 128], the largest
    sum of |q k| behind a logit [n, 16]) of queries q8 [n, 16, 128] over keys [L, 4, 128]."""
    q = formats.decode_e4m3(q8)
    k, v = formats.decode_e4m3(k8), formats.decode_e4m3(v8)
    n = q.shape[0]
    out, mean = np.zeros((n, 16, 128)), np.zeros((n, 16, 128))
    lse, size = np.full((n, 16), -np.inf), np.zeros((n, 16))
    fac = float(softmax_scale) / float(np.float32(s_enc_k))
    for h in range(16):
        z = q[:, h] @ k[:, h // 4].T * fac
        size[:, h] = np.where(seen, np.abs(q[:, h]) @ np.abs(k[:, h // 4]).T, 0).max(1, initial=0) * fac
        for j in range(n):
            if not seen[j].any():
                continue
            x = z[j, seen[j]]
            p = np.exp(x - x.max())
            lse[j, h] = x.max() + np.log(p.sum())
            p /= p.sum()
            vv = v[seen[j], h // 4] / float(np.float32(s_enc_v))
            out[j, h] = p @ vv
            mean[j, h] = p @ np.abs(vv)
    return out, lse, mean, size
