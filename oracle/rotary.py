"""Oracle: rotary positions on given rows, and what a cache slot's bytes stand for.

Test infrastructure only (see ``oracle/__init__``).  Two forms of the rotation:
``turn`` in float64 (the mathematics), and ``turn_fp32`` with every product and
sum rounded to fp32 on its own (the documented rounding, NumPy float32).

Parity: pinned (tests/test_oracle_rotary.py) by complex multiplication, by the
fused projection's oracle at whole heads and half pairs, and by hand cases.
"""

import numpy as np

from . import formats, layout

F32 = np.float32


def _pairs(x, rot, interleaved):
    w = x[..., :rot]
    return (w[..., 0::2], w[..., 1::2]) if interleaved else (w[..., : rot // 2], w[..., rot // 2:])


def _join(a, b, x, rot, interleaved):
    out = np.array(x)
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = a, b
    else:
        out[..., : rot // 2], out[..., rot // 2: rot] = a, b
    return out


def turn(x, cos_sin_rows, interleaved):
    """float64 rotation of rows [n, heads, 128] by table rows [n, rot] (cos, then sin)."""
    x = np.asarray(x, dtype=np.float64)
    t = np.asarray(cos_sin_rows, dtype=np.float64)[:, None, :]
    rot = t.shape[-1]
    if rot == 0:
        return x
    c, s = t[..., : rot // 2], t[..., rot // 2:]
    a, b = _pairs(x, rot, interleaved)
    return _join(a * c - b * s, b * c + a * s, x, rot, interleaved)


def turn_fp32(x, cos_sin_rows, interleaved):
    """The same in IEEE fp32 steps: two products and one sum, each rounded."""
    x = np.asarray(x, dtype=F32)
    t = np.asarray(cos_sin_rows, dtype=F32)[:, None, :]
    rot = t.shape[-1]
    if rot == 0:
        return x
    c, s = t[..., : rot // 2], t[..., rot // 2:]
    a, b = _pairs(x, rot, interleaved)
    return _join((a * c).astype(F32) - (b * s).astype(F32), (b * c).astype(F32) + (a * s).astype(F32), x, rot, interleaved)


def slot_values(kv_pool, idx_pool, slot, s_enc_k, s_enc_v):
    """fp32 (k [4, 128], v [4, 128], idx [128]) that a slot's bytes stand for:
    e2m1(code) * fl(sb * fl(1 / s_enc)), and the E4M3 values of the index key."""
    page, t = slot // layout.PAGE_TOKENS, slot % layout.PAGE_TOKENS
    kc, ks, vc, vs = layout.read_kv_slot(kv_pool, page, t)
    out = []
    for codes, scales, s_enc in ((kc, ks, s_enc_k), (vc, vs, s_enc_v)):
        dec = F32(1) / F32(s_enc)
        d = (formats.decode_e4m3(scales).astype(F32) * dec).astype(F32)
        v = formats.decode_e2m1(codes).astype(F32).reshape(4, 8, 16) * d[..., None]
        out.append(v.astype(F32).reshape(4, 128))
    return out[0], out[1], formats.decode_e4m3(layout.read_index_slot(idx_pool, page, t)).astype(F32)
