"""Python binding of libmsa.so: argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; this module
checks tensor dtypes, devices and shapes, passes raw pointers and the current
CUDA stream, and raises on a negative return code.  PyTorch provides device
memory and streams.  There is no fallback: if the library is missing, loading
it raises.
"""

import ctypes
import math
import os
import re
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmsa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "msa.h")

PAGE_TOKENS = 128
KV_HEADS = 4
HEAD_DIM = 128
IDX_DIM = 128
IDX_HEADS = 8
Q_HEADS = 16
TOPK = 16
KV_PAGE_BYTES = 73_728
NOALLOC_SCRATCH_BYTES = 8 << 20  # MSA_INDEXER_NOALLOC_SCRATCH_BYTES
INJECT_BARRIER_TIMEOUT = 0x1     # MSA_INJECT_BARRIER_TIMEOUT
INJECT_ATTENTION_TIMEOUT = 0x2   # MSA_INJECT_ATTENTION_TIMEOUT
STATUS_BAD_SLOT, STATUS_BAD_PAGE, STATUS_BAD_SEQ, STATUS_BAD_SELECTION, STATUS_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
STATUS_NO_PAGES = 0x20
IDX_PAGE_BYTES = 16_384

ERRORS = {-1: "invalid argument", -2: "unsupported shape", -3: "workspace too small",
          -4: "kernel launch failed", -5: "larger than the library's static scratch"}


class MsaError(RuntimeError):
    pass


class _Cache(ctypes.Structure):
    _fields_ = [
        ("kv_pool", ctypes.c_void_p),
        ("idx_pool", ctypes.c_void_p),
        ("n_pages", ctypes.c_int64),
        ("page_tokens", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("idx_dim", ctypes.c_int32),
        ("s_enc_k", ctypes.c_float),
        ("s_enc_v", ctypes.c_float),
        ("status", ctypes.c_void_p),
    ]


class _Rows(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("idx_k", ctypes.c_void_p),
        ("q_idx", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("idx_k_stride", ctypes.c_int64),
        ("q_idx_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
    ]


# The same layouts packed to bytes in one step: a third of the time for calls that are short.
_CACHE = struct.Struct("@PPqiiiiffP")
_ROWS = struct.Struct("@5P5qi0P")
assert _CACHE.size == ctypes.sizeof(_Cache) and _ROWS.size == ctypes.sizeof(_Rows)


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SIGS = {
    "msa_quantize_kv_insert": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P]),
    "msa_indexer_topk": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _P,
                                        _P, _P, ctypes.c_size_t, _P]),
    "msa_indexer_workspace_bytes": (ctypes.c_size_t, [_I32, _I32]),
    "msa_indexer_topk_noalloc": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32,
                                                _P, _P, _P]),
    "msa_sparse_attn_decode": (ctypes.c_int, [_P, _P, _I32, ctypes.c_float, _P, _P, _P, _I32, _P,
                                              _P, _I32, _I32, _I32, _P, _P, _P]),
    "msa_merge_splits": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "msa_debug_set_fault_injection": (ctypes.c_int, [_I32, ctypes.c_uint64]),
    "msa_pack_blocks": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P]),
    "msa_indexer_topk_range": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32,
                                              _I32, _P, _P, ctypes.c_size_t, _P]),
    "msa_indexer_merge_candidates": (ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _P, _P,
                                                    _P]),
    "msa_unpack_blocks": (ctypes.c_int, [_P, _I32, _P, _P, _I32, _P]),
    "msa_block_row_bytes": (ctypes.c_size_t, [_I32]),
    "msa_decode_fused": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, ctypes.c_float, _P, _I32, _P, _P, _I32,
                                        _I32, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_decode_fused_workspace_bytes": (ctypes.c_size_t, [_I32, _I32]),
    "msa_qkv_project_insert": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _P, _P, _P, _P, _I32, _P, _P,
                                              ctypes.c_float, _P, _P, _P]),
    "msa_rope_table": (ctypes.c_int, [_P, _I32, ctypes.c_double, _P]),
    "msa_rotary_insert": (ctypes.c_int, [_P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "msa_rotary_insert_axes": (ctypes.c_int, [_P, _P, _I32, _P, _I32, _I32, _I32, _P, _I32, ctypes.c_char_p, _P, _P, _P,
                                              _P]),
    "msa_rope_table_freqs": (ctypes.c_int, [_P, _I32, _P, _I32, ctypes.c_double, _P]),
    "msa_read_kv": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P, _P]),
    "msa_tree_attn": (ctypes.c_int, [_P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P, _I32, _I32, _P, _P, _P, _I32, _P,
                                     _P, _P, ctypes.c_size_t, _P]),
    "msa_tree_attn_workspace_bytes": (ctypes.c_size_t, [_I32]),
    "msa_prefill_attn": (ctypes.c_int, [_P, _P, _I32, ctypes.c_float, _P, _I32, _P, _P, _I32, _I32, _I32, _P, _I32, _I32,
                                        _P, _P, _P, ctypes.c_size_t, _P]),
    "msa_prefill_workspace_bytes": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "msa_extend_sequences": (ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _P, _P]),
    "msa_fork_sequences": (ctypes.c_int, [_P, _I32, _P, _P, _I32, _P, _I32, _P, _P, _I32, _P, ctypes.c_size_t, _P]),
    "msa_fork_workspace_bytes": (ctypes.c_size_t, [_I32]),
    "msa_release_sequences": (ctypes.c_int, [_P, _P, _I32, _P, _I32, _P, _I32, _P]),
    "msa_copy_pages": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I32, _P]),
    "msa_commit_drafts": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P]),
    "msa_absmax": (ctypes.c_int, [_P, _I64, _P, _P]),
    "msa_encode_scale": (ctypes.c_float, [ctypes.c_float]),
    "msa_debug_fp8_page": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
    "msa_read_status": (ctypes.c_int, [_P, _P, _P]),
    "msa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}


def lib():
    """The loaded libmsa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MsaError(f"{LIB_PATH} is missing: build it with nvfp4_kv_block_gb300.build.build()")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def header_symbols():
    """Names of the functions include/msa.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(msa_\w+)\s*\(", text, re.M)))


def _check(rc):
    if rc != 0:
        raise MsaError(f"libmsa error {rc}: {ERRORS.get(rc, 'unknown')}")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t, dtype, name, dims=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {t.dim()}")
    return ctypes.c_void_p(t.data_ptr())


class KVCache:
    """NVFP4 KV pool + FP8 index pool of n_pages 128-token pages, caller-owned."""

    def __init__(self, n_pages, s_enc_k, s_enc_v, device="cuda"):
        self.n_pages = int(n_pages)
        self.kv_pool = torch.zeros((self.n_pages, KV_PAGE_BYTES), dtype=torch.uint8, device=device)
        self.idx_pool = torch.zeros((self.n_pages, IDX_PAGE_BYTES), dtype=torch.uint8, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.s_enc_k = float(s_enc_k)
        self.s_enc_v = float(s_enc_v)

    @classmethod
    def from_pools(cls, kv_pool, idx_pool, s_enc_k, s_enc_v, status=None):
        """A cache over pools that the caller holds already: uint8 [n_pages, 73,728]
        and [n_pages, 16,384] in the page format, each on a 16-byte boundary, and an int32
        [1] status word (a new one if None)."""
        for t, name in ((kv_pool, "kv_pool"), (idx_pool, "idx_pool")):
            if isinstance(t, torch.Tensor) and t.data_ptr() % 16:
                raise ValueError(f"{name} must begin on a 16-byte boundary")
        _ptr(kv_pool, torch.uint8, "kv_pool", 2)
        _ptr(idx_pool, torch.uint8, "idx_pool", 2)
        n = kv_pool.shape[0]
        if tuple(kv_pool.shape) != (n, KV_PAGE_BYTES) or tuple(idx_pool.shape) != (n, IDX_PAGE_BYTES):
            raise ValueError("kv_pool must be [n, 73728] and idx_pool [n, 16384]")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=kv_pool.device)
        _ptr(status, torch.int32, "status", 1)
        if not (kv_pool.device == idx_pool.device == status.device):
            raise ValueError("the pools and the status word must be on one device")
        self = cls.__new__(cls)
        self.n_pages, self.kv_pool, self.idx_pool, self.status = n, kv_pool, idx_pool, status
        self.s_enc_k, self.s_enc_v = float(s_enc_k), float(s_enc_v)
        return self

    def struct(self):
        return _Cache(self.kv_pool.data_ptr(), self.idx_pool.data_ptr(), self.n_pages, PAGE_TOKENS,
                      KV_HEADS, HEAD_DIM, IDX_DIM, self.s_enc_k, self.s_enc_v,
                      self.status.data_ptr())

    def packed(self):
        """``struct()`` as bytes."""
        return _CACHE.pack(self.kv_pool.data_ptr(), self.idx_pool.data_ptr(), self.n_pages, PAGE_TOKENS, KV_HEADS,
                           HEAD_DIM, IDX_DIM, self.s_enc_k, self.s_enc_v, self.status.data_ptr())

    def read_status(self):
        out = ctypes.c_int32(0)
        c = self.struct()
        _check(lib().msa_read_status(ctypes.byref(c), ctypes.byref(out), _stream()))
        return out.value


def encode_scale(amax):
    return lib().msa_encode_scale(float(amax))


def absmax_(x, amax):
    """Fold max|x| into the device float ``amax`` (shape [1], caller zeroed)."""
    _check(lib().msa_absmax(_ptr(x, torch.float32, "x"), x.numel(), _ptr(amax, torch.float32, "amax"),
                            _stream()))


def quantize_kv_insert(cache, k, v, idx_k, slot_mapping):
    n = k.shape[0]
    if tuple(k.shape) != (n, KV_HEADS, HEAD_DIM) or tuple(v.shape) != (n, KV_HEADS, HEAD_DIM):
        raise ValueError("k, v must be [n, 4, 128]")
    if tuple(idx_k.shape) != (n, IDX_DIM) or tuple(slot_mapping.shape) != (n,):
        raise ValueError("idx_k must be [n, 128] and slot_mapping [n]")
    c = cache.struct()
    _check(lib().msa_quantize_kv_insert(ctypes.byref(c), _ptr(k, torch.float32, "k"),
                                        _ptr(v, torch.float32, "v"), _ptr(idx_k, torch.float32, "idx_k"),
                                        _ptr(slot_mapping, torch.int64, "slot_mapping"), n, _stream()))


def indexer_workspace_bytes(n_q_total, max_pages):
    return lib().msa_indexer_workspace_bytes(int(n_q_total), int(max_pages))


def indexer_topk(cache, q_idx, w, block_table, seq_lens, q_start_loc, ws=None, sel=None,
                 n_sel=None, topk=TOPK):
    """Select blocks for every query token.  Returns (sel [T,17], n_sel [T], ws)."""
    T = q_idx.shape[0]
    if tuple(q_idx.shape) != (T, IDX_HEADS, IDX_DIM) or tuple(w.shape) != (T, IDX_HEADS):
        raise ValueError("q_idx must be [T, 8, 128] uint8 and w [T, 8] float32")
    n_seqs, max_pages = block_table.shape
    if tuple(seq_lens.shape) != (n_seqs,) or tuple(q_start_loc.shape) != (n_seqs + 1,):
        raise ValueError("seq_lens must be [B], q_start_loc [B+1]")
    dev = q_idx.device
    if ws is None:  # zeroed: its first bytes are grid-barrier words
        ws = torch.zeros(indexer_workspace_bytes(T, max_pages), dtype=torch.uint8, device=dev)
    if sel is None:
        sel = torch.empty((T, topk + 1), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((T,), dtype=torch.int32, device=dev)
    c = cache.struct()
    _check(lib().msa_indexer_topk(
        ctypes.byref(c), _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"), IDX_HEADS,
        _ptr(block_table, torch.int32, "block_table"), max_pages, _ptr(seq_lens, torch.int32, "seq_lens"),
        _ptr(q_start_loc, torch.int32, "q_start_loc"), n_seqs, T, topk, _ptr(sel, torch.int32, "sel"),
        _ptr(n_sel, torch.int32, "n_sel"), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream()))
    return sel, n_sel, ws


def indexer_topk_range(cache, q_idx, w, block_table, seq_lens, q_start_loc, blk_lo, blk_hi, ws=None,
                       cand=None, topk=TOPK):
    """Local top-16 keys (uint64 stored as int64, [T, 16]) of the blocks
    [blk_lo, blk_hi) of every sequence.  Returns (cand, ws)."""
    T = q_idx.shape[0]
    if tuple(q_idx.shape) != (T, IDX_HEADS, IDX_DIM) or tuple(w.shape) != (T, IDX_HEADS):
        raise ValueError("q_idx must be [T, 8, 128] uint8 and w [T, 8] float32")
    n_seqs, max_pages = block_table.shape
    dev = q_idx.device
    if ws is None:
        ws = torch.zeros(indexer_workspace_bytes(T, max_pages), dtype=torch.uint8, device=dev)
    if cand is None:
        cand = torch.empty((T, topk), dtype=torch.int64, device=dev)
    c = cache.struct()
    _check(lib().msa_indexer_topk_range(
        ctypes.byref(c), _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"), IDX_HEADS,
        _ptr(block_table, torch.int32, "block_table"), max_pages, _ptr(seq_lens, torch.int32, "seq_lens"),
        _ptr(q_start_loc, torch.int32, "q_start_loc"), n_seqs, T, topk, int(blk_lo), int(blk_hi),
        _ptr(cand, torch.int64, "cand"), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream()))
    return cand, ws


def indexer_merge_candidates(cache, cand, seq_lens, q_start_loc, max_pages, sel=None, n_sel=None,
                             topk=TOPK):
    """Merge [n_shards, T, 16] candidate keys into (sel [T, 17], n_sel [T])."""
    n_shards, T, _ = cand.shape
    dev = cand.device
    if sel is None:
        sel = torch.empty((T, topk + 1), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((T,), dtype=torch.int32, device=dev)
    c = cache.struct()
    _check(lib().msa_indexer_merge_candidates(
        ctypes.byref(c), _ptr(cand, torch.int64, "cand"), n_shards, _ptr(seq_lens, torch.int32, "seq_lens"),
        _ptr(q_start_loc, torch.int32, "q_start_loc"), seq_lens.shape[0], int(max_pages), T, topk,
        _ptr(sel, torch.int32, "sel"), _ptr(n_sel, torch.int32, "n_sel"), _stream()))
    return sel, n_sel


def indexer_topk_noalloc(cache, q_idx, w, block_table, seq_lens, q_start_loc, sel=None,
                         n_sel=None, topk=TOPK):
    """indexer_topk through the allocation-free entry point (static scratch in the
    library).  Returns (sel [T,17], n_sel [T])."""
    T = q_idx.shape[0]
    if tuple(q_idx.shape) != (T, IDX_HEADS, IDX_DIM) or tuple(w.shape) != (T, IDX_HEADS):
        raise ValueError("q_idx must be [T, 8, 128] uint8 and w [T, 8] float32")
    n_seqs, max_pages = block_table.shape
    if tuple(seq_lens.shape) != (n_seqs,) or tuple(q_start_loc.shape) != (n_seqs + 1,):
        raise ValueError("seq_lens must be [B], q_start_loc [B+1]")
    dev = q_idx.device
    if sel is None:
        sel = torch.empty((T, topk + 1), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((T,), dtype=torch.int32, device=dev)
    c = cache.struct()
    _check(lib().msa_indexer_topk_noalloc(
        ctypes.byref(c), _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"), IDX_HEADS,
        _ptr(block_table, torch.int32, "block_table"), max_pages, _ptr(seq_lens, torch.int32, "seq_lens"),
        _ptr(q_start_loc, torch.int32, "q_start_loc"), n_seqs, T, topk, _ptr(sel, torch.int32, "sel"),
        _ptr(n_sel, torch.int32, "n_sel"), _stream()))
    return sel, n_sel


def sparse_attn_decode(cache, q, sel, n_sel, block_table, seq_lens, q_start_loc, n_splits,
                       softmax_scale=None, o_part=None, lse_part=None):
    T = q.shape[0]
    if tuple(q.shape) != (T, Q_HEADS, HEAD_DIM):
        raise ValueError("q must be [T, 16, 128] uint8 (E4M3)")
    n_seqs, max_pages = block_table.shape
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(HEAD_DIM)
    dev = q.device
    if o_part is None:
        o_part = torch.empty((T, n_splits, Q_HEADS, HEAD_DIM), dtype=torch.float32, device=dev)
    if lse_part is None:
        lse_part = torch.empty((T, n_splits, Q_HEADS), dtype=torch.float32, device=dev)
    c = cache.struct()
    _check(lib().msa_sparse_attn_decode(
        ctypes.byref(c), _ptr(q, torch.uint8, "q"), Q_HEADS, float(softmax_scale),
        _ptr(sel, torch.int32, "sel"), _ptr(n_sel, torch.int32, "n_sel"),
        _ptr(block_table, torch.int32, "block_table"), max_pages, _ptr(seq_lens, torch.int32, "seq_lens"),
        _ptr(q_start_loc, torch.int32, "q_start_loc"), n_seqs, T, int(n_splits),
        _ptr(o_part, torch.float32, "o_part"), _ptr(lse_part, torch.float32, "lse_part"), _stream()))
    return o_part, lse_part


def merge_splits(o_part, lse_part, out=None, lse=None):
    """LSE merge of the splits: returns out [T, H, 128] (and fills lse [T, H] if given)."""
    T, S, H, D = o_part.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.float32, device=o_part.device)
    lse_p = ctypes.c_void_p(None) if lse is None else _ptr(lse, torch.float32, "lse")
    _check(lib().msa_merge_splits(_ptr(o_part, torch.float32, "o_part"),
                                  _ptr(lse_part, torch.float32, "lse_part"), T, H, S,
                                  _ptr(out, torch.float32, "out"), lse_p, _stream()))
    return out


def block_row_bytes(n_layers):
    return lib().msa_block_row_bytes(int(n_layers))


def _layer_array(caches):
    arr = (_Cache * len(caches))()
    for i, c in enumerate(caches):
        arr[i] = c.struct()
    return arr


def pack_blocks(caches, pages, rows=None):
    """Block-outer rows [n_blocks, n_layers * 90,112] of the physical pages
    ``pages`` (int32 [n_blocks]) from the per-layer caches."""
    n = pages.shape[0]
    if rows is None:
        rows = torch.empty((n, block_row_bytes(len(caches))), dtype=torch.uint8, device=pages.device)
    arr = _layer_array(caches)
    _check(lib().msa_pack_blocks(arr, len(caches), _ptr(pages, torch.int32, "pages", 1), n,
                                 _ptr(rows, torch.uint8, "rows"), _stream()))
    return rows


def unpack_blocks(caches, rows, pages):
    """Write block-outer rows back into pages ``pages`` of every layer's pools."""
    arr = _layer_array(caches)
    _check(lib().msa_unpack_blocks(arr, len(caches), _ptr(rows, torch.uint8, "rows"),
                                   _ptr(pages, torch.int32, "pages", 1), pages.shape[0], _stream()))


QKV_HEADS = 25  # MSA_QKV_HEADS


def rope_table(max_pos, base=10000.0, device="cuda"):
    """fp32 [max_pos, 128] RoPE cos / sin table (msa_rope_table)."""
    t = torch.empty((max_pos, 128), dtype=torch.float32, device=device)
    _check(lib().msa_rope_table(_ptr(t, torch.float32, "cos_sin"), int(max_pos), float(base), _stream()))
    return t


def qkv_project_insert(cache, x, w, gamma_q, gamma_k, gamma_idx, cos_sin, positions, slot_mapping,
                       eps=1e-6, q8=None, y_out=None):
    """Fused projection -> RMS norm -> RoPE -> FP8 queries (returned, [n, 16, 128])
    and NVFP4 / FP8 cache insertion.  ``y_out`` ([n, 25, 128] fp32) receives the
    rows before rounding when given."""
    n, d = x.shape
    if tuple(w.shape) != (QKV_HEADS * HEAD_DIM, d):
        raise ValueError("w must be [25 * 128, d_model] bf16")
    if q8 is None:
        q8 = torch.empty((n, Q_HEADS, HEAD_DIM), dtype=torch.uint8, device=x.device)
    yp = ctypes.c_void_p(None) if y_out is None else _ptr(y_out, torch.float32, "y_out")
    c = cache.struct()
    _check(lib().msa_qkv_project_insert(
        ctypes.byref(c), _ptr(x, torch.bfloat16, "x", 2), _ptr(w, torch.bfloat16, "w", 2), n, d,
        _ptr(gamma_q, torch.float32, "gamma_q"), _ptr(gamma_k, torch.float32, "gamma_k"),
        _ptr(gamma_idx, torch.float32, "gamma_idx"), _ptr(cos_sin, torch.float32, "cos_sin", 2),
        cos_sin.shape[0], _ptr(positions, torch.int32, "positions"), _ptr(slot_mapping, torch.int64, "slot_mapping"),
        float(eps), _ptr(q8, torch.uint8, "q8"), yp, _stream()))
    return q8


_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # MSA_DTYPE_*


def _raw_stream(dev):
    """The current stream of CUDA device ``dev`` (an index), as an integer."""
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same without a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(cache):
    """Index of the cache's CUDA device, which has to be the current one."""
    dev = cache.kv_pool.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"the cache is on {cache.kv_pool.device}, not on the current CUDA device")
    return dev


def _arg(t, dtype, shape, dev, name):
    """Pointer of a contiguous tensor of this type and shape on CUDA device ``dev`` (raises
    otherwise).  A call has a dozen of them: the checks are one line when they hold."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _ptr(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be on the cache's device cuda:{dev}, got {t.device}")


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_max_pos=None, beta_fast=32.0,
                     beta_slow=1.0):
    """(frequencies of the rot_dim / 2 pairs, amplitude) of a rotary embedding
    (J. Su et al., 2021).

    Unscaled: base^(-2i / rot_dim).  ``scaling`` stretches a model trained on
    ``original_max_pos`` positions to ``factor`` times as many:
      "linear"  every position divided by the factor (S. Chen et al., "Extending
                Context Window of Large Language Models via Positional
                Interpolation", 2023);
      "ntk"     base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is
                stretched by the factor, the fastest not at all;
      "yarn"    pairs that turn more than ``beta_fast`` times over the original
                length keep their frequency, pairs below ``beta_slow`` turns are
                divided by the factor, a linear ramp over the pair index between;
                amplitude 0.1 ln(factor) + 1 (B. Peng, J. Quesnelle, H. Fan,
                E. Shippole, "YaRN: Efficient Context Window Extension of Large
                Language Models", 2023).  The ramp's ends are rounded outward to
                whole pairs and held to 0 and rot_dim - 1.
    """
    if rot_dim % 16 or not 0 <= rot_dim <= HEAD_DIM:
        raise ValueError("rot_dim must be a multiple of 16 from 0 to 128")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError("base must be above 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not factor >= 1.0 or not math.isfinite(factor):
        raise ValueError("factor must be at least 1")
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling != "yarn":
        return freq, 1.0
    if original_max_pos is None or original_max_pos <= 0 or not beta_fast > beta_slow > 0:
        raise ValueError("yarn needs original_max_pos > 0 and beta_fast > beta_slow > 0")

    def pair(turns):  # the (fractional) pair that turns so often over the original length
        return rot_dim * math.log(original_max_pos / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

    # The ends of the ramp as models are trained with: whole pairs, and an upper end of at most
    # rot_dim - 1, a channel's index (an end behind the last pair, rot_dim / 2 - 1, leaves that pair
    # between its frequency and the divided one).  Ends that meet are kept apart by 1e-3 of a pair: a step.
    lo = max(math.floor(pair(beta_fast)), 0)
    hi = min(math.ceil(pair(beta_slow)), rot_dim - 1)
    out = []
    for i, f in enumerate(freq):
        slow = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        out.append(f * (1.0 - slow) + f / factor * slow)
    return out, 0.1 * math.log(factor) + 1.0


def rope_table_scaled(max_pos, rot_dim=HEAD_DIM, base=10000.0, scaling=None, factor=1.0, original_max_pos=None,
                      device="cuda", **betas):
    """fp32 [max_pos, rot_dim] cos / sin table of ``rope_frequencies`` for rotary_insert
    (msa_rope_table_freqs); a table of rot_dim 128 also serves qkv_project_insert."""
    freq, amplitude = rope_frequencies(rot_dim, base, scaling, factor, original_max_pos, **betas)
    t = torch.empty((max_pos, rot_dim), dtype=torch.float32, device=device)
    arr = (ctypes.c_double * max(len(freq), 1))(*freq)
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{t.device} is not the current CUDA device")
    _check(lib().msa_rope_table_freqs(t.data_ptr(), int(max_pos), arr, int(rot_dim), amplitude, _stream()))
    return t


def _rows(t, name, shape, dtype, dev):
    """(pointer, token stride) of projected rows [n, heads, 128] or [n, 128]."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            st = t.stride()
            if st[-1] == 1 and (len(st) == 2 or st[1] == HEAD_DIM):
                ptr, stride = t.data_ptr(), st[0] if shape[0] > 1 else 0
                if not (ptr | stride * (4 if dtype is torch.float32 else 2)) & 15:
                    return ptr, stride
                raise ValueError(f"{name} and its token stride must be aligned to 16 bytes")
            raise ValueError(f"{name} must have contiguous channels and heads")
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} like q, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be on the cache's device cuda:{dev}, got {t.device}")


MAX_AXES = 4  # MSA_MAX_AXES


class RopeAxes:
    """The axis of each rotary pair: ``n_axes`` and ``pairs`` (bytes, one per pair)."""

    def __init__(self, n_axes, pairs):
        self.n_axes, self.pairs = int(n_axes), bytes(pairs)
        if not 1 <= self.n_axes <= MAX_AXES:
            raise ValueError(f"1 to {MAX_AXES} axes, not {n_axes}")
        if any(a >= self.n_axes for a in self.pairs):
            raise ValueError(f"a pair's axis must be below {n_axes}")


def rope_axes(sections, dealt=False):
    """RopeAxes of ``sections``, counts of pairs of each axis (time, height, width, ...; their
    sum is rot_dim / 2).  The sections follow one another (pairs 0 .. sections[0] - 1 are the
    first axis's), or, when ``dealt``, the axes take the pairs in turn: pair i is of axis
    i % n_axes where i < n_axes * sections[i % n_axes], else of the first axis.  So an axis a > 0
    has the count asked for where its last turn, a + n_axes * (sections[a] - 1), is below the sum,
    and fewer where the pairs end before it ([3, 5]: 4 and 4)."""
    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0:
        raise ValueError("sections must be counts of pairs")
    m = len(sections)
    if dealt:
        pairs = [i % m if i < m * sections[i % m] else 0 for i in range(sum(sections))]
    else:
        pairs = [a for a, n in enumerate(sections) for _ in range(n)]
    return RopeAxes(m, pairs)


def rotary_insert(cache, q, k, v, idx_k, cos_sin, positions, slot_mapping, q_idx=None, interleaved=False, q8=None,
                  qi8=None, axes=None):
    """Rotary positions on projected rows, FP8 queries and index queries (returned:
    uint8 [n, 16, 128] and [n, 8, 128], or None without ``q_idx``), and NVFP4 / FP8
    cache insertion at ``slot_mapping`` (negative: not inserted).

    Rows are fp32, bf16 or fp16, [n, heads, 128] ([n, 128] index keys), contiguous
    within a token; slices of one projection's output will do.  ``cos_sin`` is fp32
    [max_pos, rot_dim]: the first rot_dim channels of each head are turned, in pairs
    (i, i + rot_dim / 2), or (2i, 2i + 1) when ``interleaved``, by the table's row at
    ``positions`` (int32 [n]), or, with ``axes`` (rope_axes, one entry per pair), at each
    pair's own axis of ``positions`` (int32 [n_axes, n]).
    """
    n, dtype = q.shape[0], q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {dtype}")
    dev = _device_of(cache)
    qp, qs = _rows(q, "q", (n, Q_HEADS, HEAD_DIM), dtype, dev)
    kp, ks = _rows(k, "k", (n, KV_HEADS, HEAD_DIM), dtype, dev)
    vp, vs = _rows(v, "v", (n, KV_HEADS, HEAD_DIM), dtype, dev)
    ip, i_s = _rows(idx_k, "idx_k", (n, IDX_DIM), dtype, dev)
    if q8 is None:
        q8 = torch.empty((n, Q_HEADS, HEAD_DIM), dtype=torch.uint8, device=q.device)
    if q_idx is None:
        qi8 = qi8p = None
        qip = qis = 0
    else:
        qip, qis = _rows(q_idx, "q_idx", (n, IDX_HEADS, IDX_DIM), dtype, dev)
        if qi8 is None:
            qi8 = torch.empty((n, IDX_HEADS, IDX_DIM), dtype=torch.uint8, device=q.device)
        qi8p = _arg(qi8, torch.uint8, (n, IDX_HEADS, IDX_DIM), dev, "qi8")
    max_pos, rot_dim = cos_sin.shape
    if axes is not None:
        if len(axes.pairs) != rot_dim // 2:
            raise ValueError(f"axes are of {len(axes.pairs)} pairs, the table of {rot_dim // 2}")
        _check(lib().msa_rotary_insert_axes(
            cache.packed(), _ROWS.pack(qp, kp, vp, ip, qip, qs, ks, vs, i_s, qis, code), n,
            _arg(cos_sin, torch.float32, (max_pos, rot_dim), dev, "cos_sin"), max_pos, rot_dim, 1 if interleaved else 0,
            _arg(positions, torch.int32, (axes.n_axes, n), dev, "positions"), axes.n_axes, axes.pairs,
            _arg(slot_mapping, torch.int64, (n,), dev, "slot_mapping"),
            _arg(q8, torch.uint8, (n, Q_HEADS, HEAD_DIM), dev, "q8"), qi8p, _raw_stream(dev)))
        return q8, qi8
    _check(lib().msa_rotary_insert(
        cache.packed(), _ROWS.pack(qp, kp, vp, ip, qip, qs, ks, vs, i_s, qis, code), n,
        _arg(cos_sin, torch.float32, (max_pos, rot_dim), dev, "cos_sin"), max_pos, rot_dim, 1 if interleaved else 0,
        _arg(positions, torch.int32, (n,), dev, "positions"),
        _arg(slot_mapping, torch.int64, (n,), dev, "slot_mapping"),
        _arg(q8, torch.uint8, (n, Q_HEADS, HEAD_DIM), dev, "q8"), qi8p, _raw_stream(dev)))
    return q8, qi8


def read_kv(cache, slot_mapping, dtype=torch.bfloat16, k=None, v=None, idx_k=None):
    """The values the cache holds at ``slot_mapping`` (int64 [n]): K [n, 4, 128],
    V [n, 4, 128] and index keys [n, 128].  Rows go into the given tensors (of one
    type: fp32, bf16 or fp16), or, when none is given, into new ones of ``dtype``;
    the others are not read and come back as None.  Rows of negative slots are left
    as they were (zeros in new tensors)."""
    n = slot_mapping.shape[0]
    first = k if k is not None else v if v is not None else idx_k
    if first is not None:
        dtype = first.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"values are float32, bfloat16 or float16, not {dtype}")
    dev = _device_of(cache)
    if first is None:
        k, v = (torch.zeros((n, KV_HEADS, HEAD_DIM), dtype=dtype, device=cache.kv_pool.device) for _ in range(2))
        idx_k = torch.zeros((n, IDX_DIM), dtype=dtype, device=cache.kv_pool.device)
    _check(lib().msa_read_kv(
        cache.packed(), _arg(slot_mapping, torch.int64, (n,), dev, "slot_mapping"), n, code,
        None if k is None else _arg(k, dtype, (n, KV_HEADS, HEAD_DIM), dev, "k"),
        None if v is None else _arg(v, dtype, (n, KV_HEADS, HEAD_DIM), dev, "v"),
        None if idx_k is None else _arg(idx_k, dtype, (n, IDX_DIM), dev, "idx_k"), _raw_stream(dev)))
    return k, v, idx_k


TREE_MAX_DRAFTS = 64  # MSA_TREE_MAX_DRAFTS: query tokens of one sequence in tree_attn


class TreeBuffers:
    """Outputs and scratch of tree_attn calls with n_q_total query rows (exactly: rows
    behind the last sequence are padding, and stay as they were) and up to n_seqs
    sequences, reused across steps: out [n_q_total, 16, 128] in ``dtype`` (bf16 or
    fp16), lse [n_q_total, 16].  Padding rows count where the kernel is chosen: buffers
    of at most 16 rows a sequence keep the one that is faster for few drafts."""

    def __init__(self, n_q_total, n_seqs, dtype=torch.bfloat16, device="cuda"):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"tree_attn's output is bfloat16 or float16, not {dtype}")
        self.T, self.n_seqs = int(n_q_total), int(n_seqs)
        nbytes = lib().msa_tree_attn_workspace_bytes(self.T)
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.out = torch.zeros((self.T, Q_HEADS, HEAD_DIM), dtype=dtype, device=device)
        self.lse = torch.zeros((self.T, Q_HEADS), dtype=torch.float32, device=device)


def tree_attn(cache, q, block_table, seq_lens, q_start_loc, bufs, tree_mask=None, sel=None, n_sel=None,
              softmax_scale=None):
    """Attention of each sequence's query tokens (drafts, up to 64, already in the
    cache) over its whole cached context and over the drafts that ``tree_mask``
    names (int64 [T], bit i of a draft's word: it sees draft i of its sequence;
    None: drafts 0 .. itself).  With ``sel`` [B, 17] and ``n_sel`` [B] (ascending block
    ids, e.g. of indexer_topk for one token per sequence) only those blocks of the
    context are visited, and the blocks that hold drafts.  Returns bufs.out
    [T, 16, 128]; bufs.lse [T, 16] has the log-sum-exp of the logits."""
    T = bufs.T
    n_seqs, max_pages = block_table.shape
    if n_seqs > bufs.n_seqs:
        raise ValueError(f"bufs are for up to {bufs.n_seqs} sequences")
    if (sel is None) != (n_sel is None):
        raise ValueError("sel and n_sel come together")
    dev = _device_of(cache)
    _check(lib().msa_tree_attn(
        cache.packed(), _arg(q, torch.uint8, (T, Q_HEADS, HEAD_DIM), dev, "q"), Q_HEADS,
        HEAD_DIM ** -0.5 if softmax_scale is None else float(softmax_scale),
        _arg(block_table, torch.int32, (n_seqs, max_pages), dev, "block_table"), max_pages,
        _arg(seq_lens, torch.int32, (n_seqs,), dev, "seq_lens"),
        _arg(q_start_loc, torch.int32, (n_seqs + 1,), dev, "q_start_loc"), n_seqs, T,
        None if tree_mask is None else _arg(tree_mask, torch.int64, (T,), dev, "tree_mask"),
        None if sel is None else _arg(sel, torch.int32, (n_seqs, TOPK + 1), dev, "sel"),
        None if sel is None else _arg(n_sel, torch.int32, (n_seqs,), dev, "n_sel"), _DTYPES[bufs.out.dtype],
        _arg(bufs.out, bufs.out.dtype, (T, Q_HEADS, HEAD_DIM), dev, "bufs.out"),
        _arg(bufs.lse, torch.float32, (T, Q_HEADS), dev, "bufs.lse"), bufs.ws.data_ptr(), bufs.ws.numel(),
        _raw_stream(dev)))
    return bufs.out


class PrefillBuffers:
    """Outputs and scratch of prefill_attn calls with n_q_total query rows (exactly: rows behind
    the last sequence stay as they were), up to n_seqs sequences and n_pages pages of their
    contexts (the sum of ceil(seq_len / 128), or of those within the window; a page counts for
    each sequence that shares it): out [n_q_total, 16, 128] in ``dtype`` (bf16 or fp16), lse
    [n_q_total, 16], and 196,608 bytes of scratch a page.  ``ws``: scratch of other buffers, to share it between layers or steps (calls that
    share it must not overlap on the GPU)."""

    def __init__(self, n_q_total, n_seqs, n_pages, dtype=torch.bfloat16, device="cuda", ws=None):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"prefill_attn's output is bfloat16 or float16, not {dtype}")
        self.T, self.n_seqs, self.n_pages = int(n_q_total), int(n_seqs), int(n_pages)
        nbytes = lib().msa_prefill_workspace_bytes(self.T, self.n_seqs, self.n_pages)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if ws is None else ws
        self.out = torch.zeros((self.T, Q_HEADS, HEAD_DIM), dtype=dtype, device=device)
        self.lse = torch.zeros((self.T, Q_HEADS), dtype=torch.float32, device=device)


def prefill_attn(cache, q, block_table, seq_lens, q_start_loc, bufs, window=0, ends=None, softmax_scale=None):
    """Attention of each sequence's query tokens (its last ones, any number of them, already in
    the cache) over its cached context: token i at position pos sees the positions t with
    start <= t < end, start = max(0, pos + 1 - window) (0 without a window), end = pos + 1
    or, with ``ends`` (int32 [T]), its entry there (at most the sequence's length: the tokens of
    an image that see all of it).  Returns bufs.out [T, 16, 128] (zeros where a token sees
    nothing); bufs.lse [T, 16] has the log-sum-exp of the logits."""
    T = bufs.T
    n_seqs, max_pages = block_table.shape
    if n_seqs > bufs.n_seqs:
        raise ValueError(f"bufs are for up to {bufs.n_seqs} sequences")
    if not 0 <= window < 1 << 31:
        raise ValueError(f"a window is 0 or a number of tokens, not {window}")
    dev = _device_of(cache)
    _check(lib().msa_prefill_attn(
        cache.packed(), _arg(q, torch.uint8, (T, Q_HEADS, HEAD_DIM), dev, "q"), Q_HEADS,
        HEAD_DIM ** -0.5 if softmax_scale is None else float(softmax_scale),
        _arg(block_table, torch.int32, (n_seqs, max_pages), dev, "block_table"), max_pages,
        _arg(seq_lens, torch.int32, (n_seqs,), dev, "seq_lens"),
        _arg(q_start_loc, torch.int32, (n_seqs + 1,), dev, "q_start_loc"), n_seqs, T, int(window),
        None if ends is None else _arg(ends, torch.int32, (T,), dev, "ends"), bufs.n_pages, _DTYPES[bufs.out.dtype],
        _arg(bufs.out, bufs.out.dtype, (T, Q_HEADS, HEAD_DIM), dev, "bufs.out"),
        _arg(bufs.lse, torch.float32, (T, Q_HEADS), dev, "bufs.lse"),
        _arg(bufs.ws, torch.uint8, bufs.ws.shape, dev, "bufs.ws"), bufs.ws.numel(), _raw_stream(dev)))
    return bufs.out


class CacheLayers:
    """The caches of a model's layers, in which page p is the same block: the array that
    the calls on all layers take, made once.  The caches' pools stay theirs."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("at least one cache")
        if any(c.kv_pool.device != self.caches[0].kv_pool.device for c in self.caches):
            raise ValueError("the caches must be on one device")
        self.n = len(self.caches)
        self.array = _layer_array(self.caches)

    @staticmethod
    def of(x):
        """``x`` if it is one, else the CacheLayers of a cache or of a list of caches."""
        return x if isinstance(x, CacheLayers) else CacheLayers([x] if isinstance(x, KVCache) else x)


_POOL = struct.Struct("@PPiP")


class PagePool:
    """Counts of the block-table entries that hold each of n_pages pages: ``refs`` int32
    [n_pages], and the free ones' mask, which the calls below keep in step (refs is read,
    not written, by anyone else).  Calls on one pool must not overlap on the GPU: one stream,
    or streams that wait for one another.  ``status``: int32 [1] word of sticky STATUS_*
    bits."""

    def __init__(self, n_pages, status=None, device="cuda"):
        self._set(torch.zeros(int(n_pages), dtype=torch.int32, device=device), status)

    @classmethod
    def from_refs(cls, refs, status=None):
        """A pool over counts that the caller holds already (int32 [n_pages], no smaller than 0)."""
        _ptr(refs, torch.int32, "refs", 1)
        self = cls.__new__(cls)
        self._set(refs, status)
        return self

    def _set(self, refs, status):
        self.n_pages, self.refs = refs.shape[0], refs
        if self.n_pages == 0:
            raise ValueError("a pool has at least one page")
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=refs.device)
        _ptr(status, torch.int32, "status", 1)
        if status.device != refs.device:
            raise ValueError("refs and the status word must be on one device")
        self.status = status
        bits = torch.zeros(-(-self.n_pages // 32) * 32, dtype=torch.int64, device=refs.device)
        bits[: self.n_pages] = refs == 0
        words = (bits.view(-1, 32) << torch.arange(32, device=refs.device)).sum(1)
        self.free_mask = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        self._ws = torch.zeros(lib().msa_fork_workspace_bytes(4096), dtype=torch.uint8, device=refs.device)

    def packed(self):
        return _POOL.pack(self.refs.data_ptr(), self.free_mask.data_ptr(), self.n_pages, self.status.data_ptr())


def _table(pool, block_table, seq_lens):
    """(device, rows, columns, pointers) of a block table and its lengths."""
    dev = pool.refs.get_device()
    if dev != _current_device():
        raise ValueError(f"the pool is on {pool.refs.device}, not on the current CUDA device")
    n_seqs, max_pages = block_table.shape
    return (dev, n_seqs, max_pages, _arg(block_table, torch.int32, (n_seqs, max_pages), dev, "block_table"),
            _arg(seq_lens, torch.int32, (n_seqs,), dev, "seq_lens"))


def extend_sequences(pool, block_table, seq_lens, q_start_loc, slots):
    """Room for q_start_loc[b + 1] - q_start_loc[b] new tokens of each sequence: pages of
    the pool for the entries of its row that have none (lowest pages first), its length
    grown in place.  ``slots`` (int64 [n_tokens], returned) gets the slot of every new token,
    or -1 where a sequence could not grow and for rows behind the last sequence; none grows
    where q_start_loc goes back."""
    dev, n_seqs, max_pages, table, lens = _table(pool, block_table, seq_lens)
    n = slots.shape[0]
    _check(lib().msa_extend_sequences(pool.packed(), table, max_pages, lens,
                                      _arg(q_start_loc, torch.int32, (n_seqs + 1,), dev, "q_start_loc"), n_seqs, n,
                                      _arg(slots, torch.int64, (n,), dev, "slots"), _raw_stream(dev)))
    return slots


def fork_sequences(layers, pool, block_table, seq_lens, src, dst):
    """Row dst[i] of the table, which has to be empty (no tokens, no entry that holds a page),
    becomes a second copy of row src[i] (int32 [n] each): full pages are shared, the tokens of
    the last one are copied to a page of its own in every layer (``layers``: CacheLayers, a list
    of caches or one cache)."""
    layers = CacheLayers.of(layers)
    dev, n_seqs, max_pages, table, lens = _table(pool, block_table, seq_lens)
    _same_device(layers, dev)
    n = src.shape[0]
    _check(lib().msa_fork_sequences(layers.array, layers.n, pool.packed(), table, max_pages, lens, n_seqs,
                                    _arg(src, torch.int32, (n,), dev, "src"), _arg(dst, torch.int32, (n,), dev, "dst"), n,
                                    pool._ws.data_ptr(), pool._ws.numel(), _raw_stream(dev)))


def release_sequences(pool, block_table, seq_lens, rows):
    """Gives the pages of the table's rows ``rows`` (int32 [n]) back and empties the rows."""
    dev, n_seqs, max_pages, table, lens = _table(pool, block_table, seq_lens)
    n = rows.shape[0]
    _check(lib().msa_release_sequences(pool.packed(), table, max_pages, lens, n_seqs,
                                       _arg(rows, torch.int32, (n,), dev, "rows"), n, _raw_stream(dev)))


def _same_device(layers, dev):
    at = layers.caches[0].kv_pool.get_device()
    if at != dev or at != _current_device():
        raise ValueError(f"the caches are on {layers.caches[0].kv_pool.device}, not on the current CUDA device")


def copy_pages(layers, src, dst, tokens=None):
    """Page src[i] to page dst[i] (int32 [n] each; negative: none) in every layer, or its
    first tokens[i] tokens (int32 [n]).  Targets are distinct and no pair's source."""
    layers = CacheLayers.of(layers)
    dev = src.get_device()
    _same_device(layers, dev)
    n = src.shape[0]
    _check(lib().msa_copy_pages(layers.array, layers.n, _arg(src, torch.int32, (n,), dev, "src"),
                                _arg(dst, torch.int32, (n,), dev, "dst"),
                                None if tokens is None else _arg(tokens, torch.int32, (n,), dev, "tokens"), n,
                                _raw_stream(dev)))


def commit_drafts(layers, block_table, seq_lens, q_start_loc, accepted, new_lens=None):
    """Of each sequence's last q_start_loc[b + 1] - q_start_loc[b] tokens (drafts that
    tree_attn verified) those whose bits ``accepted`` (int64 [B]) has move together behind
    its context, in every layer.  Returns the new lengths (``new_lens`` or a new tensor,
    never seq_lens itself); the row keeps its pages.  A fork of a sequence comes before its
    drafts or behind their commit: its full pages are shared."""
    layers = CacheLayers.of(layers)
    dev = seq_lens.get_device()
    _same_device(layers, dev)
    n_seqs, max_pages = block_table.shape
    if new_lens is None:
        new_lens = torch.empty_like(seq_lens)
    _check(lib().msa_commit_drafts(
        layers.array, layers.n, _arg(block_table, torch.int32, (n_seqs, max_pages), dev, "block_table"), max_pages,
        _arg(seq_lens, torch.int32, (n_seqs,), dev, "seq_lens"),
        _arg(q_start_loc, torch.int32, (n_seqs + 1,), dev, "q_start_loc"), n_seqs,
        _arg(accepted, torch.int64, (n_seqs,), dev, "accepted"), _arg(new_lens, torch.int32, (n_seqs,), dev, "new_lens"),
        _raw_stream(dev)))
    return new_lens


def set_fault_injection(flags=0, wait_limit_ns=0):
    """Test hook: wait limit of every later launch (0 = the 2 s default) and
    fault-injection flags (INJECT_BARRIER_TIMEOUT, INJECT_ATTENTION_TIMEOUT); 0, 0 restores
    the defaults."""
    _check(lib().msa_debug_set_fault_injection(int(flags), int(wait_limit_ns)))


def debug_fp8_page(cache, page):
    k8 = torch.empty((KV_HEADS, PAGE_TOKENS, HEAD_DIM), dtype=torch.uint8, device=cache.kv_pool.device)
    v8 = torch.empty_like(k8)
    c = cache.struct()
    _check(lib().msa_debug_fp8_page(ctypes.byref(c), int(page), _ptr(k8, torch.uint8, "k8"),
                                    _ptr(v8, torch.uint8, "v8"), _stream()))
    return k8, v8


def choose_splits(n_q_total, n_sms=152):
    """Splits per query token for the attention kernel.

    The attention kernel runs one persistent CTA per SM; work items are
    (token, KV head, split), dealt round-robin, each with up to
    ceil(17 / splits) pages.  The busiest CTA then streams about
    ceil(items / SMs) x (pages per item + an item overhead of about two pages);
    pick the split count that minimises that, with a small charge per split
    for the partial outputs written and merged, preferring fewer splits on ties.
    At most 4 splits (items of at least 5 pages): with a handful of tokens the
    attention's per-item start-up and the merge launch outweigh the shorter
    items (measured on 4 tokens of 512K context: 2 to 5 splits give the same
    step time, 9 add 2.5 us and 17 add 7 us).
    """
    best, best_cost = 1, None
    for s in range(1, 5):
        items = KV_HEADS * max(1, n_q_total) * s
        cost = math.ceil(items / n_sms) * (math.ceil((TOPK + 1) / s) + 2.0)
        cost *= 1.0 + 0.02 * s
        if best_cost is None or cost < best_cost - 1e-9:
            best, best_cost = s, cost
    return best


class DecodeBuffers:
    """Preallocated outputs and scratch of one decode step (reused across steps)."""

    def __init__(self, n_q_total, max_pages, n_splits, device="cuda"):
        self.T, self.n_splits = n_q_total, n_splits
        self.ws = torch.zeros(indexer_workspace_bytes(n_q_total, max_pages), dtype=torch.uint8, device=device)
        self.sel = torch.empty((n_q_total, TOPK + 1), dtype=torch.int32, device=device)
        self.n_sel = torch.empty((n_q_total,), dtype=torch.int32, device=device)
        self.o_part = torch.empty((n_q_total, n_splits, Q_HEADS, HEAD_DIM), dtype=torch.float32, device=device)
        self.lse_part = torch.empty((n_q_total, n_splits, Q_HEADS), dtype=torch.float32, device=device)
        # one split: its normalised output is already the answer (no merge launch)
        self.out = (self.o_part.view(n_q_total, Q_HEADS, HEAD_DIM) if n_splits == 1 else
                    torch.empty((n_q_total, Q_HEADS, HEAD_DIM), dtype=torch.float32, device=device))


FUSED_MAX_SEQS = 64     # limits of msa_decode_fused (low concurrency)
FUSED_MAX_TOKENS = 64


class FusedBuffers:
    """Outputs and scratch of the single-launch decode step (reused across steps)."""

    def __init__(self, n_q_total, max_pages, device="cuda"):
        self.T = n_q_total
        nbytes = lib().msa_decode_fused_workspace_bytes(int(n_q_total), int(max_pages))
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)  # zeroed: barrier words
        self.sel = torch.empty((n_q_total, TOPK + 1), dtype=torch.int32, device=device)
        self.n_sel = torch.empty((n_q_total,), dtype=torch.int32, device=device)
        self.out = torch.empty((n_q_total, Q_HEADS, HEAD_DIM), dtype=torch.float32, device=device)


def decode_fused(cache, q, q_idx, w, block_table, seq_lens, q_start_loc, bufs, softmax_scale=None):
    """The decode step in one launch (scan, top-k, attention, merge) for low
    concurrency.  Returns bufs.out [T, 16, 128]; bufs.sel / bufs.n_sel hold the
    selection."""
    T = q.shape[0]
    if tuple(q.shape) != (T, Q_HEADS, HEAD_DIM) or tuple(q_idx.shape) != (T, IDX_HEADS, IDX_DIM):
        raise ValueError("q must be [T, 16, 128] and q_idx [T, 8, 128] uint8 (E4M3)")
    n_seqs, max_pages = block_table.shape
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(HEAD_DIM)
    c = cache.struct()
    _check(lib().msa_decode_fused(
        ctypes.byref(c), _ptr(q, torch.uint8, "q"), _ptr(q_idx, torch.uint8, "q_idx"), _ptr(w, torch.float32, "w"),
        Q_HEADS, IDX_HEADS, float(softmax_scale), _ptr(block_table, torch.int32, "block_table"), max_pages,
        _ptr(seq_lens, torch.int32, "seq_lens"), _ptr(q_start_loc, torch.int32, "q_start_loc"), n_seqs, T, TOPK,
        _ptr(bufs.sel, torch.int32, "sel"), _ptr(bufs.n_sel, torch.int32, "n_sel"),
        _ptr(bufs.out, torch.float32, "out"), _ptr(bufs.ws, torch.uint8, "ws"), bufs.ws.numel(), _stream()))
    return bufs.out


def decode_step(cache, q, q_idx, w, block_table, seq_lens, q_start_loc, bufs, softmax_scale=None):
    """One decode step: indexer top-k, sparse attention splits, and the LSE merge
    of the splits (3 kernels; 2 with a single split, whose output is final)."""
    indexer_topk(cache, q_idx, w, block_table, seq_lens, q_start_loc, ws=bufs.ws, sel=bufs.sel,
                 n_sel=bufs.n_sel)
    sparse_attn_decode(cache, q, bufs.sel, bufs.n_sel, block_table, seq_lens, q_start_loc,
                       bufs.n_splits, softmax_scale, o_part=bufs.o_part, lse_part=bufs.lse_part)
    if bufs.n_splits > 1:
        merge_splits(bufs.o_part, bufs.lse_part, out=bufs.out)
    return bufs.out
