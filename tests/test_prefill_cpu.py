"""Refusals of the prompt attention on the host, before any CUDA call."""

import ctypes

import pytest
import torch

from nvfp4_kv_block_gb300 import ops
from test_abi_cpu import _cache, lib  # noqa: F401

P = ctypes.c_void_p
FAKE = P(32)


def test_prefill_is_checked_on_the_host(lib):  # noqa: F811
    def call(change=None, **kw):
        c = _cache(kv_pool=160, idx_pool=160, n_pages=4, **kw)
        #       q     heads scale table cols lens  start seqs T  window ends n_vis dtype out  lse   ws    bytes    stream
        args = [FAKE, 16, 0.1, FAKE, 4, FAKE, FAKE, 1, 0, 0, None, 8, 1, FAKE, None, FAKE, 1 << 40, None]
        for i, v in (change or {}).items():
            args[i] = v
        return lib.msa_prefill_attn(ctypes.byref(c), *args)

    assert call() == 0
    for change, code in [({1: 8}, -2), ({2: 0.0}, -1), ({2: float("nan")}, -1), ({4: 0}, -1), ({4: 65537}, -2), ({7: -1}, -1),
                         ({7: 4097}, -2), ({8: -1}, -1), ({8: 262145}, -2), ({9: -1}, -1), ({11: -1}, -1), ({11: (1 << 20) + 1}, -2),
                         ({12: 0}, -1), ({12: 3}, -1), ({8: 1, 0: None}, -1), ({8: 1, 13: None}, -1), ({8: 1, 15: None}, -1),
                         ({8: 1, 7: 0}, -1), ({0: P(8)}, -1), ({13: P(16)}, -1), ({15: P(8)}, -1), ({16: 255}, -3),
                         ({8: 1, 16: 1 << 20}, -3), ({2: 2.0}, -1), ({2: 1e30}, -1)]:
        assert call(change) == code, change
    # scores of at most 2^26: the scale's end moves with the keys'
    assert call({2: 1.8}) == 0 and call({2: 1.8}, s_enc_k=0.9) == -1
    assert call(s_enc_v=2e30) == -1 and call(s_enc_v=1e-37) == -1
    small, large = (lib.msa_prefill_workspace_bytes(*x) for x in ((100, 1, 1), (100, 1, 2)))
    assert large - small in range(4 * 49152, 4 * 49152 + 257) and lib.msa_prefill_workspace_bytes(0, 1, 1) == 256
    off = _cache(kv_pool=168, idx_pool=160, n_pages=4)
    assert lib.msa_prefill_attn(ctypes.byref(off), FAKE, 16, 0.1, FAKE, 4, FAKE, FAKE, 1, 0, 0, None, 8, 1, FAKE, None, FAKE, 1 << 40, None) == -1


@pytest.mark.parametrize("window", [-1, 1 << 31, (1 << 32) + 5])
def test_a_window_is_a_number_of_tokens(lib, window):  # noqa: F811
    bufs = ops.PrefillBuffers(3, 1, 2, device="cpu")
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="window"):
        ops.prefill_attn(None, None, table, None, None, bufs, window=window)
    with pytest.raises(ValueError, match="sequences"):
        ops.prefill_attn(None, None, table.expand(2, 2), None, None, bufs)
    with pytest.raises(TypeError):
        ops.PrefillBuffers(3, 1, 2, torch.float32, device="cpu")
