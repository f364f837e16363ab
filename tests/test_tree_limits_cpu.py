"""Limits of the tree attention's scales, refused on the host (calls without tokens: nothing is launched)."""

import ctypes

import pytest

from test_abi_cpu import _cache, lib  # noqa: F401


@pytest.mark.parametrize("s_enc_v,code", [(1.0, 0), (448.0, 0), (1.4e-36, 0), (2.0**-119, 0), (2.0**100, 0),
                                          (2.0**-120, -1), (1e-38, -1), (2.0**101, -1), (3e38, -1)])
def test_value_scales(lib, s_enc_v, code):  # noqa: F811
    """With 2^8 / s_enc_v at 2^128 or above an output of zero was 0 * inf; above 2^100 the factor of a
    long row loses bits as a subnormal number."""
    fake = ctypes.c_void_p(16)
    cache = _cache(kv_pool=16, idx_pool=16, s_enc_v=s_enc_v)
    assert lib.msa_tree_attn(ctypes.byref(cache), fake, 16, 0.1, fake, 4, fake, fake, 1, 0, None, None, None, 1, fake,
                             fake, fake, 1 << 32, None) == code
