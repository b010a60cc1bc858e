"""Sizes past the paged calls' 31-bit positions, refused without a GPU."""

import ctypes

import pytest

from quantized_decode_attention_head_b200 import _lib

P = 0x10000  # a 16-byte aligned address that nothing reads
UNSUPPORTED = 2


@pytest.mark.parametrize("prefix,width,tokens", [
    (None, 2**27, 2), (None, 2**27 - 1, 20), (2**31 - 70, 4, 7), (2**31 - 1, 1, 1), (None, 4, 2**28)])
def test_positions_past_31_bits(prefix, width, tokens):
    cfg = _lib.PagedConfig(n_layers=1, n_pages=10, page_size=16, n_q_heads=8, n_kv_heads=4, head_dim=64, dtype=0)
    h = ctypes.c_void_p(0)
    assert _lib.lib().rq_paged_cache_init(ctypes.byref(cfg), P, P, ctypes.byref(h)) == 0
    b = _lib.PagedBatch(n_seqs=1, n_tokens=tokens, max_new=tokens, table_width=width, page_table=P, kv_lens=P, cu_new=P)
    rest = (P, 512, P, None, 0.0, 0, 0, P, 2**60, None)
    if prefix is None:
        got = _lib.lib().rq_paged_attention(h, 0, ctypes.byref(b), *rest)
    else:
        got = _lib.lib().rq_paged_shared_attention(h, 0, ctypes.byref(b), P, prefix, *rest)
    _lib.lib().rq_paged_cache_destroy(h)
    assert got == UNSUPPORTED
