"""Refusals of the paged calls without a GPU: every bad argument comes back as
a status before any CUDA call."""

import ctypes

import pytest

from quantized_decode_attention_head_b200 import _lib

P = 0x10000  # a 16-byte aligned address that nothing reads
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


def config(**kw):
    c = dict(n_layers=2, n_pages=10, page_size=16, n_q_heads=8, n_kv_heads=4, head_dim=64, dtype=0)
    c.update(kw)
    return _lib.PagedConfig(**c)


def init(cfg, k=P, v=P):
    h = ctypes.c_void_p(0)
    st = _lib.lib().rq_paged_cache_init(ctypes.byref(cfg), k, v, ctypes.byref(h))
    return st, h


@pytest.fixture
def cache():
    st, h = init(config())
    assert st == OK
    yield h
    _lib.lib().rq_paged_cache_destroy(h)


def batch(**kw):
    b = dict(n_seqs=2, n_tokens=2, max_new=1, table_width=4, page_table=P, kv_lens=P, cu_new=None)
    b.update(kw)
    return _lib.PagedBatch(**b)


@pytest.mark.parametrize("kw,st", [
    (dict(), OK), (dict(page_size=128, dtype=1, head_dim=128), OK), (dict(n_q_heads=32, n_kv_heads=4), OK),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(head_dim=80), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(n_q_heads=12), UNSUPPORTED),
    (dict(n_q_heads=9), UNSUPPORTED), (dict(n_layers=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_pages=2**24, page_size=128), UNSUPPORTED), (dict(n_kv_heads=0), INVALID),
])
def test_init(kw, st):
    got, h = init(config(**kw))
    assert got == st
    _lib.lib().rq_paged_cache_destroy(h)


def test_init_pointers():
    for k, v in ((None, P), (P, None), (P + 2, P), (P, P + 8)):
        assert init(config(), k, v)[0] == INVALID
    assert _lib.lib().rq_paged_cache_init(None, P, P, ctypes.byref(ctypes.c_void_p())) == INVALID
    _lib.lib().rq_paged_cache_destroy(None)


def attention(cache, b=None, shared=False, **kw):
    a = dict(layer=0, prefix=P, prefix_len=40, q=P, q_stride=512, out=P, lse=None, scale=0.0, window=0, sink=0, ws=P,
             ws_bytes=1 << 30)
    a.update(kw)
    b = b if b is not None else batch()
    rest = (a["q"], a["q_stride"], a["out"], a["lse"], a["scale"], a["window"], a["sink"], a["ws"], a["ws_bytes"], None)
    if shared:
        return _lib.lib().rq_paged_shared_attention(cache, a["layer"], ctypes.byref(b), a["prefix"], a["prefix_len"], *rest)
    return _lib.lib().rq_paged_attention(cache, a["layer"], ctypes.byref(b), *rest)


BAD_BATCH = [dict(n_seqs=-1), dict(n_tokens=-1), dict(max_new=-1), dict(table_width=0), dict(page_table=None),
             dict(kv_lens=None), dict(page_table=P + 2), dict(kv_lens=P + 1), dict(cu_new=P + 2),
             dict(n_tokens=1)]  # two sequences of one token each in one row


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(q=None), dict(out=None), dict(ws=None), dict(q=P + 8), dict(out=P + 2),
    dict(ws=P + 8), dict(lse=P + 2), dict(q_stride=504), dict(q_stride=516), dict(q_stride=-512), dict(window=-1),
    dict(sink=-1), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_attention_arguments(cache, shared, kw):
    assert attention(cache, shared=shared, **kw) == INVALID


@pytest.mark.parametrize("shared", [False, True])
def test_attention_batch_and_workspace(cache, shared):
    for kw in BAD_BATCH:
        assert attention(cache, batch(**kw), shared) == INVALID, kw
    assert attention(cache, shared=shared, ws_bytes=128) == WORKSPACE
    assert attention(None, shared=shared) == INVALID
    # nothing to do: no launch
    assert attention(cache, batch(n_seqs=0, n_tokens=0, page_table=None, kv_lens=None), shared, q=None, out=None) == OK


def test_shared_prefix_arguments(cache):
    for kw in (dict(prefix=None), dict(prefix=P + 2), dict(prefix_len=-1)):
        assert attention(cache, shared=True, **kw) == INVALID


def test_workspace_bytes(cache):
    n = ctypes.c_size_t(0)
    f = _lib.lib().rq_paged_workspace_bytes
    assert f(cache, 4, 4, ctypes.byref(n)) == OK and n.value > 0
    small = n.value
    assert f(cache, 400, 40000, ctypes.byref(n)) == OK and n.value >= small
    assert f(cache, -1, 4, ctypes.byref(n)) == INVALID and f(cache, 4, -1, ctypes.byref(n)) == INVALID
    assert f(None, 4, 4, ctypes.byref(n)) == INVALID and f(cache, 4, 4, None) == INVALID


def rotation(**kw):
    r = dict(cos_sin=P, n_positions=100, rot_dim=64, interleaved=0, positions=None, n_axes=1, sections=(32, 0, 0, 0))
    r.update(kw)
    r["sections"] = (ctypes.c_int * 4)(*r["sections"])
    return _lib.Rotation(**r)


def append(cache, b=None, rot=None, **kw):
    a = dict(layer=0, k=P, ks=256, v=P, vs=256, q=P, qs=512, q_out=P, status=P)
    a.update(kw)
    return _lib.lib().rq_paged_append(cache, a["layer"], ctypes.byref(b if b is not None else batch()),
                                      None if rot is False else ctypes.byref(rot or rotation()), a["k"], a["ks"], a["v"],
                                      a["vs"], a["q"], a["qs"], a["q_out"], a["status"], None)


@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(k=P + 2), dict(v=P + 4), dict(ks=255), dict(ks=260),
    dict(vs=248), dict(q_out=None), dict(q=P + 2), dict(q_out=P + 8), dict(qs=504), dict(qs=520 + 4), dict(status=P + 1)])
def test_append_arguments(cache, kw):
    assert append(cache, **kw) == INVALID


def test_append_batch_and_rotation(cache):
    for kw in BAD_BATCH:
        assert append(cache, batch(**kw)) == INVALID, kw
    assert append(cache, rot=False) == INVALID  # queries without a rotation
    for kw, st in ((dict(cos_sin=None), INVALID), (dict(cos_sin=P + 4), INVALID), (dict(n_positions=0), INVALID),
                   (dict(rot_dim=0), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED), (dict(rot_dim=128), UNSUPPORTED),
                   (dict(n_axes=0), UNSUPPORTED), (dict(n_axes=5), UNSUPPORTED), (dict(positions=P + 2), INVALID),
                   (dict(n_axes=2, sections=(16, 16, 0, 0)), INVALID),  # several axes need positions
                   (dict(sections=(31, 0, 0, 0)), INVALID), (dict(sections=(33, 0, 0, 0)), INVALID),
                   (dict(positions=P, n_axes=3, sections=(40, -16, 8, 0)), INVALID)):
        assert append(cache, rot=rotation(**kw)) == st, kw
    assert append(cache, batch(n_seqs=0, n_tokens=0, page_table=None, kv_lens=None), k=None, v=None, q=None) == OK
