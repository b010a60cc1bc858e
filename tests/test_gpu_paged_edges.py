"""The paged 16-bit cache on the GPU where callers leave the usual path: other
streams, lengths past the table, freed pages, weights of very different size."""

import pytest
import torch

from paged_helpers import Batch, angles
from quantized_decode_attention_head_b200 import PagedKVCache

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(bt):
    return PagedKVCache(bt.k_pages, bt.v_pages, bt.hq)


def attend(bt, cache, window=0, n_sink=0, **kw):
    a = dict(cu_new=bt.cu, max_new=bt.max_new, window=window, n_sink=n_sink)
    a.update(kw)
    if bt.prefix:
        return cache.rq_paged_shared_attention(bt.layer, bt.q, bt.prefix_pages, bt.prefix, bt.table, bt.kv_lens, **a)
    return cache.rq_paged_attention(bt.layer, bt.q, bt.table, bt.kv_lens, **a)


# --------------------------------------------------- queries rotated in place
@pytest.mark.parametrize("lens,prefix", [([(2000, 1), (40, 1)], 0), ([(700, 90), (30, 2)], 0), ([(60, 1), (9, 1)], 700)])
def test_rotated_in_place_and_attended_at_once(lens, prefix):
    """The append writes the queries over themselves and the attention behind
    it, resident already, reads them; so do the kernels that merge their parts:
    bit for bit what separate tensors give, over many rounds in the same memory."""
    bt = Batch(lens, 8, 2, 128, 32, BF, seed=41, prefix=prefix)
    g = torch.Generator().manual_seed(42)
    rounds = 30
    qs = [torch.randn((bt.rows, 8, 128), generator=g).to(BF).cuda() for _ in range(rounds)]
    new = [torch.randn((bt.rows, 2, 128), generator=g).to(BF).cuda() for _ in range(2)]
    cs = angles(4096, 128)
    cache = make(bt)
    ws = cache.make_workspace(len(lens), bt.rows)
    want = []
    for q in qs:
        bt.q = cache.rq_paged_append(0, *new, bt.table, bt.kv_lens, cu_new=bt.cu, q=q, cos_sin=cs)
        torch.cuda.synchronize()
        want.append(attend(bt, cache, 500, 3, workspace=ws))
        torch.cuda.synchronize()
    bt.q = torch.empty_like(qs[0])
    got = []
    for q in qs:
        bt.q.copy_(q)
        cache.rq_paged_append(0, *new, bt.table, bt.kv_lens, cu_new=bt.cu, q=bt.q, q_out=bt.q, cos_sin=cs)
        got.append(attend(bt, cache, 500, 3, workspace=ws))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cache.read_status(ws) == 0 and cache.read_status() == 0
