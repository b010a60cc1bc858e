"""The paged 16-bit cache on the GPU against plain 64-bit forms: append with
rotation, attention with window and first tokens, attention behind a shared
prefix."""

import math

import pytest
import torch

from paged_helpers import F64, Batch, angles, check, check_lse, reference, rotate
from quantized_decode_attention_head_b200 import PagedKVCache

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def make(bt):
    return PagedKVCache(bt.k_pages, bt.v_pages, bt.hq)


def attend(bt, cache, window=0, n_sink=0, **kw):
    a = dict(cu_new=bt.cu, max_new=bt.max_new, window=window, n_sink=n_sink)
    a.update(kw)
    if bt.prefix:
        return cache.rq_paged_shared_attention(bt.layer, bt.q, bt.prefix_pages, bt.prefix, bt.table, bt.kv_lens, **a)
    return cache.rq_paged_attention(bt.layer, bt.q, bt.table, bt.kv_lens, **a)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,hq,hkv,d,page", [(BF, 8, 4, 64, 16), (FP, 8, 1, 128, 32), (BF, 4, 4, 128, 64), (FP, 2, 2, 64, 128)])
@pytest.mark.parametrize("rot,interleaved,axes", [(1.0, False, 1), (0.5, False, 3), (1.0, True, 1), (0.5, True, 4), (0, False, 1)])
def test_append_rotates_and_places(dtype, hq, hkv, d, page, rot, interleaved, axes):
    lens = [(37, 5), (1, 1), (200, 130), (0, 0), (page + 1, 2), (page, page)]
    bt = Batch(lens, hq, hkv, d, page, dtype, seed=d + page, layers=2, layer=1)
    rot = int(rot * d)
    g = torch.Generator().manual_seed(1)
    k_new, v_new = (torch.randn((bt.total, hkv, d), generator=g).to(dtype).cuda() for _ in range(2))
    want_k, want_v = bt.k_pages.clone(), bt.v_pages.clone()
    place = torch.cat([torch.arange(kv - n, kv) for kv, n in lens]).cuda()
    seq = torch.cat([torch.full((n,), b) for b, (_, n) in enumerate(lens)]).long().cuda()
    kw = {}
    want_q = None
    if rot:
        cs = angles(301, rot)
        half = rot // 2
        pos = place[None].expand(axes, -1)
        if axes > 1:
            pos = torch.randint(0, 301, (axes, bt.total), generator=g, dtype=torch.int32).cuda()
            sections = [half // 4, 0, half - half // 4 - 1, 1][:axes]
            sections[-1] = half - sum(sections[:-1])
            kw = dict(positions=pos, sections=sections)
        else:
            sections = [half]
        axis = torch.repeat_interleave(torch.arange(axes), torch.tensor(sections)).cuda()
        at = pos.long()[axis].T
        j = torch.arange(half, device="cuda")
        cos, sin = cs[at, j], cs[at, half + j]
        want_q = rotate(bt.q, cos, sin, interleaved, rot).to(dtype)
        rk = rotate(k_new, cos, sin, interleaved, rot)
        kw.update(q=bt.q, cos_sin=cs, interleaved=interleaved)
        # the rounded fp32 form itself against 64 bits: two products and a
        # difference, each off by 2^-24 of |a c| + |b s| at most, then one rounding
        ex = rotate(k_new, cos, sin, interleaved, rot, F64)
        room = rotate(k_new.abs(), cos.abs(), -sin.abs(), interleaved, rot, F64).abs() + ex.abs() + k_new.abs() * 2
        assert ((rk.to(F64) - ex).abs() <= 2.0**-22 * room).all()
        rk = rk.to(dtype)
    else:
        rk = k_new
    page_of = bt.table[seq, place // page].long()
    want_k[1][page_of, :, place % page] = rk
    want_v[1][page_of, :, place % page] = v_new
    cache = make(bt)
    got_q = cache.rq_paged_append(1, k_new, v_new, bt.table, bt.kv_lens, cu_new=bt.cu, **kw)
    assert torch.equal(bt.k_pages, want_k) and torch.equal(bt.v_pages, want_v)
    assert (got_q is None) if want_q is None else torch.equal(got_q, want_q)
    assert cache.read_status() == 0


def test_append_parts_of_one_projection_in_place_and_padding():
    lens = [(9, 9), (30, 4)]
    bt = Batch(lens, 8, 2, 64, 16, BF, seed=3)
    rows = bt.total + 3  # three rows behind the last sequence
    wide = torch.randn((rows, 12, 64), generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    cs = angles(64, 64)
    ref = PagedKVCache(bt.k_pages.clone(), bt.v_pages.clone(), 8)
    want = ref.rq_paged_append(0, k.contiguous(), v.contiguous(), bt.table, bt.kv_lens, cu_new=bt.cu, q=q.contiguous(), cos_sin=cs)
    cache = make(bt)
    got = torch.full((rows, 8, 64), 7.0, dtype=BF, device="cuda")
    assert cache.rq_paged_append(0, k, v, bt.table, bt.kv_lens, cu_new=bt.cu, q=q, q_out=got, cos_sin=cs) is got
    assert torch.equal(got[: bt.total], want[: bt.total]) and (got[bt.total :] == 7.0).all()
    assert torch.equal(cache.k_pages, ref.k_pages) and torch.equal(cache.v_pages, ref.v_pages)
    own = q.contiguous()
    cache.rq_paged_append(0, k, v, bt.table, bt.kv_lens, cu_new=bt.cu, q=own, q_out=own, cos_sin=cs)
    assert torch.equal(own[: bt.total], want[: bt.total])
    assert cache.read_status() == 0


def test_append_leaves_out_what_is_out_of_range():
    bt = Batch([(20, 2), (20, 2), (20, 2), (1, 3)], 4, 2, 64, 16, BF, seed=5)
    bt.table[1, 1] = bt.k_pages.shape[1]  # no such page
    k_new = torch.ones((bt.total, 2, 64), dtype=BF, device="cuda")
    cs = angles(64, 64)
    pos = torch.full((bt.total,), 3, dtype=torch.int32, device="cuda")
    pos[4] = 64  # sequence 2, first token: no such angle
    before = bt.k_pages.clone()
    cache = make(bt)
    q = cache.rq_paged_append(0, k_new, k_new, bt.table, bt.kv_lens, cu_new=bt.cu, q=bt.q, cos_sin=cs, positions=pos)
    assert cache.read_status() == 8
    changed = (bt.k_pages != before).flatten(2).any(2)[0]
    wrote = {int(p) for p in torch.nonzero(changed).flatten()}
    # sequence 0 wrote its second page, sequence 2 too (its second token), sequence 3 its only page (its last token)
    assert wrote == {int(bt.table[0, 1]), int(bt.table[2, 1]), int(bt.table[3, 0])}
    assert (bt.k_pages[0, int(bt.table[2, 1]), :, 2] == before[0, int(bt.table[2, 1]), :, 2]).all()
    assert (q[4] == 0).all() and (q[5] != 0).any() and (q[2] != 0).any()


# ---------------------------------------------------------------- attention
SHAPES = [(BF, 8, 4, 64, 16), (FP, 8, 1, 128, 32), (BF, 4, 4, 128, 64), (FP, 4, 2, 64, 128), (BF, 8, 2, 128, 128)]
LENS = {
    "one token": [(1, 1), (33, 1), (0, 1), (128, 1), (700, 1), (129, 1), (64, 1)],
    "one sequence": [(2111, 1)],
    "drafts": [(5, 4), (130, 2), (600, 3), (4, 4), (0, 0), (257, 1)],
    "pieces": [(40, 40), (500, 1), (300, 77), (513, 130), (9, 9), (0, 1), (640, 256)],
    "prompt": [(385, 385)],
}
WINDOWS = [(0, 0), (64, 0), (100, 4), (1, 0), (33, 130), (5000, 7)]


@pytest.mark.parametrize("what", list(LENS))
@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention(shape, what, window, n_sink):
    dtype, hq, hkv, d, page = shape
    bt = Batch(LENS[what], hq, hkv, d, page, dtype, seed=len(what) + window)
    ref = reference(bt, window, n_sink)
    bt.poison(window, n_sink)
    cache = make(bt)
    lse = torch.empty((bt.rows, hq), device="cuda")
    ws = cache.make_workspace(len(bt.lens), bt.rows)
    for _ in range(2):  # the workspace serves again
        got = attend(bt, cache, window, n_sink, lse=lse, workspace=ws)
        check(bt, got, ref, what)
        check_lse(bt, lse, ref, what)
    assert cache.read_status(ws) == 0


@pytest.mark.parametrize("what,lens", [
    ("tokens", [(1, 1), (33, 1), (0, 1), (150, 1), (7, 1)]), ("drafts", [(4, 4), (77, 2), (3, 3)]),
    ("pieces", [(200, 90), (41, 1), (5, 5), (140, 140)]), ("many", [(3 + i % 5, 1) for i in range(70)])])
@pytest.mark.parametrize("prefix", [1, 129, 515, 1024])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (64, 4), (300, 200), (2000, 1)])
@pytest.mark.parametrize("shape", SHAPES[:4], ids=str)
def test_shared_prefix(shape, what, lens, prefix, window, n_sink):
    dtype, hq, hkv, d, page = shape
    bt = Batch(lens, hq, hkv, d, page, dtype, seed=prefix + window, prefix=prefix)
    ref = reference(bt, window, n_sink)
    bt.poison(window, n_sink)
    cache = make(bt)
    lse = torch.empty((bt.rows, hq), device="cuda")
    ws = cache.make_workspace(len(bt.lens), bt.rows)
    got = attend(bt, cache, window, n_sink, lse=lse, workspace=ws)
    check(bt, got, ref, what)
    check_lse(bt, lse, ref, what)
    assert cache.read_status(ws) == 0


@pytest.mark.parametrize("prefix", [0, 300])
def test_more_sequences_than_a_block_scans(prefix):
    """The line of work spans several blocks of 128 sequences, empty and long ones among them."""
    lens = [((i * 37) % 150 if i % 11 else 0, 1) for i in range(300)]
    lens[205] = (2500, 1)
    bt = Batch(lens, 8, 2, 64, 16, BF, seed=23, prefix=prefix)
    cache = make(bt)
    ws = cache.make_workspace(300, bt.rows)
    check(bt, attend(bt, cache, workspace=ws), reference(bt))
    assert cache.read_status(ws) == 0


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("lens", [[(70, 1), (9, 1)], [(300, 150), (20, 3), (1, 1)]])
def test_strided_queries_padding_scale_and_layer(lens, prefix):
    bt = Batch(lens, 8, 2, 128, 32, BF, seed=8, layers=3, layer=2, extra_rows=5, prefix=prefix)
    wide = torch.randn((bt.rows, 12, 128), generator=torch.Generator().manual_seed(9)).to(BF).cuda()
    bt.q = wide[:, :8]
    ref = reference(bt, scale=0.3)
    out = torch.full((bt.rows, 8, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((bt.rows, 8), 7.0, device="cuda")
    got = attend(bt, make(bt), softmax_scale=0.3, out=out, lse=lse)
    assert got is out
    check(bt, out, ref)
    check_lse(bt, lse, ref)
    assert (out[bt.total :] == 7.0).all() and (lse[bt.total :] == 7.0).all()


@pytest.mark.parametrize("lens", [[(100, 1), (100, 1)], [(100, 60), (100, 60)]])
def test_bad_pages_and_lengths_are_not_seen(lens):
    """A page that does not exist, and a length past the table: the tokens
    there are not seen, the others are, and the status says so."""
    bt = Batch(lens, 4, 2, 64, 16, BF, seed=11)
    cache = make(bt)
    ws = cache.make_workspace(2, bt.rows)
    good = attend(bt, cache, workspace=ws)
    assert cache.read_status(ws) == 0
    bt.table[1, 2] = -5
    bt.table[1, 3] = 1 << 30
    got = attend(bt, cache, workspace=ws)
    assert cache.read_status(ws) == 8
    n = lens[0][1]
    assert torch.equal(got[:n], good[:n])
    # sequence 1 without tokens 32..63
    g = bt.hq // bt.hkv
    k, v = (_held(bt, x) for x in (bt.k_pages, bt.v_pages))
    p = torch.arange(100 - n, 100, device="cuda")[:, None]
    j = torch.arange(100, device="cuda")
    see = (j <= p) & ((j < 32) | (j >= 64))
    for h in range(bt.hq):
        x = (bt.q[n:, h].to(F64) @ k[h // g].T / 8.0).masked_fill(~see, -math.inf)
        want = torch.softmax(x, 1) @ v[h // g]
        assert (got[n:, h].to(F64) - want).abs().max() <= 3 * 2.0**-8 * v.abs().max()
    bt.kv_lens[1] = 1 << 20
    attend(bt, cache, workspace=ws)
    assert cache.read_status(ws) == 8


@pytest.mark.parametrize("lens", [[(40, 1), (40, 1), (40, 1)], [(60, 30), (60, 30), (60, 30)]])
def test_offsets_out_of_order_stay_inside_the_tensors(lens):
    """Offsets past the packed rows, negative or decreasing: flagged, rows of
    whole sequences right, the rows behind left as they were."""
    bt = Batch(lens, 4, 2, 64, 16, BF, seed=29)
    cache = make(bt)
    ws = cache.make_workspace(3, bt.rows)
    good = attend(bt, cache, workspace=ws)
    n = lens[0][1]
    out = torch.full_like(good, 7.0)
    bt.cu[2], bt.cu[3] = 5 * n, 1  # sequence 1 runs past the end, sequence 2 goes back
    attend(bt, cache, out=out, workspace=ws)
    assert cache.read_status(ws) == 8
    assert torch.equal(out[:n], good[:n]) and torch.isfinite(out.float()).all()
    new = torch.ones((bt.total, 2, 64), dtype=BF, device="cuda")
    cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, cu_new=bt.cu)
    assert cache.read_status() == 8


def test_one_workspace_for_batches_of_all_kinds():
    """A workspace made for the largest batch serves others in turn: many
    sequences, one, prompts, a shared prefix."""
    kinds = [([(700, 1)] * 40, 0), ([(3000, 1)], 0), ([(300, 300), (9, 1)], 0), ([(50, 1)] * 20, 600), ([(2000, 2)] * 3, 0)]
    bts = [Batch(lens, 8, 2, 64, 32, FP, seed=31 + i, prefix=p) for i, (lens, p) in enumerate(kinds)]
    refs = [reference(b) for b in bts]
    caches = [make(b) for b in bts]
    ws = caches[0].make_workspace(40, 301)
    for _ in range(3):
        for b, c, r in zip(bts, caches, refs):
            check(b, attend(b, c, workspace=ws), r)
    assert caches[0].read_status(ws) == 0


def _held(bt, pages):
    t = bt.table[1].long().clamp(0, pages.shape[1] - 1)
    return pages[0][t].transpose(0, 1).reshape(bt.hkv, -1, bt.d)[:, :100].to(F64)


def test_captured_calls_follow_the_device_tensors():
    """A graph of append and attention, replayed after the lengths moved on:
    eight tokens of three sequences, against the same steps run one by one."""
    lens = [(17, 1), (60, 1), (127, 1)]
    steps = 8
    room = [(kv + steps, 1) for kv, _ in lens]
    bt = Batch(room, 8, 4, 128, 16, BF, seed=13)
    bt.lens = lens
    g = torch.Generator().manual_seed(14)
    toks = [[torch.randn((3, h, 128), generator=g).to(BF).cuda() for h in (4, 4, 8)] for _ in range(steps)]
    cs = angles(256, 128)
    start = torch.tensor([kv for kv, _ in lens], dtype=torch.int32, device="cuda")

    def step(cache, kv_lens, k, v, q, ws):
        qr = cache.rq_paged_append(0, k, v, bt.table, kv_lens, q=q, cos_sin=cs)
        return cache.rq_paged_attention(0, qr, bt.table, kv_lens, window=90, n_sink=2, workspace=ws)

    plain = PagedKVCache(bt.k_pages.clone(), bt.v_pages.clone(), 8)
    ws = plain.make_workspace(3, 3)
    want = [step(plain, start + i, *toks[i], ws) for i in range(steps)]
    cache = make(bt)
    ws2 = cache.make_workspace(3, 3)
    lens_t = start.clone()
    ins = [t.clone() for t in toks[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, lens_t, *ins, ws2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, lens_t, *ins, ws2)
    for i in range(steps):
        lens_t.copy_(start + i)
        for a, b in zip(ins, toks[i]):
            a.copy_(b)
        graph.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(cache.k_pages, plain.k_pages)
    # and the last step against 64 bits
    bt.lens = [(kv + steps - 1, 1) for kv, _ in lens]
    half = 64
    pos = (start + steps - 2).long()  # the place of the last step's token
    bt.q = rotate(toks[-1][2], cs[pos, :half], cs[pos, half:], False, 128).to(BF)
    check(bt, want[-1], reference(bt, 90, 2))


def test_another_stream_and_its_own_workspace():
    bts = [Batch([(900, 1), (50, 1)], 8, 4, 128, 64, BF, seed=s) for s in (15, 16)]
    refs = [reference(b) for b in bts]
    caches = [make(b) for b in bts]
    streams = [torch.cuda.Stream() for _ in bts]
    wss = [c.make_workspace(2, 2) for c in caches]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for b, c, s, w in zip(bts, caches, streams, wss):
            outs.append(attend(b, c, workspace=w, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        check(bts[i % 2], o, refs[i % 2])


def test_prompt_appended_then_read_token_by_token():
    """A prompt in pieces and single tokens, appended and attended as a server
    does, equals one pass over the whole."""
    n, d, page = 210, 64, 32
    g = torch.Generator().manual_seed(17)
    k, v, q = (torch.randn((n, h, d), generator=g).to(FP).cuda() for h in (2, 2, 4))
    cs = angles(n, d)

    def serve(pieces):
        pages = [torch.zeros((1, 9, 2, page, d), dtype=FP, device="cuda") for _ in range(2)]
        cache = PagedKVCache(*pages, 4)
        table = torch.tensor([[5, 0, 7, 2, 3, 8, 1]], dtype=torch.int32, device="cuda")
        ws = cache.make_workspace(1, n)
        outs, at = [], 0
        for m in pieces:
            lens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
            cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            sl = slice(at, at + m)
            qr = cache.rq_paged_append(0, k[sl], v[sl], table, lens, cu_new=cu, q=q[sl], cos_sin=cs)
            outs.append(cache.rq_paged_attention(0, qr, table, lens, cu_new=cu, window=70, n_sink=3, workspace=ws))
            at += m
        assert cache.read_status(ws) == 0 and cache.read_status() == 0
        return torch.cat(outs), pages

    whole, pages = serve([n])
    parts, pages2 = serve([100, 1, 1, 4, 50, 1, 53])
    assert torch.equal(pages[0], pages2[0]) and torch.equal(pages[1], pages2[1])
    # both are within the tolerance of the same 64-bit values
    bt = Batch([(n, n)], 4, 2, d, page, FP)
    bt.k_pages, bt.v_pages = pages
    bt.table = torch.tensor([[5, 0, 7, 2, 3, 8, 1]], device="cuda")
    bt.q = rotate(q, cs[:, :32], cs[:, 32:], False, d).to(FP)
    ref = reference(bt, 70, 3)
    check(bt, whole, ref)
    check(bt, parts, ref)


def test_offsets_past_32_bits():
    """Pages at the far end of a cache of more than 2^32 bytes and 2^31 values."""
    hkv, page, d = 8, 128, 128
    n_pages = (2**31) // (hkv * page * d) + 40
    k_pages = torch.zeros((1, n_pages, hkv, page, d), dtype=BF, device="cuda")
    v_pages = torch.zeros_like(k_pages)
    bt = Batch([(300, 1), (200, 150)], 16, hkv, d, page, BF, seed=19)
    shift = n_pages - bt.k_pages.shape[1]
    k_pages[:, shift:], v_pages[:, shift:] = bt.k_pages, bt.v_pages
    ref = reference(bt)
    bt.table = torch.where(bt.table >= 0, bt.table + shift, bt.table)
    cache = PagedKVCache(k_pages, v_pages, 16)
    check(bt, attend(bt, cache), ref)
    new = torch.ones((bt.total, hkv, d), dtype=BF, device="cuda")
    cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, cu_new=bt.cu)
    assert (k_pages[0, int(bt.table[0, 2]), :, 299 - 256] == 1).all() and cache.read_status() == 0


def test_python_refusals():
    bt = Batch([(20, 1), (5, 1)], 4, 2, 64, 16, BF)
    cache = make(bt)
    ok = dict(q=bt.q, page_table=bt.table, kv_lens=bt.kv_lens)
    for bad, err in ((dict(q=bt.q.half()), TypeError), (dict(q=bt.q[:, :3]), ValueError), (dict(q=bt.q.cpu()), ValueError),
                     (dict(q=bt.q[:1]), ValueError), (dict(page_table=bt.table.long()), TypeError),
                     (dict(page_table=bt.table[0]), ValueError), (dict(kv_lens=bt.kv_lens[:1]), ValueError),
                     (dict(q=bt.q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            cache.rq_paged_attention(0, **{**ok, **bad})
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        cache.rq_paged_attention(1, **ok)
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        cache.rq_paged_attention(0, **ok, window=-1)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        cache.rq_paged_attention(0, **ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="do not hold"):
        cache.rq_paged_shared_attention(0, bt.q, bt.table[0, :1].contiguous(), 17, bt.table, bt.kv_lens)
    with pytest.raises(ValueError, match="go with cos_sin"):
        cache.rq_paged_append(0, bt.q[:, :2], bt.q[:, :2], bt.table, bt.kv_lens, q=bt.q)
