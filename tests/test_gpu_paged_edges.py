"""The paged 16-bit cache on the GPU where callers leave the usual path: other
streams, lengths past the table, freed pages, weights of very different size."""

import ctypes
import math

import pytest
import torch

from paged_helpers import F64, Batch, angles, check, check_lse, reference, rotate
from quantized_decode_attention_head_b200 import PagedKVCache, QuantizedKVCache, _lib
from quantized_decode_attention_head_b200.api import rq_measure_distortion

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


# ------------------------------------------------------------------ streams
def stream_of(address):
    """The stream whose memory the allocator counts this address to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= address < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not memory of the allocator")


def test_what_a_call_allocates_is_memory_of_its_stream():
    bt = Batch([(900, 1), (50, 1)], 8, 4, 128, 64, BF, seed=15)
    cache = make(bt)
    used = []

    def spy(fn):
        def call(*args):
            used.append(args[-3])  # the workspace
            return fn(*args)
        return call

    cache._attention_fns = tuple(spy(f) for f in cache._attention_fns)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = attend(bt, cache, stream=s)
    assert stream_of(out.data_ptr()) == stream_of(used[-1]) == s.cuda_stream
    new = torch.ones((2, 4, 128), dtype=BF, device="cuda")
    q = cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, q=bt.q, cos_sin=angles(1000, 128), stream=s)
    assert stream_of(q.data_ptr()) == s.cuda_stream
    assert stream_of(cache.make_workspace(2, 2, stream=s).data_ptr()) == s.cuda_stream
    torch.cuda.synchronize()
    here = attend(bt, cache)
    assert stream_of(here.data_ptr()) == stream_of(used[-1]) == torch.cuda.current_stream().cuda_stream
    # the quantized cache likewise
    old = QuantizedKVCache(1, 1, 4, 2, 64, 0, 32, 128, [[4, 4]], [[4, 4]])
    assert stream_of(old.make_workspace(stream=s).data_ptr()) == s.cuda_stream
    k = torch.randn((1, 1, 2, 64, 64), device="cuda").to(BF)
    torch.cuda.synchronize()
    old.rq_quantize_kv(k, k, stream=s)
    qq = torch.randn((1, 4, 64), device="cuda").to(BF)
    torch.cuda.synchronize()
    assert stream_of(old.rq_decode_attention(0, qq, stream=s).data_ptr()) == s.cuda_stream
    kn = k[0, :, :, 0].contiguous()
    torch.cuda.synchronize()
    assert stream_of(old.rq_decode_step(0, qq, kn, kn, stream=s).data_ptr()) == s.cuda_stream
    torch.cuda.synchronize()


def test_two_streams_without_a_workspace():
    """Long sequences, split and counted in the workspace, on two streams in
    turn, while the current stream takes and fills memory of the same size."""
    bts = [Batch([(4000, 1), (50, 1)], 8, 4, 128, 64, BF, seed=s) for s in (15, 16)]
    bts.append(Batch([(30, 1), (200, 150)], 8, 4, 128, 64, BF, seed=17, prefix=1500))
    refs = [reference(b) for b in bts]
    caches = [make(b) for b in bts]
    streams = [torch.cuda.Stream() for _ in bts]
    sizes = [c.rq_paged_workspace_bytes(2, b.rows) for c, b in zip(caches, bts)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for b, c, s, n in zip(bts, caches, streams, sizes):
            outs.append(attend(b, c, stream=s))
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xA5)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        check(bts[i % 3], o, refs[i % 3])


def test_distortion_measured_on_another_stream():
    x = torch.randn((3, 256, 64), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    want = rq_measure_distortion(x, "K", [2, 4])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the measurement waits behind this
    got = rq_measure_distortion(x, "K", [2, 4], stream=s)
    # the kernel adds 256 * 64 / 32 = 512 positive group sums in the order they
    # arrive: each of 512 additions is off by 2^-53 of the sum at most, in both runs
    assert (abs(got - want) <= 2 * 512 * 2.0**-53 * want).all()


# ------------------------------------------------------------------- status
@pytest.mark.parametrize("lens,prefix", [([(100, 1), (100, 1)], 0), ([(100, 60), (100, 60)], 0), ([(40, 1)], 200)])
def test_a_timeout_is_not_replaced_by_an_index(lens, prefix):
    """A wait that gave up stays in the status word when a later call of the
    workspace meets a page that does not exist."""
    bt = Batch(lens, 4, 2, 64, 16, BF, seed=11, prefix=prefix)
    cache = make(bt)
    ws = cache.make_workspace(2, bt.rows)
    bt.table[0, 1] = 1 << 30
    attend(bt, cache, workspace=ws)
    assert cache.read_status(ws) == 8
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _lib.lib().rq_decode_workspace_init(ctypes.c_void_p(ws.data_ptr()), ws.numel(), stream) == 0
    assert _lib.lib().rq_selftest_device_timeout(ctypes.c_void_p(ws.data_ptr()), ws.numel(), 2_000_000, stream) == 0
    torch.cuda.synchronize()
    assert cache.read_status(ws) == 7
    attend(bt, cache, workspace=ws)
    assert cache.read_status(ws) == 7


# ----------------------------------------------------- lengths and offsets
@pytest.mark.parametrize("positions", [False, True])
def test_append_past_the_table_keeps_what_is_there(positions):
    """Lengths past the table, and far from it: tokens whose place lies in the
    table are written there, the others nowhere."""
    bt = Batch([(32, 1), (32, 5), (32, 3), (20, 2), (32, 2), (32, 2)], 4, 2, 64, 16, BF, seed=51)
    lens = [33, 35, 40, 20, 2**31 - 1, -(2**31)]
    bt.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    g = torch.Generator().manual_seed(52)
    k, v = (torch.randn((bt.total, 2, 64), generator=g).to(BF).cuda() for _ in range(2))
    cs = angles(64, 64)
    kw = dict(positions=torch.arange(bt.total, dtype=torch.int32, device="cuda")) if positions else {}
    want_k, want_v = bt.k_pages.clone(), bt.v_pages.clone()
    want_q = torch.zeros_like(bt.q)
    t = 0
    for b, (_, n) in enumerate(bt.lens):
        for i in range(n):
            at = lens[b] - n + i
            p = t if positions else at
            if 0 <= p < 64:
                c, s = cs[p, :32][None], cs[p, 32:][None]
                want_q[t] = rotate(bt.q[t : t + 1], c, s, False, 64).to(BF)[0]
                if 0 <= at < 32:
                    page = int(bt.table[b, at // 16])
                    want_k[0, page, :, at % 16] = rotate(k[t : t + 1], c, s, False, 64).to(BF)[0]
                    want_v[0, page, :, at % 16] = v[t]
            t += 1
    cache = make(bt)
    q = cache.rq_paged_append(0, k, v, bt.table, bt.kv_lens, cu_new=bt.cu, q=bt.q, cos_sin=cs, **kw)
    assert cache.read_status() == 8
    assert torch.equal(bt.k_pages, want_k) and torch.equal(bt.v_pages, want_v) and torch.equal(q, want_q)


@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (30, 3)])
@pytest.mark.parametrize("prefix", [0, 150])
def test_attention_past_the_table_sees_what_is_there(n, window, n_sink, prefix):
    """A length past the table: its queries stand where the length puts them
    and see the keys that the table holds; other sequences are as ever."""
    bt = Batch([(64, n), (64, n)], 4, 2, 64, 16, BF, seed=53, prefix=prefix)
    bt.kv_lens[1] = 64 + 7
    cache = make(bt)
    ws = cache.make_workspace(2, bt.rows)
    got = attend(bt, cache, window, n_sink, workspace=ws)
    assert cache.read_status(ws) == 8
    k, v = bt.held(bt.k_pages, 1), bt.held(bt.v_pages, 1)
    p = prefix + 71 - n + torch.arange(n, device="cuda")[:, None]
    j = torch.arange(prefix + 64, device="cuda")
    see = j <= p
    if window:
        see &= (p - j < window) | (j < n_sink)
    for h in range(4):
        x = (bt.q[n:, h].to(F64) @ k[h // 2].T / 8.0).masked_fill(~see, -math.inf)
        w = torch.softmax(x, 1)
        # one rounding of each weight and one of the result (2^-8 each), sums and exponentials far below
        tol = 2.0**-8 * 1.01 * (w @ v[h // 2]).abs() + 2.0**-8 * 1.01 * (w @ v[h // 2].abs())
        assert ((got[n:, h].to(F64) - w @ v[h // 2]).abs() <= tol).all(), h
    bt.kv_lens[1] = 64
    same = attend(bt, cache, window, n_sink, workspace=ws)
    assert torch.equal(got[:n], same[:n])
    # as far as a length goes, and below zero
    bt.kv_lens[1] = 2**31 - 1
    far = attend(bt, cache, 0, 0, workspace=ws)
    bt.kv_lens[1] = -(2**31)
    none = attend(bt, cache, window, n_sink, workspace=ws)
    bt.kv_lens[1] = 64 + n
    every = attend(bt, cache, 0, 0, workspace=ws)
    assert torch.equal(far[n:], every[n:]) and torch.equal(none[:n], same[:n])
    assert prefix or (none[n:] == 0).all()


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("cu,bad", [([0, 1, 2, 4], 2), ([-1, 1, 2, 3], 0)])
def test_a_sequence_whose_offsets_leave_the_rows_has_no_new_tokens(n, cu, bad):
    """Offsets in units of n rows of three sequences, one reaching outside:
    nothing of it is written, the others are as ever."""
    bt = Batch([(60, n)] * 3, 4, 2, 64, 16, BF, seed=55)
    cache = make(bt)
    ws = cache.make_workspace(3, bt.rows)
    good = attend(bt, cache, workspace=ws)
    bt.cu.copy_(torch.tensor([n * x for x in cu], dtype=torch.int32))
    out = torch.full_like(good, 7.0)
    attend(bt, cache, out=out, workspace=ws)
    assert cache.read_status(ws) == 8
    for b in range(3):
        rows = slice(b * n, b * n + n)
        assert torch.equal(out[rows], good[rows]) if b != bad else (out[rows] == 7.0).all()
    new = torch.ones((bt.total, 2, 64), dtype=BF, device="cuda")
    before = bt.k_pages.clone()
    cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, cu_new=bt.cu)
    assert cache.read_status() == 8
    for b in range(3):
        pages = bt.table[b].long()
        same = (bt.k_pages[0, pages] == before[0, pages]).all()
        assert bool(same) == (b == bad)


# -------------------------------------------------------------- freed pages
def free_unseen(bt, window, n_sink):
    """Table entries of pages that no query of the sequence sees become page
    numbers that do not exist; those of the prefix where no sequence does."""
    pre = torch.zeros(len(bt.prefix_pages), dtype=torch.bool)
    for b, (kv, n) in enumerate(bt.lens):
        seen = bt.seen(b, window, n_sink).any(0).cpu() if n else torch.zeros(bt.prefix + kv, dtype=torch.bool)
        for j in torch.nonzero(seen[: bt.prefix]).flatten().tolist():
            pre[j // bt.page] = True
        own = seen[bt.prefix :]
        for i in range(-(-kv // bt.page)):
            if not own[i * bt.page : (i + 1) * bt.page].any():
                bt.table[b, i] = -1 if i % 2 else 1 << 30
    bt.prefix_pages[~pre.to(bt.prefix_pages.device)] = -7


@pytest.mark.parametrize("lens,prefix", [
    ([(700, 1), (300, 2), (40, 1)], 0), ([(700, 200), (555, 90), (129, 129)], 0), ([(1000, 300)], 0),
    ([(90, 1), (40, 1)], 1000), ([(333, 120), (40, 40), (9, 1)], 700)])
@pytest.mark.parametrize("window,n_sink", [(100, 0), (70, 4), (33, 130), (1, 0), (1, 17), (400, 20)])
@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (64, 64)])
def test_pages_freed_behind_the_window(lens, prefix, window, n_sink, page, d):
    bt = Batch(lens, 8, 2, d, page, BF, seed=61 + page, prefix=prefix)
    ref = reference(bt, window, n_sink)
    bt.poison(window, n_sink)
    free_unseen(bt, window, n_sink)
    cache = make(bt)
    lse = torch.empty((bt.rows, 8), device="cuda")
    ws = cache.make_workspace(len(lens), bt.rows)
    check(bt, attend(bt, cache, window, n_sink, lse=lse, workspace=ws), ref)
    check_lse(bt, lse, ref)
    assert cache.read_status(ws) == 0


# ----------------------------------------------- weights of very different size
@pytest.mark.parametrize("keys,new,prefix,seqs", [
    (131072, 1, 0, 1), (40000, 3, 0, 1), (2000, 1, 0, 400), (40000, 40, 0, 1), (20, 1, 30000, 3), (300, 90, 20000, 1)])
@pytest.mark.parametrize("below", [20.0, 25.6, 28.0])
def test_one_key_outweighs_a_long_tail_in_fp16(keys, new, prefix, seqs, below):
    """The first key's weight is about 2^below times that of any other: the
    others count in the sum, so they have to count in the product.  With many
    sequences (the same pages for all) no sequence's keys are divided among
    blocks, so that one running maximum holds for most of them.

    Weights are held to 2^-11 relative (twice that far in two terms) or, where
    that is more, to half the smallest step of fp16, 2^-25, at the factor that
    they are held larger by: 2^14 in two terms, 2^6 at least in one (more than
    16 rows a kv head, or over a prefix); the result is rounded once.  Scores
    and exponentials add 2^-17 (68 products of at most 2^5 at 2^-23)."""
    d, hq, hkv = 64, 4, 2
    bt = Batch([(keys, new)], hq, hkv, d, 64, FP, seed=71, prefix=prefix)
    g = torch.Generator().manual_seed(72)
    total = prefix + keys
    bt.table = bt.table.expand(seqs, -1).contiguous()
    bt.kv_lens = bt.kv_lens.expand(seqs).contiguous()
    bt.cu = torch.arange(0, (seqs + 1) * new, new, dtype=torch.int32, device="cuda")
    bt.q = bt.q.repeat(seqs, 1, 1)
    # q = 4 e_0 plus a little in channel 1; key 0 has its score in channel 0, the others none there
    bt.q.zero_()
    bt.q[..., 0] = 4.0
    bt.q[..., 1] = 0.25 * torch.rand((seqs * new, hq), generator=g).to(FP).cuda()
    top = below * math.log(2.0) / 4.0 * 8.0  # scale 1/8: the score is below * ln 2
    k = torch.zeros((hkv, total, d), dtype=FP)
    k[:, :, 1] = torch.randn((hkv, total), generator=g).to(FP)
    k[:, 0] = 0.0
    k[:, 0, 0] = top
    v = 0.5 + torch.rand((hkv, total, d), generator=g)
    v[:, 0] = torch.randn((hkv, d), generator=g) * 2.0**-12
    v = v.to(FP)
    for pages, rows in ((bt.k_pages, k), (bt.v_pages, v)):
        place(bt, pages, rows)
    floor = 2.0**-39 if prefix == 0 and 2 * new <= 16 else 2.0**-31
    lse = torch.empty((seqs * new, hq), device="cuda")
    cache = make(bt)
    got = attend(bt, cache, lse=lse).to(F64)
    k, v = k.cuda().to(F64), v.cuda().to(F64)
    p = total - new + torch.arange(new, device="cuda")[:, None]
    see = (torch.arange(total, device="cuda") <= p).repeat(seqs, 1)
    for h in range(hq):
        x = (bt.q[:, h].to(F64) @ k[h // 2].T / 8.0).masked_fill(~see, -math.inf)
        w = torch.softmax(x, 1)
        out, a = w @ v[h // 2], w @ v[h // 2].abs()
        tol = 2.0**-11 * 1.01 * (out.abs() + a) + 2.0**-17 * a + total * floor * 1.5 + 2.0**-25
        err = (got[:, h] - out).abs()
        assert (err <= tol).all(), f"{float((err / tol).max()):.2f} times the tolerance"
        assert ((lse[:, h].to(F64) - torch.logsumexp(x, 1)).abs() <= 2.0**-17).all()


def place(bt, pages, rows):
    """rows [kv heads, prefix + keys, d] of the batch's only sequence, into its pages."""
    pre, own = rows[:, : bt.prefix], rows[:, bt.prefix :]
    for part, numbers in ((pre, bt.prefix_pages), (own, bt.table[0])):
        n = part.shape[1]
        if n:
            full = torch.zeros((bt.hkv, -(-n // bt.page) * bt.page, bt.d), dtype=rows.dtype)
            full[:, :n] = part
            blocks = full.view(bt.hkv, -1, bt.page, bt.d).transpose(0, 1)
            pages[0, numbers[: blocks.shape[0]].long()] = blocks.to(pages.device)


# ------------------------------------------- how the SMs and keys are divided
@pytest.mark.parametrize("lens,prefix", [
    ([(40 + 37 * i % 300, 1) for i in range(24)], 9000), ([(300, 2)] * 5, 2000), ([(3000, 1)] * 40, 700),
    ([(20 + i % 90, 1) for i in range(300)], 5000), ([(0, 1), (0, 1)], 4000)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (600, 4)])
def test_a_wider_table_changes_nothing(lens, prefix, window, n_sink):
    """A captured call keeps its table at the longest length it may meet: the
    division of the SMs between the prefix and what follows it goes by the
    lengths, so results are the same bit for bit."""
    bt = Batch(lens, 8, 2, 64, 16, BF, seed=81, prefix=prefix)
    ref = reference(bt, window, n_sink)
    cache = make(bt)
    ws = cache.make_workspace(len(lens), bt.rows)
    got = []
    for wide in (1, 16, 300):
        table = torch.full((len(lens), wide * bt.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        table[:, : bt.table.shape[1]] = bt.table
        lse = torch.empty((bt.rows, 8), device="cuda")
        out = cache.rq_paged_shared_attention(0, bt.q, bt.prefix_pages, prefix, table, bt.kv_lens, cu_new=bt.cu,
                                              max_new=bt.max_new, window=window, n_sink=n_sink, lse=lse, workspace=ws)
        check(bt, out, ref)
        check_lse(bt, lse, ref)
        got.append((out, lse))
    assert cache.read_status(ws) == 0
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("kv", [30, 400])
def test_a_prefix_that_fills_the_device(n, kv):
    """More blocks of rows over the prefix than SMs: nothing is split, and what
    follows the prefix has all SMs."""
    lens = [(max(n, (i * 7) % kv), n) for i in range(700 // n)]
    bt = Batch(lens, 64, 8, 64, 16, BF, seed=83, prefix=300)
    ref = reference(bt)
    cache = make(bt)
    lse = torch.empty((bt.rows, 64), device="cuda")
    ws = cache.make_workspace(len(lens), bt.rows)
    for _ in range(2):
        check(bt, attend(bt, cache, lse=lse, workspace=ws), ref)
        check_lse(bt, lse, ref)
    assert cache.read_status(ws) == 0


def test_a_captured_call_divides_by_the_lengths_it_finds():
    """Replayed with lengths that make the tails a small part, then most of the
    work, and sequences that come and go."""
    lens = [(4000, 1)] * 20
    bt = Batch(lens, 8, 2, 64, 32, BF, seed=82, prefix=3000)
    cache = make(bt)
    ws = cache.make_workspace(20, bt.rows)
    lse = torch.empty((bt.rows, 8), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(bt, cache, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attend(bt, cache, lse=lse, workspace=ws)
    for kv in ([4000] * 20, [5] * 20, [4000] + [0] * 19, [1 + 200 * i for i in range(20)]):
        bt.kv_lens.copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        bt.lens = [(n, 1) for n in kv]
        ref = reference(bt)
        check(bt, out, ref, str(kv[:2]))
        check_lse(bt, lse, ref)
    assert cache.read_status(ws) == 0


# --------------------------------------------------------- long walks and many parts
@pytest.mark.parametrize("what,lens,prefix,hq,hkv", [
    ("prefix in 128 parts", [(50, 1), (9, 1)], 66000, 4, 1),
    ("prefix in many parts, pieces behind it", [(600, 300), (9, 1), (70, 70)], 20000, 8, 2),
    ("one piece, its keys in many parts", [(30000, 40)], 0, 4, 1),
    ("47 tiles in one go", [(6000 - i, 40) for i in range(40)], 0, 4, 4),
    ("one token, its keys in 296 parts", [(100000, 1)], 0, 8, 1),
    ("a prompt of 4000 without a window", [(4000, 4000)], 0, 2, 2)])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)])
def test_many_parts_and_long_walks(what, lens, prefix, hq, hkv, dtype, d):
    bt = Batch(lens, hq, hkv, d, 64, dtype, seed=91, prefix=prefix)
    ref = reference(bt)
    cache = make(bt)
    lse = torch.empty((bt.rows, hq), device="cuda")
    ws = cache.make_workspace(len(lens), bt.rows)
    for _ in range(2):
        check(bt, attend(bt, cache, lse=lse, workspace=ws), ref, what)
        check_lse(bt, lse, ref, what)
    assert cache.read_status(ws) == 0


# ------------------------------------------------ status of calls on other streams
def test_status_reads_wait_for_every_stream():
    """Calls queued on another stream, behind some milliseconds of work, report
    a page that does not exist to a status read that follows at once."""
    bt = Batch([(100, 1), (100, 1)], 4, 2, 64, 16, BF, seed=11)
    cache = make(bt)
    ws = cache.make_workspace(2, bt.rows)
    bt.table[1, 6] = 1 << 30
    new = torch.ones((2, 2, 64), dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    attend(bt, cache, workspace=ws, stream=s)
    assert cache.read_status(ws) == 8
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, stream=s)
    assert cache.read_status() == 8


def test_a_new_cache_serves_another_stream_at_once():
    """The status word of the appends is cleared before the constructor
    returns, however much is queued on the current stream."""
    bt = Batch([(100, 1), (100, 1)], 4, 2, 64, 16, BF, seed=11)
    bt.table[1, 6] = 1 << 30
    new = torch.ones((2, 2, 64), dtype=BF, device="cuda")
    make(bt).rq_paged_append(0, new, new, bt.table, bt.kv_lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    cache = make(bt)
    cache.rq_paged_append(0, new, new, bt.table, bt.kv_lens, stream=s)
    torch.cuda.synchronize()
    assert cache.read_status() == 8


# ------------------------------------------------------------------ refusals
def test_integers_past_32_bits_are_refused():
    """They would reach the C call cut to 32 bits: a window of 2^32 + 10 as 10."""
    bt = Batch([(20, 1), (5, 1)], 4, 2, 64, 16, BF)
    cache = make(bt)
    big = 2**32 + 10
    for kw in (dict(window=big), dict(n_sink=big), dict(max_new=big), dict(window=-big), dict(window=2**31)):
        with pytest.raises(ValueError, match="32 bits"):
            cache.rq_paged_attention(0, bt.q, bt.table, bt.kv_lens, cu_new=bt.cu, **kw)
    for layer in (2**32, -(2**32)):
        with pytest.raises(ValueError, match="32 bits"):
            cache.rq_paged_attention(layer, bt.q, bt.table, bt.kv_lens)
        with pytest.raises(ValueError, match="32 bits"):
            cache.rq_paged_append(layer, bt.q[:, :2], bt.q[:, :2], bt.table, bt.kv_lens)
    with pytest.raises(ValueError, match="32 bits"):
        cache.make_workspace(2**32, 4)
    with pytest.raises(ValueError, match="32 bits"):
        PagedKVCache(bt.k_pages, bt.v_pages, 2**32 + 4)
    with pytest.raises(ValueError, match="32 bits"):
        cache.rq_paged_append(0, bt.q[:, :2], bt.q[:, :2], bt.table, bt.kv_lens, cos_sin=angles(64, 64),
                              sections=[2**32 + 32])
