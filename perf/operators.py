"""What is measured of the paged 16-bit cache: appending with the rotation of
positions, attention with a sliding window and first tokens that stay visible,
and attention of a batch that shares a long prefix.

Shapes (one layer): pages [1, pages, kv heads, page size, head dim] for keys
and for values; a table [sequences, pages per sequence] of page numbers;
``kv_lens`` = tokens of each sequence after the append; queries and new tokens
are packed one sequence behind another, ``cu`` (sequences + 1) marks where each
begins.  Query i of sequence b, which has n_b of them, stands at position
prefix + kv_lens[b] - n_b + i and sees every key at or before it that is less
than ``window`` positions back (no window: all of them) or among the first
``sinks`` positions.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- the cases
def _case(kind, name=None, **kw):
    c = dict(kind=kind, dtype="bf16", hq=32, hkv=8, d=128, page=64, seqs=1, kv=128, new=1, ragged=False, window=0,
             sinks=0, prefix=0, axes=1, rot=0, interleaved=False)
    c.update(kw)
    if not c["rot"]:
        c["rot"] = c["d"]
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one serving step of eight sequences: the call is all latency
        _case("append", "append_step", seqs=8, kv=4096),
        # prompts of several lengths enter the cache together, their positions on three axes (images between text)
        _case("append", "append_prompts", seqs=6, kv=8192, new=8192, ragged=True, axes=3),
        # a small model: half types, short pages, odd lengths, neighbouring channels paired, half of a head rotated
        _case("append", "append_small_model", dtype="fp16", hq=8, hkv=4, d=64, page=16, seqs=3, kv=301, new=77, ragged=True,
              interleaved=True, rot=32),
        # a local layer of a small model, two short sequences: latency again
        _case("attend", "attend_small_model", dtype="fp16", hq=8, hkv=4, d=64, page=16, seqs=2, kv=512, window=128, sinks=4),
        # one decode step of a full batch of different lengths, all tokens visible
        _case("attend", "attend_batch", seqs=64, kv=8192, ragged=True),
        # one decode step of a local layer: long sequences, of which a window and the first tokens are read
        _case("attend", "attend_window", seqs=16, kv=32768, ragged=True, window=4096, sinks=4, page=128),
        # one decode step of one very long sequence: the work has to be split along it
        _case("attend", "attend_long", kv=131072),
        # a scheduler's mixed step: pieces of prompts and single tokens over what is cached already
        _case("attend", "attend_chunks", seqs=5, kv=4099, new=333, ragged=True, window=1000, sinks=3, page=32),
        # a whole prompt through a local layer: bound by the tensor cores
        _case("attend", "attend_prompt", kv=8192, new=8192, window=4096, sinks=4),
        # a small batch behind a short system prompt that ends inside a page
        _case("shared", "shared_small_model", dtype="fp16", hq=8, hkv=4, d=64, page=16, seqs=8, kv=40, ragged=True, prefix=515),
        # a full batch behind one long document
        _case("shared", "shared_document", seqs=64, kv=512, ragged=True, prefix=32768),
        # drafts of four tokens to check behind a shared prompt, in a local layer with first tokens
        _case("shared", "shared_drafts", seqs=16, kv=300, new=4, prefix=8192, window=6000, sinks=4, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "shared", "shared"])
    c = dict(dtype=rng.choice(["bf16", "bf16", "fp16"]), d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    c["hkv"] = rng.choice([1, 2, 4, 8])
    c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 4, 8])
    c["seqs"] = _log(rng, 1, 64)
    c["ragged"] = rng.random() < 0.7
    if kind == "append":
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 32768 // c["seqs"]))
        c["kv"] = c["new"] + _log(rng, 1, 4096)
        c["axes"] = rng.choice([1, 1, 3])
        c["interleaved"] = rng.random() < 0.3
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
        return _case("append", **c)
    c["new"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    # bounded so that the scores of the plain form stay within a few GB and no case passes the largest listed one
    most = 131072 if c["new"] == 1 else max(64, min(16384, 2 ** 28 // (c["hq"] * c["new"] * c["seqs"])))
    if kind == "attend":
        c["kv"] = max(c["new"], _log(rng, 33, max(64, min(most, 524288 // c["seqs"]))))
    else:
        c["prefix"] = _log(rng, 17, max(64, min(most, 32768)))
        c["kv"] = max(c["new"], _log(rng, 1, 1024))
    if rng.random() < 0.5:
        c["window"] = _log(rng, 16, max(64, c["kv"] + c.get("prefix", 0)))
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(5, 200)])
    return _case(kind, **c)


def _lengths(case):
    """(tokens after the append, new tokens) of each sequence: the first has the most, the last of a ragged batch may be empty."""
    r = random.Random("%(seqs)d %(kv)d %(new)d" % case)
    out = []
    for b in range(case["seqs"]):
        kv, n = case["kv"], case["new"]
        if case["ragged"] and b:
            kv = _log(r, max(1, kv // 16), kv)
            n = min(kv, _log(r, 1, n) if n > 1 else 1)
        if case["ragged"] and b >= 2 and b == case["seqs"] - 1 and case["kind"] == "attend" and case["new"] == 1:
            kv = 0  # a free place in the batch: its query sees nothing
        out.append((kv, n))
    return out


def _sections(case):
    """How many channel pairs turn by each axis."""
    half, a = case["rot"] // 2, case["axes"]
    if a == 1:
        return [half]
    first = half // 4
    return [first, (half - first) // 2, half - first - (half - first) // 2]


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, ps, seqs = case["hq"], case["hkv"], case["d"], case["page"], case["seqs"]
    lens = _lengths(case)
    total = sum(n for _, n in lens)
    per_seq = max(1, -(-max(kv for kv, _ in lens) // ps))
    n_prefix = -(-case["prefix"] // ps)
    n_pages = sum(max(1, -(-kv // ps)) for kv, _ in lens) + n_prefix + 2

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    # keys with channels of different magnitudes, the same for a head's tokens
    spread = torch.exp(0.5 * torch.randn(hkv, 1, d, generator=g, device=dev)).to(dt)
    k_pages = normal(1, n_pages, hkv, ps, d).mul_(spread)
    v_pages = normal(1, n_pages, hkv, ps, d)
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    # the pages lie in no order; places of a row behind its last page hold no page
    table = torch.full((seqs, per_seq), -1, dtype=torch.int32)
    at, host = n_prefix, order.cpu()
    for b, (kv, _) in enumerate(lens):
        k = -(-kv // ps)
        table[b, :k] = host[at : at + k]
        at += max(1, k)
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=table.to(dev), max_new=max(n for _, n in lens),
             kv_lens=torch.tensor([kv for kv, _ in lens], dtype=torch.int32, device=dev),
             cu=torch.tensor(cu, dtype=torch.int32, device=dev), prefix_pages=order[:n_prefix].clone(),
             q=normal(total, hq, d))
    if case["kind"] == "append":
        s["k_new"] = normal(total, hkv, d).mul_(spread[:, 0])
        s["v_new"] = normal(total, hkv, d)
        half = case["rot"] // 2
        top = case["kv"] + 8
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["axes"] > 1:
            s["positions"] = torch.randint(0, top, (case["axes"], total), generator=g, device=dev, dtype=torch.int32)
    return s


# ------------------------------------------------------------- the plain forms
def _rows(s):
    """The sequence of each packed token and its place among the sequence's new tokens."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b]


def _rotate(x, cos, sin, case):
    x = x.float()
    half = case["rot"] // 2
    cos, sin = cos[:, None], sin[:, None]
    rot, rest = x[..., : case["rot"]], x[..., case["rot"] :]
    if case["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _plain_append(s):
    case, ps = s["case"], s["case"]["page"]
    b, i = _rows(s)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    place = s["kv_lens"].long()[b] - n[b] + i
    half = case["rot"] // 2
    cos_sin = s["cos_sin"]
    if case["axes"] > 1:
        axis = torch.repeat_interleave(torch.arange(case["axes"], device=b.device),
                                       torch.tensor(_sections(case), device=b.device), output_size=half)
        p = s["positions"].long()[axis].T  # [tokens, pairs]
        j = torch.arange(half, device=b.device)
        cos, sin = cos_sin[p, j], cos_sin[p, half + j]
    else:
        cos, sin = cos_sin[place, :half], cos_sin[place, half:]
    page = s["table"].long()[b, place // ps]
    dt = s["k_pages"].dtype
    s["k_pages"][0][page, :, place % ps] = _rotate(s["k_new"], cos, sin, case).to(dt)
    s["v_pages"][0][page, :, place % ps] = s["v_new"]
    return {"q": _rotate(s["q"], cos, sin, case).to(dt), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, ps, P = case["hq"], case["hkv"], case["d"], case["page"], case["prefix"]
    seqs, width = s["table"].shape
    b, i = _rows(s)
    cu, lens = s["cu"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    dev = s["q"].device

    def rows_of(pages, table):  # the tokens of each sequence in order, [sequences, kv heads, tokens, head dim]
        return pages[0][table.long().clamp(min=0)].transpose(1, 2).flatten(2, 3).float()

    place = torch.arange(width * ps, device=dev)
    held = place < lens[:, None]
    keys, values = rows_of(s["k_pages"], s["table"]), rows_of(s["v_pages"], s["table"])
    values = values.masked_fill(~held[:, None, :, None], 0.0)
    # queries [sequences, kv heads, queries of the group, head dim], each sequence's padded to the longest
    most = s["max_new"]
    step = torch.arange(most, device=dev)
    q = s["q"][(cu[:-1, None] + step).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(seqs, most, hkv, hq // hkv, d).transpose(1, 2).flatten(2, 3)
    scores = q @ keys.transpose(2, 3)
    key_at = P + place
    if P:
        pk, pv = rows_of(s["k_pages"], s["prefix_pages"][None])[:, :, :P], rows_of(s["v_pages"], s["prefix_pages"][None])[:, :, :P]
        scores = torch.cat([q @ pk.transpose(2, 3), scores], -1)
        key_at = torch.arange(P + width * ps, device=dev)
        held = torch.cat([held.new_ones(seqs, P), held], 1)
    at = (P + lens - n)[:, None] + step  # [sequences, queries]
    sees = held[:, None] & (key_at <= at[..., None])
    if case["window"]:
        sees &= (key_at > at[..., None] - case["window"]) | (key_at < case["sinks"])
    sees = sees.repeat_interleave(hq // hkv, 1)[:, None]
    scores = scores.mul_(1.0 / math.sqrt(d)).masked_fill_(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    weight = p.sum(-1, keepdim=True)
    out = p[..., P:] @ values
    if P:
        out += p[..., :P] @ pv
    out = out / weight.masked_fill(weight == 0, 1.0)
    out = out.view(seqs, hkv, most, hq // hkv, d).transpose(1, 2).reshape(seqs, most, hq, d)
    return out[b, i].to(s["q"].dtype)


# -------------------------------------------------------- the framework's calls
def _own(s):
    case = s["case"]
    if "cache" not in s:
        from quantized_decode_attention_head_b200 import PagedKVCache

        s["cache"] = PagedKVCache(s["k_pages"], s["v_pages"], case["hq"])
        s["workspace"] = s["cache"].make_workspace(case["seqs"], s["q"].shape[0])
    cache = s["cache"]
    cu = None if case["new"] == 1 else s["cu"]
    if case["kind"] == "append":
        q = cache.rq_paged_append(0, s["k_new"], s["v_new"], s["table"], s["kv_lens"], cu_new=cu, q=s["q"],
                                  cos_sin=s["cos_sin"], positions=s.get("positions"),
                                  sections=_sections(case) if case["axes"] > 1 else None,
                                  interleaved=case["interleaved"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if case["kind"] == "attend":
        return cache.rq_paged_attention(0, s["q"], s["table"], s["kv_lens"], cu_new=cu, max_new=s["max_new"],
                                        window=case["window"], n_sink=case["sinks"], workspace=s["workspace"])
    return cache.rq_paged_shared_attention(0, s["q"], s["prefix_pages"], case["prefix"], s["table"], s["kv_lens"],
                                           cu_new=cu, max_new=s["max_new"], window=case["window"],
                                           n_sink=case["sinks"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    if state["case"]["kind"] == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ------------------------------------------------------------ what a pass needs
def _visible(case, kv, n):
    """(keys that any of a sequence's n queries sees, sum over the queries of the keys that each sees), prefix left out and of the prefix."""
    P, w, sinks = case["prefix"], case["window"], case["sinks"]
    pairs_own = pairs_pre = 0
    for i in range(n):
        at = P + kv - n + i
        lo = max(0, at + 1 - w) if w else 0
        first = min(sinks, lo)
        pre = min(P, first) + max(0, P - max(lo, 0)) if lo < P else min(P, first)
        pairs_pre += pre
        pairs_own += max(0, at + 1) - lo + first - pre if at >= 0 else 0
    lo = max(0, P + kv - n + 1 - w) if w else 0
    first = min(sinks, lo)
    keys = P + kv - lo + first
    pre = min(P, first) + max(0, P - lo)
    return keys - pre, pairs_own, pre, pairs_pre


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = _lengths(case)
    total = sum(n for _, n in lens)
    if case["kind"] == "append":
        # q and k read and written, v read and written, the angles of each token's position
        return {"bytes": total * ((2 * hq + 4 * hkv) * d * 2 + case["rot"] * 4 + 4 * (case["axes"] if case["axes"] > 1 else 0)),
                "flops": total * (hq + hkv) * case["rot"] * 3}
    rows = [_visible(case, kv, n) for kv, n in lens]
    keys = sum(r[0] for r in rows) + max(r[2] for r in rows)  # a shared key is read once
    pairs = sum(r[1] + r[3] for r in rows)
    return {"bytes": keys * hkv * d * 2 * 2 + total * hq * d * 2 * 2, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    lens = _lengths(case)
    w = work(case)
    if w["flops"] > 6e11 or w["bytes"] > 4e9:
        return None
    s = prepare(case, seed)
    ps, d, P = case["page"], case["d"], case["prefix"]
    start = 0
    f64 = torch.float64
    if case["kind"] == "append":
        half = case["rot"] // 2
        pages_k, pages_v = s["k_pages"].to(f64), s["v_pages"].to(f64)
        turn = torch.complex(s["cos_sin"][:, :half].to(f64), s["cos_sin"][:, half:].to(f64))
        pair = torch.arange(half, device="cuda")
        first = 2 * pair if case["interleaved"] else pair
        second = first + 1 if case["interleaved"] else first + half
        out_q = s["q"].to(f64)
        for b, (kv, n) in enumerate(lens):
            at = torch.arange(kv - n, kv, device="cuda")
            where = at[:, None].expand(n, half)
            if case["axes"] > 1:
                parts, lo = [], 0
                for a, size in enumerate(_sections(case)):
                    parts.append(s["positions"][a, start : start + n].long()[:, None].expand(n, size))
                    lo += size
                where = torch.cat(parts, 1)
            by = turn[where, pair][:, None]
            page = s["table"][b].long()[at // ps]
            for x, heads in ((out_q, case["hq"]), (s["k_new"].to(f64), case["hkv"])):
                y = x[start : start + n].clone()
                z = torch.complex(y[..., first], y[..., second]) * by
                y[..., first], y[..., second] = z.real, z.imag
                if heads == case["hq"] and x is out_q:
                    out_q[start : start + n] = y
                else:
                    pages_k[0, page, :, at % ps] = y
            pages_v[0, page, :, at % ps] = s["v_new"][start : start + n].to(f64)
            start += n
        return {"q": out_q, "k_pages": pages_k, "v_pages": pages_v}
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    group = case["hq"] // case["hkv"]
    pre = s["prefix_pages"].long()
    for b, (kv, n) in enumerate(lens):
        pages = s["table"][b, : -(-kv // ps)].long()
        at = P + kv - n + torch.arange(n, device="cuda")
        key = torch.arange(P + kv, device="cuda")
        back = at[:, None] - key
        hidden = back < 0
        if case["window"]:
            hidden = hidden | ((back >= case["window"]) & (key >= case["sinks"]))
        for h in range(case["hkv"] if kv else 0):
            ks, vs = (torch.cat([x[0, pre, h].reshape(-1, d)[:P], x[0, pages, h].reshape(-1, d)[:kv]]).to(f64)
                      for x in (s["k_pages"], s["v_pages"]))
            for j in range(h * group, h * group + group):
                e = (s["q"][start : start + n, j].to(f64) @ ks.T) / d ** 0.5
                e = torch.softmax(e.masked_fill(hidden, -math.inf), 1)
                out[start : start + n, j] = e @ vs
        start += n
    return out
