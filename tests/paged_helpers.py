"""Plain 64-bit forms of the paged cache's operators, and batches for them."""

from __future__ import annotations

import math

import torch

F64 = torch.float64


class Batch:
    """Sequences of (tokens held, new tokens) over pages in a scattered order;
    table entries past a sequence's last page are -1."""

    def __init__(self, lens, hq, hkv, d, page, dtype, seed=0, prefix=0, layers=1, layer=0, extra_rows=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.d, self.page, self.dtype = lens, hq, hkv, d, page, dtype
        self.prefix, self.layer, self.device = prefix, layer, device
        self.total = sum(n for _, n in lens)
        self.rows = self.total + extra_rows
        n_prefix = -(-prefix // page)
        used = sum(-(-kv // page) for kv, _ in lens) + n_prefix
        n_pages = used + 3
        order = torch.randperm(n_pages, generator=g)
        width = max([1] + [-(-kv // page) for kv, _ in lens])
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = n_prefix
        for b, (kv, _) in enumerate(lens):
            k = -(-kv // page)
            self.table[b, :k] = order[at : at + k].int()
            at += k
        self.prefix_pages = order[:n_prefix].int().to(device)
        self.table = self.table.to(device)
        self.kv_lens = torch.tensor([kv for kv, _ in lens], dtype=torch.int32, device=device)
        cu = [0]
        for _, n in lens:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.max_new = max([1] + [n for _, n in lens])
        shape = (layers, n_pages, hkv, page, d)
        self.k_pages = torch.randn(shape, generator=g).to(dtype).to(device)
        self.v_pages = torch.randn(shape, generator=g).to(dtype).to(device)
        self.q = torch.randn((self.rows, hq, d), generator=g).to(dtype).to(device)

    def held(self, pages, b):
        """The tokens of sequence b (prefix first) in order, [kv heads, tokens, head dim], 64 bits."""
        kv = self.lens[b][0]
        own = pages[self.layer][self.table[b, : -(-kv // self.page)].long()]
        own = own.transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :kv]
        pre = pages[self.layer][self.prefix_pages.long()].transpose(0, 1).reshape(self.hkv, -1, self.d)[:, : self.prefix]
        return torch.cat([pre, own], 1).to(F64)

    def seen(self, b, window, n_sink):
        """[new tokens, keys] of sequence b: which keys each query sees."""
        kv, n = self.lens[b]
        p = torch.arange(self.prefix + kv - n, self.prefix + kv, device=self.device)[:, None]
        j = torch.arange(self.prefix + kv, device=self.device)
        see = j <= p
        if window:
            see &= (p - j < window) | (j < n_sink)
        return see

    def poison(self, window, n_sink):
        """NaN in every place of the pages that no query sees (the layer's and other layers')."""
        nan = float("nan")
        for pages in (self.k_pages, self.v_pages):
            keep = torch.zeros(pages.shape[:2] + pages.shape[3:4], dtype=torch.bool, device=self.device)
            for b, (kv, n) in enumerate(self.lens):
                any_sees = self.seen(b, window, n_sink).any(0) if n else None
                if any_sees is None:
                    continue
                for j in torch.nonzero(any_sees).flatten().tolist():
                    if j < self.prefix:
                        keep[self.layer, int(self.prefix_pages[j // self.page]), j % self.page] = True
                    else:
                        t = j - self.prefix
                        keep[self.layer, int(self.table[b, t // self.page]), t % self.page] = True
            pages.masked_fill_(~keep[:, :, None, :, None], nan)


def reference(bt: Batch, window=0, n_sink=0, scale=None):
    """(out, lse, tolerance of out, of lse) in 64 bits for the packed rows [0, total).

    Tolerance, with u = half a step of the type (relative): the result is
    rounded once (u |out|) and each weight at most once to the type (u A, A =
    sum p |v| / sum p); fp32 products and sums of a score are off by at most
    delta = (d + 4) 2^-23 scale sum |q k|, which moves a weight, and their sum,
    by that factor each (2 delta A), the exponential by 2^-21 (both); weights
    below the smallest normal fp16 number keep an absolute error of 2^-25.
    The logarithm of the sum: delta, the exponential's 2^-21, and its own
    roundings, 2^-22 of the value."""
    scale = 1.0 / math.sqrt(bt.d) if scale is None else scale
    g = bt.hq // bt.hkv
    out = torch.zeros((bt.total, bt.hq, bt.d), dtype=F64, device=bt.device)
    tol = torch.zeros_like(out)
    lse = torch.full((bt.total, bt.hq), -math.inf, dtype=F64, device=bt.device)
    lse_tol = torch.zeros_like(lse)
    u = torch.finfo(bt.dtype).eps / 2
    t = 0
    for b, (kv, n) in enumerate(bt.lens):
        if n and kv + bt.prefix:
            see = bt.seen(b, window, n_sink)
            any_sees = see.any(0)
            k, v = bt.held(bt.k_pages, b), bt.held(bt.v_pages, b)
            k = torch.where(any_sees[None, :, None], k, torch.zeros_like(k))
            v = torch.where(any_sees[None, :, None], v, torch.zeros_like(v))
            q = bt.q[t : t + n].to(F64).view(n, bt.hkv, g, bt.d).permute(1, 2, 0, 3)
            x = scale * torch.einsum("hgnd,hkd->hgnk", q, k)
            ax = scale * torch.einsum("hgnd,hkd->hgnk", q.abs(), k.abs()).masked_fill(~see, 0.0)
            x = x.masked_fill(~see, -math.inf)
            some = see.any(1)
            w = torch.softmax(x[:, :, some], -1)
            o = torch.einsum("hgnk,hkd->hgnd", w, v)
            a = torch.einsum("hgnk,hkd->hgnd", w, v.abs())
            delta = ((bt.d + 4) * 2.0**-23 * ax[:, :, some]).amax(-1, keepdim=True)
            e = u * o.abs() + a * (u + 2 * delta + 2.0**-20) + 1e-30
            if bt.dtype is torch.float16:
                e = e + (see[some].sum(1) * 2.0**-25)[None, None, :, None] * v.abs().amax(1)[:, None, None, :] + 2.0**-25
            rows = t + torch.nonzero(some).flatten()
            out[rows] = o.permute(2, 0, 1, 3).reshape(-1, bt.hq, bt.d)
            tol[rows] = e.permute(2, 0, 1, 3).reshape(-1, bt.hq, bt.d)
            lse_tol[rows] = delta[..., 0].permute(2, 0, 1).reshape(-1, bt.hq) + 2.0**-20
            lse[rows] = torch.logsumexp(x[:, :, some], -1).permute(2, 0, 1).reshape(-1, bt.hq)
        t += n
    return out, lse, tol, lse_tol + 2.0**-22 * lse.abs().nan_to_num(posinf=0.0)


def check(bt: Batch, got, ref, what=""):
    out, _, tol, _ = ref
    err = (got[: bt.total].to(F64) - out).abs()
    assert torch.isfinite(got[: bt.total].float()).all(), what
    over = err - tol
    assert (over <= 0).all(), f"{what}: off by {float(err.max()):.3e}, {float((err / (tol + 1e-300)).max()):.2f} times the tolerance"


def check_lse(bt: Batch, got, ref, what=""):
    _, lse, _, tol = ref
    got = got[: bt.total].to(F64)
    assert torch.equal(torch.isinf(got), torch.isinf(lse)), what
    fin = torch.isfinite(lse)
    assert ((got - lse)[fin].abs() <= tol[fin]).all(), what


def rotate(x, cos, sin, interleaved, rot, f=torch.float32):
    """x [tokens, heads, d] turned pairwise, cos and sin [tokens, rot/2], every operation rounded to f."""
    x = x.to(f)
    c, s = cos[:, None].to(f), sin[:, None].to(f)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * c - b * s, b * c + a * s
    return y


def angles(n, rot, device="cuda"):
    half = rot // 2
    f = 10000.0 ** (-torch.arange(half, dtype=F64) / half)
    a = torch.arange(n, dtype=F64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().to(device)
