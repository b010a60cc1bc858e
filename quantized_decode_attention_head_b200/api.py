"""Python binding with the C ABI's names (include/rq.h).

PyTorch supplies device memory and streams; every computation happens in
librq.so.  Functions take torch tensors and pass their data pointers.
"""

from __future__ import annotations

import contextlib
import ctypes

import numpy as np

from ._lib import CacheConfig, PagedBatch, PagedConfig, Rotation, check, lib


def _stream_ptr(stream=None, device=None):
    """The raw cudaStream_t of `stream`, or of the current stream of `device`
    (default: the current device)."""
    import torch

    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    idx = torch.cuda.current_device() if device is None else device
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(idx))


def _allocates_on(stream):
    """Context for what a call allocates (and reads back) itself.  Memory
    belongs to the stream that is current when torch allocates it, and is
    handed out again in that stream's order: so with `stream` given it has to
    be allocated with that stream current, or other work may get a temporary
    while the call's kernels still use it."""
    import torch

    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _dptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _check_tensor(name, t, dtype, shape=None, device_type="cuda", align=16):
    import torch

    # one cheap test on the common path; the detailed message only on failure
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda == (device_type == "cuda")
            and t.is_contiguous() and (shape is None or t.shape == tuple(shape)) and t.data_ptr() % align == 0):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != device_type:
        raise ValueError(f"{name} must be on {device_type}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must start on a {align}-byte boundary (a view at an offset into a larger tensor?)")


def _same_device(name, t, device):
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the device of the pages")


def _int32(**values):
    """ctypes cuts what does not fit; called where a shift shows bits past it (or a sign)."""
    for name, v in values.items():
        if not -(2**31) <= v < 2**31:
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def rq_allocate_bits(w, alpha, beta, avg_bits, allowed):
    """RateQuant allocation (host).  Returns dict(b_cont, b_int, log_lambda)."""
    w = np.ascontiguousarray(w, dtype=np.float64)
    n = w.size
    alpha = np.ascontiguousarray(np.broadcast_to(np.asarray(alpha, dtype=np.float64), (n,)))
    beta = np.ascontiguousarray(np.broadcast_to(np.asarray(beta, dtype=np.float64), (n,)))
    allowed = np.ascontiguousarray(allowed, dtype=np.int32)
    b_cont = np.zeros(n, dtype=np.float64)
    b_int = np.zeros(n, dtype=np.int32)
    nu = ctypes.c_double(0.0)
    dp = ctypes.POINTER(ctypes.c_double)
    ip = ctypes.POINTER(ctypes.c_int)
    code = lib().rq_allocate_bits(
        n,
        w.ctypes.data_as(dp),
        alpha.ctypes.data_as(dp),
        beta.ctypes.data_as(dp),
        float(avg_bits),
        allowed.ctypes.data_as(ip),
        allowed.size,
        b_cont.ctypes.data_as(dp),
        b_int.ctypes.data_as(ip),
        ctypes.byref(nu),
    )
    check("rq_allocate_bits", code)
    return {"b_cont": b_cont, "b_int": b_int.astype(np.int64), "log_lambda": nu.value}


def rq_measure_distortion(x, role, bits, stream=None):
    """Mean squared error of this library's quantizer per (head, bit width).
    x: bf16 CUDA tensor [n_heads, n_tokens, head_dim]; role "K" or "V".
    Returns a float64 numpy array [n_heads, len(bits)]."""
    import torch

    if x.dim() != 3:
        raise ValueError("x must be [n_heads, n_tokens, head_dim]")
    _check_tensor("x", x, torch.bfloat16, align=2)
    h, t, d = x.shape
    bits = np.ascontiguousarray(bits, dtype=np.int32)
    with _allocates_on(stream):
        mse = torch.empty((h, bits.size), dtype=torch.float64, device=x.device)
        check("rq_measure_distortion", lib().rq_measure_distortion(
            _dptr(x), h, t, d, 0 if role == "K" else 1, bits.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), bits.size,
            _dptr(mse), _stream_ptr(stream)))
        return mse.cpu().numpy()


def rq_fit_distortion(bits, mse, r2_min=0.96):
    """Per-head (alpha, beta, r2) of D(b) = alpha * beta^-b from an
    [n_heads, n_bits] table, with the poor-fit fallback (host)."""
    bits = np.ascontiguousarray(bits, dtype=np.int32)
    mse = np.ascontiguousarray(mse, dtype=np.float64)
    n = mse.shape[0]
    alpha, beta, r2 = np.zeros(n), np.zeros(n), np.zeros(n)
    dp = ctypes.POINTER(ctypes.c_double)
    check("rq_fit_distortion", lib().rq_fit_distortion(
        n, bits.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), bits.size, mse.ctypes.data_as(dp), float(r2_min),
        alpha.ctypes.data_as(dp), beta.ctypes.data_as(dp), r2.ctypes.data_as(dp)))
    return alpha, beta, r2


def rq_cap_weights(w, factor=5.0):
    """w_i <- min(w_i, factor * mean(w)) (host)."""
    w = np.ascontiguousarray(w, dtype=np.float64)
    out = np.zeros_like(w)
    dp = ctypes.POINTER(ctypes.c_double)
    check("rq_cap_weights", lib().rq_cap_weights(w.size, w.ctypes.data_as(dp), float(factor), out.ctypes.data_as(dp)))
    return out


def _config(n_layers, batch, n_q_heads, n_kv_heads, head_dim, n_sink, n_recent, max_tokens, k_bits, v_bits, group=32,
            k_norm=False, hybrid=False):
    kb = np.ascontiguousarray(np.asarray(k_bits, dtype=np.int32).reshape(-1))
    vb = np.ascontiguousarray(np.asarray(v_bits, dtype=np.int32).reshape(-1))
    ip = ctypes.POINTER(ctypes.c_int)
    cfg = CacheConfig(
        n_layers, batch, n_q_heads, n_kv_heads, head_dim, group, n_sink, n_recent, max_tokens,
        kb.ctypes.data_as(ip), vb.ctypes.data_as(ip), int(bool(k_norm)), int(bool(hybrid)),
    )
    return cfg, (kb, vb)


def rq_cache_bytes(**cfg_kwargs) -> int:
    cfg, _keep = _config(**cfg_kwargs)
    out = ctypes.c_size_t(0)
    check("rq_cache_bytes", lib().rq_cache_bytes(ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


class QuantizedKVCache:
    """Owns a device buffer (torch uint8 tensor) and the library's host handle."""

    def __init__(self, n_layers, batch, n_q_heads, n_kv_heads, head_dim, n_sink, n_recent, max_tokens,
                 k_bits, v_bits, device="cuda", group=32, k_norm=False, hybrid=False):
        import torch

        self.n_layers, self.batch = n_layers, batch
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.n_sink, self.n_recent, self.max_tokens = n_sink, n_recent, max_tokens
        self.k_bits = np.asarray(k_bits, dtype=np.int32).reshape(n_layers, n_kv_heads)
        self.v_bits = np.asarray(v_bits, dtype=np.int32).reshape(n_layers, n_kv_heads)
        cfg, keep = _config(n_layers, batch, n_q_heads, n_kv_heads, head_dim, n_sink, n_recent, max_tokens,
                            self.k_bits, self.v_bits, group, k_norm, hybrid)
        self.k_norm = bool(k_norm)
        self.hybrid = bool(hybrid)
        nbytes = ctypes.c_size_t(0)
        check("rq_cache_bytes", lib().rq_cache_bytes(ctypes.byref(cfg), ctypes.byref(nbytes)))
        self.nbytes = nbytes.value
        self.buffer = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.buffer.data_ptr()) % 256
        self.buffer = self.buffer[off : off + self.nbytes]
        handle = ctypes.c_void_p(0)
        check("rq_cache_init", lib().rq_cache_init(ctypes.byref(cfg), _dptr(self.buffer), self.nbytes,
                                                   ctypes.byref(handle), _stream_ptr(None, self.buffer.get_device())))
        self.handle = handle
        # kept for the destructor, which may run while the interpreter is
        # tearing module globals down
        self._destroy = lib().rq_cache_destroy
        del keep

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h is not None and h.value and destroy is not None:
            destroy(h)
            self.handle = None

    # -- queries -----------------------------------------------------------
    def length(self, layer=0) -> int:
        t = ctypes.c_int(0)
        check("rq_cache_length", lib().rq_cache_length(self.handle, layer, ctypes.byref(t)))
        return t.value

    def k_norm_factors(self, layer, b, kv_head):
        """The stream's per-channel K normalization factors n[D] (a device view)."""
        import torch

        lay = self.stream_layout(layer, b, kv_head)
        d = self.head_dim
        rows = (2 * self.n_sink + 2 * (self.n_recent + 32)) * d * 2
        off = lay["window_offset"] + rows
        return self.buffer[off : off + 4 * d].view(torch.float32)

    def stream_layout(self, layer, b, kv_head):
        to, wo = ctypes.c_size_t(0), ctypes.c_size_t(0)
        rb, nt = ctypes.c_int(0), ctypes.c_int(0)
        check("rq_cache_stream_layout", lib().rq_cache_stream_layout(
            self.handle, layer, b, kv_head, ctypes.byref(to), ctypes.byref(rb), ctypes.byref(nt), ctypes.byref(wo)))
        return {"tile_offset": to.value, "record_bytes": rb.value, "n_tiles": nt.value, "window_offset": wo.value}

    # -- path ----------------------------------------------------------------
    def rq_quantize_kv(self, k, v, stream=None):
        import torch

        L, B, H, D = self.n_layers, self.batch, self.n_kv_heads, self.head_dim
        T = k.shape[3] if k.dim() == 5 else -1
        _check_tensor("k", k, torch.bfloat16, (L, B, H, T, D))
        _check_tensor("v", v, torch.bfloat16, (L, B, H, T, D))
        check("rq_quantize_kv", lib().rq_quantize_kv(self.handle, _dptr(k), _dptr(v), T, _stream_ptr(stream)))

    def rq_append_token(self, layer, k_new, v_new, stream=None):
        import torch

        nl = self.n_layers if layer == -1 else 1
        shape = (nl, self.batch, self.n_kv_heads, self.head_dim) if layer == -1 else (
            self.batch, self.n_kv_heads, self.head_dim)
        _check_tensor("k_new", k_new, torch.bfloat16, shape)
        _check_tensor("v_new", v_new, torch.bfloat16, shape)
        check("rq_append_token", lib().rq_append_token(self.handle, layer, _dptr(k_new), _dptr(v_new),
                                                       _stream_ptr(stream)))

    def rq_decode_workspace_bytes(self, n_splits=0) -> int:
        out = ctypes.c_size_t(0)
        check("rq_decode_workspace_bytes", lib().rq_decode_workspace_bytes(self.handle, n_splits, ctypes.byref(out)))
        return out.value

    def make_workspace(self, n_splits=0, stream=None):
        import torch

        nb = self.rq_decode_workspace_bytes(n_splits)
        with _allocates_on(stream):
            ws = torch.empty(nb, dtype=torch.uint8, device=self.buffer.device)
        check("rq_decode_workspace_init", lib().rq_decode_workspace_init(_dptr(ws), nb, _stream_ptr(stream)))
        return ws

    def rq_decode_attention(self, layer, q, out=None, softmax_scale=0.0, n_splits=0, workspace=None, stream=None):
        import torch

        nl = self.n_layers if layer == -1 else 1
        shape = (nl, self.batch, self.n_q_heads, self.head_dim) if layer == -1 else (
            self.batch, self.n_q_heads, self.head_dim)
        _check_tensor("q", q, torch.bfloat16, shape)
        if out is None:
            with _allocates_on(stream):
                out = torch.empty(shape, dtype=torch.float32, device=q.device)
        _check_tensor("out", out, torch.float32, shape)
        if workspace is None:
            workspace = self.make_workspace(n_splits, stream)
        check("rq_decode_attention", lib().rq_decode_attention(
            self.handle, layer, _dptr(q), _dptr(out), float(softmax_scale), int(n_splits), _dptr(workspace),
            workspace.numel(), _stream_ptr(stream, q.get_device())))
        return out

    def rq_decode_step(self, layer, q, k_new, v_new, out=None, softmax_scale=0.0, n_splits=0, workspace=None,
                       stream=None):
        """rq_append_token(layer, k_new, v_new) then rq_decode_attention(layer, q),
        in one launch (the step before a tile flush also packs that tile
        ahead); two launches only when the completed tile was not packed
        ahead by the previous step."""
        import torch

        nl = self.n_layers if layer == -1 else 1
        qshape = (nl, self.batch, self.n_q_heads, self.head_dim) if layer == -1 else (
            self.batch, self.n_q_heads, self.head_dim)
        kshape = (nl, self.batch, self.n_kv_heads, self.head_dim) if layer == -1 else (
            self.batch, self.n_kv_heads, self.head_dim)
        _check_tensor("q", q, torch.bfloat16, qshape)
        _check_tensor("k_new", k_new, torch.bfloat16, kshape)
        _check_tensor("v_new", v_new, torch.bfloat16, kshape)
        if out is None:
            with _allocates_on(stream):
                out = torch.empty(qshape, dtype=torch.float32, device=q.device)
        _check_tensor("out", out, torch.float32, qshape)
        if workspace is None:
            workspace = self.make_workspace(n_splits, stream)
        check("rq_decode_step", lib().rq_decode_step(
            self.handle, layer, _dptr(q), _dptr(k_new), _dptr(v_new), _dptr(out), float(softmax_scale),
            int(n_splits), _dptr(workspace), workspace.numel(), _stream_ptr(stream, q.get_device())))
        return out

    @staticmethod
    def rq_decode_read_status(workspace) -> int:
        st = ctypes.c_int(0)
        check("rq_decode_read_status", lib().rq_decode_read_status(_dptr(workspace), ctypes.byref(st)))
        return st.value


class PagedKVCache:
    """A cache of 16-bit keys and values in pages, bound to the caller's page
    tensors (kept alive by this object): k_pages, v_pages, contiguous bf16 or
    fp16 CUDA tensors [n_layers, n_pages, n_kv_heads, page_size, head_dim].

    A batch is described with every call.  page_table: int32 [n_seqs, width],
    token t of a sequence lies in row t % page_size of page
    page_table[sequence, t // page_size].  kv_lens: int32 [n_seqs], tokens of
    each sequence, new ones included.  cu_new: int32 [n_seqs + 1], where each
    sequence's new tokens begin among the packed ones; None: one new token
    each.  All three are CUDA tensors, read when the kernel runs.

    Calls run on `stream`, or on the current stream of the pages' device; what
    they allocate (results, a workspace that is not given) is memory of that
    stream, as if it were the current one.  As the C handle, an object is for
    one thread of control.
    """

    def __init__(self, k_pages, v_pages, n_q_heads):
        import torch

        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 5:
            raise ValueError("k_pages must be a tensor [n_layers, n_pages, n_kv_heads, page_size, head_dim]")
        if k_pages.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"k_pages must be torch.bfloat16 or torch.float16, got {k_pages.dtype}")
        _check_tensor("k_pages", k_pages, k_pages.dtype)
        _check_tensor("v_pages", v_pages, k_pages.dtype, k_pages.shape)
        _same_device("v_pages", v_pages, k_pages.get_device())
        self.k_pages, self.v_pages = k_pages, v_pages
        self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k_pages.shape
        self.n_q_heads = int(n_q_heads)
        _int32(n_q_heads=self.n_q_heads)
        self.dtype = k_pages.dtype
        self.device = k_pages.get_device()
        cfg = PagedConfig(self.n_layers, self.n_pages, self.page_size, self.n_q_heads, self.n_kv_heads,
                          self.head_dim, 0 if self.dtype is torch.bfloat16 else 1)
        handle = ctypes.c_void_p(0)
        with torch.cuda.device(self.device):
            check("rq_paged_cache_init", lib().rq_paged_cache_init(
                ctypes.byref(cfg), _dptr(k_pages), _dptr(v_pages), ctypes.byref(handle)))
            # RQ_ERR_DEVICE_INDEX of the appends (attention calls report in their workspace)
            self.append_status = torch.zeros(1, dtype=torch.int32, device=k_pages.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()  # appends may run on other streams
        self.handle = handle
        self._destroy = lib().rq_paged_cache_destroy
        # the structures that calls fill in, and what a call needs of torch
        self._b, self._r = PagedBatch(), Rotation()
        self._b_ref, self._r_ref = ctypes.byref(self._b), ctypes.byref(self._r)
        self._status_ptr = self.append_status.data_ptr()
        self._i32, self._f32, self._empty_like = torch.int32, torch.float32, torch.empty_like
        self._contiguous = torch.contiguous_format
        self._device_guard = torch.cuda.device
        self._append_fn = lib().rq_paged_append
        self._attention_fns = lib().rq_paged_attention, lib().rq_paged_shared_attention
        self._raw_stream, self._current = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h is not None and h.value and destroy is not None:
            destroy(h)
            self.handle = None

    # -- arguments -----------------------------------------------------------
    def _ints(self, name, t, shape):
        """Address of an int32 tensor of the pages' device."""
        # one cheap test on the common path; the detailed message only on failure
        if t.dtype is self._i32 and t.get_device() == self.device and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
        _check_tensor(name, t, self._i32, shape, align=4)
        _same_device(name, t, self.device)
        return t.data_ptr()

    def _batch(self, n_tokens, page_table, kv_lens, cu_new, max_new):
        """Fills the batch structure in; returns the number of sequences."""
        if page_table.dim() != 2 or page_table.shape[1] < 1:
            raise ValueError("page_table must be a tensor [n_seqs, width], width >= 1")
        shape = page_table.shape
        n_seqs, b = shape[0], self._b
        b.n_seqs, b.table_width = shape
        b.n_tokens = n_tokens
        b.page_table = self._ints("page_table", page_table, shape)
        b.kv_lens = self._ints("kv_lens", kv_lens, (n_seqs,))
        if cu_new is None:
            if n_tokens < n_seqs:
                raise ValueError(f"{n_tokens} packed tokens for {n_seqs} sequences of one new token each")
            b.cu_new, b.max_new = None, 1
        else:
            b.cu_new = self._ints("cu_new", cu_new, (n_seqs + 1,))
            if max_new is not None and max_new >> 31:
                _int32(max_new=max_new)
            b.max_new = n_tokens if max_new is None else max_new
        return n_seqs

    def _packed(self, name, t, heads):
        """Tokens of `heads` contiguous heads each; the tokens may lie apart
        (a part of a wider tensor).  Returns the elements between tokens."""
        d = self.head_dim
        if t.dtype is not self.dtype:
            raise TypeError(f"{name} must be {self.dtype}, got {t.dtype}")
        if t.get_device() != self.device:
            raise ValueError(f"{name} must be on the device of the pages")
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected (tokens, {heads}, {d})")
        s0, s1, s2 = t.stride()
        if shape[0] <= 1:
            s0 = heads * d
        if s2 != 1 or (s1 != d and heads > 1) or s0 < heads * d or s0 % 8:
            raise ValueError(f"{name}: a token's heads must be contiguous and tokens lie a multiple of 8 elements apart")
        if t.data_ptr() % 16:
            raise ValueError(f"{name} must start on a 16-byte boundary (a view at an offset into a larger tensor?)")
        return s0

    def _new_like(self, q, stream):
        """A contiguous tensor of q's type and shape, memory of `stream`."""
        if stream is None:
            return self._empty_like(q, memory_format=self._contiguous)
        with _allocates_on(stream):
            return self._empty_like(q, memory_format=self._contiguous)

    def _launch(self, func, fn, stream, *args):
        """Calls fn on `stream` (default: the current stream of the pages'
        device), with that device current."""
        if self._current() == self.device:
            code = fn(*args, self._raw_stream(self.device) if stream is None else stream.cuda_stream)
        else:
            with self._device_guard(self.device):
                code = fn(*args, self._raw_stream(self.device) if stream is None else stream.cuda_stream)
        if code:
            check(func, code)

    # -- calls ---------------------------------------------------------------
    def rq_paged_append(self, layer, k_new, v_new, page_table, kv_lens, cu_new=None, q=None, q_out=None, cos_sin=None,
                        positions=None, sections=None, interleaved=False, stream=None):
        """Write the batch's new keys and values [tokens, n_kv_heads, head_dim]
        into the layer's pages.  With cos_sin (fp32 [n_positions, rot_dim]:
        rot_dim/2 cosines, then as many sines, of each position) the keys are
        rotated on the way and q [tokens, n_q_heads, head_dim], if given, is
        rotated into q_out (default: a new tensor), which is returned.
        positions: int32 [tokens], or [axes, tokens] with `sections`, how many
        channel pairs turn by each axis; None: a token's place in its
        sequence.  interleaved: channels 2j, 2j + 1 are a pair (else j and
        j + rot_dim/2)."""
        ks = self._packed("k_new", k_new, self.n_kv_heads)
        vs = self._packed("v_new", v_new, self.n_kv_heads)
        n = k_new.shape[0]
        if v_new.shape[0] != n:
            raise ValueError(f"v_new has {v_new.shape[0]} tokens, k_new {n}")
        self._batch(n, page_table, kv_lens, cu_new, None)
        if layer >> 31:
            _int32(layer=layer)
        rot, qs, q_ptr, out_ptr = None, 0, None, None
        if cos_sin is None:
            if q is not None or positions is not None or sections is not None:
                raise ValueError("q, positions and sections go with cos_sin")
        else:
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin must be a tensor [n_positions, rot_dim]")
            _check_tensor("cos_sin", cos_sin, self._f32)
            _same_device("cos_sin", cos_sin, self.device)
            rot = self._r
            rot.cos_sin = cos_sin.data_ptr()
            rot.n_positions, rot.rot_dim = cos_sin.shape
            rot.interleaved = 1 if interleaved else 0
            axes, rot.positions = 1, None
            if positions is not None:
                axes = positions.shape[0] if positions.dim() == 2 else 1
                rot.positions = self._ints("positions", positions, (axes, n) if positions.dim() == 2 else (n,))
            if not 1 <= axes <= 4:
                raise ValueError(f"positions on {axes} axes: 1 to 4 are supported")
            if sections is None:
                if axes != 1:
                    raise ValueError("positions on several axes need sections")
                sections = (rot.rot_dim // 2,)
            if len(sections) != axes:
                raise ValueError(f"{len(sections)} sections for positions on {axes} axes")
            for pairs in sections:
                if pairs >> 31:
                    _int32(sections=pairs)
            rot.n_axes = axes
            rot.sections[:axes] = sections
            if q is not None:
                qs = self._packed("q", q, self.n_q_heads)
                if q.shape[0] != n:
                    raise ValueError(f"q has {q.shape[0]} tokens, k_new {n}")
                if q_out is None:
                    q_out = self._new_like(q, stream)
                else:
                    _check_tensor("q_out", q_out, self.dtype, q.shape)
                    _same_device("q_out", q_out, self.device)
                q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        self._launch("rq_paged_append", self._append_fn, stream, self.handle, layer, self._b_ref, None if rot is None else self._r_ref,
                     k_new.data_ptr(), ks, v_new.data_ptr(), vs, q_ptr, qs, out_ptr, self._status_ptr)
        return q_out

    def rq_paged_workspace_bytes(self, n_seqs, n_tokens) -> int:
        _int32(n_seqs=n_seqs, n_tokens=n_tokens)
        out = ctypes.c_size_t(0)
        check("rq_paged_workspace_bytes", lib().rq_paged_workspace_bytes(self.handle, n_seqs, n_tokens,
                                                                         ctypes.byref(out)))
        return out.value

    def make_workspace(self, n_seqs, n_tokens, stream=None):
        """Workspace for every attention call of at most n_seqs sequences and
        n_tokens packed tokens.  Calls that share one must not overlap."""
        import torch

        nb = self.rq_paged_workspace_bytes(n_seqs, n_tokens)
        with _allocates_on(stream):
            ws = torch.empty(nb, dtype=torch.uint8, device=self.k_pages.device)
        self._launch("rq_decode_workspace_init", lib().rq_decode_workspace_init, stream, _dptr(ws), nb)
        return ws

    def rq_paged_attention(self, layer, q, page_table, kv_lens, cu_new=None, max_new=None, window=0, n_sink=0,
                           softmax_scale=0.0, out=None, lse=None, workspace=None, stream=None):
        """Causal attention of the batch's new tokens q [tokens, n_q_heads,
        head_dim] over the pages of one layer, which hold their keys and values
        already.  max_new: the most new tokens any sequence has (default: all
        of q's; give it with cu_new where sequences have few new tokens each,
        or the call launches the kernels of prompts too).  window: a query sees the last `window` tokens up to itself
        and the sequence's first n_sink (0: all tokens).  Returns out, in q's
        type; rows behind the last sequence are left as they were.  lse: fp32
        [tokens, n_q_heads], filled with the natural logarithm of each
        softmax's denominator.  Without a workspace the call makes one, whose
        status word nobody can read."""
        return self._attention("rq_paged_attention", self._attention_fns[0], (), layer, q, page_table, kv_lens, cu_new, max_new, window,
                               n_sink, softmax_scale, out, lse, workspace, stream)

    def rq_paged_shared_attention(self, layer, q, prefix_pages, prefix_len, page_table, kv_lens, cu_new=None,
                                  max_new=None, window=0, n_sink=0, softmax_scale=0.0, out=None, lse=None,
                                  workspace=None, stream=None):
        """rq_paged_attention of sequences that all begin with the prefix_len
        tokens in prefix_pages (int32 [ceil(prefix_len / page_size)]), which
        are read once for the whole batch; page_table and kv_lens count what
        follows the prefix, window and n_sink count from its first token."""
        pages = self._ints("prefix_pages", prefix_pages, (prefix_pages.numel(),))
        prefix_len = int(prefix_len)
        if prefix_len < 0 or prefix_pages.numel() * self.page_size < prefix_len:
            raise ValueError(f"{prefix_pages.numel()} pages of {self.page_size} do not hold {prefix_len} tokens")
        return self._attention("rq_paged_shared_attention", self._attention_fns[1], (pages, prefix_len), layer, q,
                               page_table, kv_lens, cu_new, max_new, window, n_sink, softmax_scale, out, lse,
                               workspace, stream)

    def _attention(self, func, fn, prefix, layer, q, page_table, kv_lens, cu_new, max_new, window, n_sink,
                   softmax_scale, out, lse, workspace, stream):
        qs = self._packed("q", q, self.n_q_heads)
        n = q.shape[0]
        n_seqs = self._batch(n, page_table, kv_lens, cu_new, max_new)
        if (layer | window | n_sink) >> 31:
            _int32(layer=layer, window=window, n_sink=n_sink)
        if out is None:
            out = self._new_like(q, stream)
        else:
            _check_tensor("out", out, self.dtype, q.shape)
            _same_device("out", out, self.device)
        lse_ptr = None
        if lse is not None:
            _check_tensor("lse", lse, self._f32, (n, self.n_q_heads), align=4)
            _same_device("lse", lse, self.device)
            lse_ptr = lse.data_ptr()
        if workspace is None:
            workspace = self.make_workspace(n_seqs, n, stream)
        elif workspace.get_device() != self.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the pages")
        self._launch(func, fn, stream, self.handle, layer, self._b_ref, *prefix, q.data_ptr(), qs, out.data_ptr(), lse_ptr,
                     softmax_scale, window, n_sink, workspace.data_ptr(), workspace.nbytes)
        return out

    def read_status(self, workspace=None) -> int:
        """Blocking read of the status word of an attention workspace, or
        (None) of the appends, after the calls queued on any stream of the
        pages' device: 0, or RQ_ERR_DEVICE_INDEX / _TIMEOUT."""
        word = self.append_status if workspace is None else workspace
        with self._device_guard(self.device):
            return QuantizedKVCache.rq_decode_read_status(word)
