"""Attention over a paged 8-bit key/value cache: Python binding of the moe_kv_* and moe_paged_attention entry points.

Argument marshalling only, as in the rest of the package; ``include/moe.h`` states formats, limits and errors.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import moe_expert_layer_fwd_gb300 as _m

_byref = ctypes.byref


class _Bound:
    """torch's names and the library's functions, looked up once: a decode step makes these calls dozens of times, and
    the host has a few microseconds for each."""

    def __init__(self):
        torch, lib = _m._torch(), _m.lib()
        self.torch, self.bf16, self.i32, self.u8, self.f32 = torch, torch.bfloat16, torch.int32, torch.uint8, torch.float32
        self.append, self.gather, self.attention = lib.moe_kv_append, lib.moe_kv_gather, lib.moe_paged_attention
        self.workspace_size, self.status_bytes = lib.moe_paged_attention_workspace_size, lib.moe_status_bytes()
        self.raw_stream = torch._C._cuda_getCurrentRawStream


_bound = None


def _b() -> _Bound:
    global _bound
    if _bound is None:
        _bound = _Bound()
    return _bound


def _stream_of(stream, t):
    """The stream of the call: the given one, or torch's current one on the tensor's device."""
    return stream.cuda_stream if stream is not None else _b().raw_stream(t.get_device())


def _new(stream, like, shape, dtype=None):
    """A new tensor on the stream that the call runs on."""
    if stream is None:
        return _b().torch.empty(shape, dtype=dtype or like.dtype, device=like.device)
    with _b().torch.cuda.stream(stream):
        return _b().torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def _need(t, what: str, dtype, shape):
    """The address of a contiguous CUDA tensor of this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return _m._ptr(t)


def _rows(t, what: str, heads: int, D: int):
    """(pointer, token stride) of a [T, heads, D] bf16 tensor whose heads are dense."""
    if t.dtype is not _b().bf16 or t.dim() != 3 or t.shape[1:] != (heads, D):
        raise ValueError(f"{what}: expected a bfloat16 tensor [T, {heads}, {D}], got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    row, head, one = t.stride()
    if one != 1 or (head != D and heads > 1):
        raise ValueError(f"{what}: the heads of a token must be dense, got strides {t.stride()}")
    return t.data_ptr(), row if t.shape[0] > 1 else heads * D  # one token has no stride


class KVCache(NamedTuple):
    """The pool of one layer: E4M3 codes [n_pages, Hkv, page, D] and E8M0 scales [n_pages, Hkv], all uint8."""
    k_codes: object
    v_codes: object
    k_scale: object
    v_scale: object

    @staticmethod
    def empty(n_pages: int, Hkv: int, page: int = 64, D: int = 128, device="cuda") -> "KVCache":
        torch = _m._torch()
        return KVCache(*(torch.empty((n_pages, Hkv, page, D), dtype=torch.uint8, device=device) for _ in range(2)),
                       *(torch.zeros((n_pages, Hkv), dtype=torch.uint8, device=device) for _ in range(2)))

    def _struct(self) -> "_m.moe_kv_cache":
        k_codes, v_codes, k_scale, v_scale = self
        u8, shape = _m._torch().uint8 if _bound is None else _bound.u8, k_codes.shape
        if len(shape) != 4:
            raise ValueError(f"k_codes: expected [n_pages, Hkv, page, D], got {tuple(shape)}")
        return _m.moe_kv_cache(_need(k_codes, "k_codes", u8, shape), _need(v_codes, "v_codes", u8, shape),
                               _need(k_scale, "k_scale", u8, shape[:2]), _need(v_scale, "v_scale", u8, shape[:2]))


def _table(page_table):
    """(address, sequences, columns) of a page table."""
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected [B, max_pages], got {tuple(page_table.shape)}")
    shape = page_table.shape
    return _need(page_table, "page_table", _b().i32, shape), shape[0], shape[1]


def _status_ws(like, ws, stream=None):
    """The workspace given, or a new one with a clear status word, on the stream that the call runs on."""
    if ws is None:
        with _b().torch.cuda.stream(stream):
            return _b().torch.zeros(max(_b().status_bytes, 256), dtype=_b().u8, device=like.device)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous CUDA tensor")
    return ws


def moe_rope_table(max_pos: int, rot_dim: int = 128, base: float = 1e6, cos_sin=None, device="cuda", stream=None):
    """cos_sin [max_pos, rot_dim] fp32 of moe_kv_append: row p = cos(p f_i) | sin(p f_i), f_i = base^(-2i/rot_dim)."""
    torch = _m._torch()
    if cos_sin is None:
        with torch.cuda.stream(stream):
            cos_sin = torch.empty((max_pos, rot_dim), dtype=torch.float32, device=device)
    _m._check(_m.lib().moe_rope_table(max_pos, rot_dim, base, _need(cos_sin, "cos_sin", torch.float32,
                                                                  (max_pos, rot_dim)), _stream_of(stream, cos_sin)),
              "moe_rope_table")
    return cos_sin


def moe_kv_append(q, k, v, cache: KVCache, q_start, kv_len, page_table, cos_sin=None, rot_dim: Optional[int] = None,
                  interleaved: bool = False, q_norm_weight=None, k_norm_weight=None, eps: float = 1e-6, q_out=None,
                  ws=None, stream=None):
    """Normalises (when weights are given) and rotates the new queries and keys, stores the new keys and values in the
    cache; returns the queries [T, Hq, D] (None when q is None).  q, k, v may be views of one projection's rows."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    kp, ks = _rows(k, "k", Hkv, D)
    vp, vs = _rows(v, "v", Hkv, D)
    T = k.shape[0]
    Hq, qp, qs, op = Hkv, None, 0, None
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("q, k and v must have the same number of tokens")
    if q is not None:
        Hq = q.shape[1]
        qp, qs = _rows(q, "q", Hq, D)
        if q_out is not None:
            op = _need(q_out, "q_out", b.bf16, (T, Hq, D))
    max_pos, cs = 0, None
    if cos_sin is None:
        rot_dim = rot_dim or 0
    else:
        max_pos = cos_sin.shape[0]
        if rot_dim is None:
            rot_dim = cos_sin.shape[1]
        cs = _need(cos_sin, "cos_sin", b.f32, (max_pos, rot_dim))
    ws = _status_ws(k, ws, stream)
    starts, lens = _need(q_start, "q_start", b.i32, (B + 1,)), _need(kv_len, "kv_len", b.i32, (B,))
    qw = None if q_norm_weight is None else _need(q_norm_weight, "q_norm_weight", b.bf16, (D,))
    kw = None if k_norm_weight is None else _need(k_norm_weight, "k_norm_weight", b.bf16, (D,))
    d = _m.moe_kv_desc(B, T, Hq, Hkv, D, page, n_pages, max_pages)
    if q is not None and q_out is None:
        q_out = _new(stream, k, (T, Hq, D))
        op = q_out.data_ptr()
    status = b.append(_byref(d), qp, qs, kp, ks, vp, vs, starts, lens, table, cs, max_pos, rot_dim, interleaved, qw, kw, eps,
                      op, _byref(kv), ws.data_ptr(), ws.numel(), _stream_of(stream, k))
    if status:
        _m._check(status, "moe_kv_append")
    return q_out


def moe_kv_gather(cache: KVCache, start, out_start, page_table, n_rows: int, k=None, v=None, ws=None, stream=None):
    """Reads cached tokens back: returns (k, v) [n_rows, Hkv, D] bf16, where rows out_start[b] .. out_start[b+1] - 1
    are the tokens of sequence b from start[b] on."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    shape = (n_rows, Hkv, D)
    starts, out_starts = _need(start, "start", b.i32, (B,)), _need(out_start, "out_start", b.i32, (B + 1,))
    d = _m.moe_kv_desc(B, 0, Hkv, Hkv, D, page, n_pages, max_pages)
    ws = _status_ws(page_table, ws, stream)
    kp = None if k is None else _need(k, "k", b.bf16, shape)
    vp = None if v is None else _need(v, "v", b.bf16, shape)
    if k is None:
        k = _new(stream, page_table, shape, b.bf16)
        kp = k.data_ptr()
    if v is None:
        v = _new(stream, page_table, shape, b.bf16)
        vp = v.data_ptr()
    status = b.gather(_byref(d), starts, out_starts, table, _byref(kv), n_rows, kp, vp, ws.data_ptr(), ws.numel(),
                      _stream_of(stream, page_table))
    if status:
        _m._check(status, "moe_kv_gather")
    return k, v


def _workspace(desc, max_q: int, like, stream=None):
    b = _b()
    need = b.workspace_size(_byref(desc), max_q)
    if need == 0:
        raise _m.MoEError(_m.MOE_ERR_UNSUPPORTED, "moe_paged_attention_workspace_size")
    ws = _new(stream, like, (need,), b.u8)
    _m._check(_m.lib().moe_workspace_init(ws.data_ptr(), need, _stream_of(stream, ws)), "moe_workspace_init")
    return ws


def moe_paged_attention_workspace(T: int, B: int, Hq: int, Hkv: int, D: int, max_q: int, device="cuda"):
    """An initialised workspace for moe_paged_attention calls of these sizes (and for the cache calls of any size)."""
    return _workspace(_m.moe_kv_desc(B, T, Hq, Hkv, D, 16, 0, 0), max_q, _b().torch.empty(0, device=device))


def moe_paged_attention(q, cache: KVCache, q_start, kv_len, page_table, max_q: int, scale: Optional[float] = None,
                        causal: bool = True, window: int = 0, out=None, ws=None, stream=None):
    """Softmax attention of the new queries q [T, Hq, D] over their sequences' cached tokens; returns [T, Hq, D] bf16.
    scale defaults to D ** -0.5; max_q: at least the new tokens of any one sequence (more than T counts as T)."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    T, Hq = q.shape[0], q.shape[1]
    max_q = min(max_q, T)
    qp, qs = _rows(q, "q", Hq, D)
    d = _m.moe_kv_desc(B, T, Hq, Hkv, D, page, n_pages, max_pages)
    starts, lens = _need(q_start, "q_start", b.i32, (B + 1,)), _need(kv_len, "kv_len", b.i32, (B,))
    ws = _workspace(d, max_q, q, stream) if ws is None else _status_ws(q, ws)
    if out is None:
        out = _new(stream, q, (T, Hq, D))
        op = out.data_ptr()
    else:
        op = _need(out, "out", b.bf16, (T, Hq, D))
    status = b.attention(_byref(d), qp, qs, starts, lens, table, _byref(kv), max_q, D ** -0.5 if scale is None else scale,
                         causal, window, op, ws.data_ptr(), ws.numel(), _stream_of(stream, q))
    if status:
        _m._check(status, "moe_paged_attention")
    return out


class AttentionLayer:
    """The attention of one decoder layer with its own cache and workspace: append, then attend.

    ``forward`` takes the rows of the merged projection [T, (Hq + 2 Hkv) * D] (query heads, key heads, value heads)
    and returns the attention output [T, Hq * D], the input of the output projection.  Pages are the caller's to hand
    out: page_table names them, and a page freed by one sequence may be given to another at any time.  Calls of one layer share its
    workspace and run one after another; ``status`` says what they found."""

    def __init__(self, n_pages: int, Hq: int, Hkv: int, D: int = 128, page: int = 64, max_pos: int = 32768,
                 rot_dim: Optional[int] = None, rope_base: float = 1e6, interleaved: bool = False, q_norm_weight=None,
                 k_norm_weight=None, eps: float = 1e-6, scale: Optional[float] = None, window: int = 0, device="cuda"):
        if window < 0 or (scale is not None and not 0.0 < scale < float("inf")):
            raise ValueError(f"expected window >= 0 and a positive finite scale, got {window} and {scale}")
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.cache = KVCache.empty(n_pages, Hkv, page, D, device)
        rot_dim = D if rot_dim is None else rot_dim
        self.cos_sin = moe_rope_table(max_pos, rot_dim, rope_base, device=device) if rot_dim else None
        self.interleaved, self.q_norm_weight, self.k_norm_weight, self.eps = interleaved, q_norm_weight, k_norm_weight, eps
        self.scale, self.window = scale, window
        self.ws, self._outgrown = _status_ws(self.cache.k_codes, None), []

    def forward(self, qkv, q_start, kv_len, page_table, max_q: int, out=None, stream=None):
        T, B = qkv.shape[0], page_table.shape[0]
        q, k, v = qkv.view(T, self.Hq + 2 * self.Hkv, self.D).split([self.Hq, self.Hkv, self.Hkv], dim=1)
        # What the attention refuses is refused before the tokens are in the cache.
        max_q = min(max_q, T)
        if max_q * B < T or (max_q < 1 and T > 0):
            raise _m.MoEError(_m.MOE_ERR_INVALID_ARG, "AttentionLayer.forward: max_q")
        if out is not None:
            if out.numel() != T * self.Hq * self.D or not out.is_contiguous():
                raise ValueError(f"out: expected a contiguous tensor [{T}, {self.Hq * self.D}], got {tuple(out.shape)}")
            out = out.view(T, self.Hq, self.D)
            _need(out, "out", _b().bf16, out.shape)
        d = _m.moe_kv_desc(B, T, self.Hq, self.Hkv, self.D, 16, 0, 0)
        ws = self._workspace_for(d, max_q, stream)
        rq = moe_kv_append(q, k, v, self.cache, q_start, kv_len, page_table, self.cos_sin, None, self.interleaved,
                           self.q_norm_weight, self.k_norm_weight, self.eps, ws=ws, stream=stream)
        o = moe_paged_attention(rq, self.cache, q_start, kv_len, page_table, max_q, self.scale, True, self.window,
                                out, ws, stream)
        if ws is not self.ws:
            with _b().torch.cuda.stream(stream):
                self.ws[:_b().status_bytes].bitwise_or_(ws[:_b().status_bytes])
        return o.view(T, self.Hq * self.D)

    def _workspace_for(self, d, max_q: int, stream):
        """The layer's workspace, a larger one from now on if this call needs it.

        The smaller one is kept: a captured graph, or a call still running on another stream, goes on using it (there are few
        sizes).  A call that is being captured does not make the layer's workspace grow -- clearing the new one's status word would
        become a part of the graph, done again by every replay -- but has one of its own, whose status is added to the layer's."""
        b = _b()
        if self.ws.numel() >= b.workspace_size(_byref(d), max_q):
            return self.ws
        with b.torch.cuda.stream(stream):
            ws = _workspace(d, max_q, self.ws, stream)
            if not b.torch.cuda.is_current_stream_capturing():
                self._outgrown.append(self.ws)
                ws[:b.status_bytes].copy_(self.ws[:b.status_bytes])  # what an earlier call reported stays readable
                self.ws = ws
        return ws

    def status(self, stream=None) -> int:
        """What the calls so far reported, MOE_OK or the first error found (synchronises): that of the present workspace or, from graphs
        captured before it grew, of the ones before it."""
        found = (_m.moe_get_device_status(ws, stream) for ws in (self.ws, *self._outgrown))
        return next((s for s in found if s != _m.MOE_OK), _m.MOE_OK)

    def clear_status(self, stream=None) -> None:
        """Forgets what was reported."""
        for ws in (self.ws, *self._outgrown):
            _m.moe_workspace_init(ws, stream)
