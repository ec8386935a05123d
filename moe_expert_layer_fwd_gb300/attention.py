"""Attention over a paged 8-bit key/value cache: Python binding of the moe_kv_*, moe_rope_* and moe_paged_attention* entry points.

Argument marshalling only, as in the rest of the package; ``include/moe.h`` states formats, limits and errors.
"""
from __future__ import annotations

import ctypes
import operator
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
        self.rope_rows, self.append_at, self.shared = lib.moe_rope_rows, lib.moe_kv_append_at, lib.moe_paged_attention_shared
        self.weights, self.evict, self.shared_size = lib.moe_kv_weights, lib.moe_kv_evict, lib.moe_paged_attention_shared_workspace_size
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


def _count(n):
    """A window or a number of tokens as the int of the C interface: beyond all tokens is all of them, and below none is refused
    there.  (ctypes would keep the low bits.)"""
    return max(-1, min(n, (1 << 31) - 1))


def _need_aligned(what: str, *addresses):
    """Refuses what the library refuses, before anything else of the call has run."""
    if any(a and a & 15 for a in addresses):
        raise _m.MoEError(_m.MOE_ERR_INVALID_ARG, f"{what}: expected tensors that begin on 16 bytes")


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


def moe_kv_workspace(device="cuda"):
    """A workspace for the calls that need no more than a status word: all of this module but the attention's."""
    return _b().torch.zeros(max(_b().status_bytes, 256), dtype=_b().u8, device=device)


def _axis_bytes(axes, n_axes: int, rot_dim: int) -> bytes:
    """The axis of each frequency as a byte.  Element by element: bytes() of an array or a tensor would be its memory."""
    codes = bytes(axes if type(axes) in (list, tuple, bytes) else [operator.index(a) for a in axes])  # (raises for what is no byte)
    if len(codes) * 2 != rot_dim:
        raise ValueError(f"axes: expected one for each of {rot_dim // 2} frequencies, got {len(codes)}")
    if codes and max(codes) >= n_axes:
        raise ValueError(f"axes: expected numbers of the {n_axes} axes, got {tuple(codes)}")
    return codes


def moe_rope_rows(positions, axes, cos_sin, rows=None, ws=None, stream=None):
    """The rotation of each new token, rows [T, rot_dim] fp32 for moe_kv_append_at: frequency f turns by positions[axes[f], t].
    positions [n_axes, T] int32 (a row's tokens dense; one row expanded will do), axes: rot_dim / 2 integers (a list, an array), cos_sin as moe_rope_table makes it."""
    b = _b()
    if positions.dim() != 2 or positions.dtype is not b.i32 or not positions.is_cuda:
        raise ValueError(f"positions: expected a CUDA int32 tensor [n_axes, T], got {positions.dtype} {tuple(positions.shape)}")
    n_axes, T = positions.shape
    if T > 1 and positions.stride(1) != 1:
        raise ValueError(f"positions: the tokens of an axis must be dense, got strides {positions.stride()}")
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin: expected [max_pos, rot_dim], got {tuple(cos_sin.shape)}")
    max_pos, rot_dim = cos_sin.shape
    codes = _axis_bytes(axes, n_axes, rot_dim)
    cs = _need(cos_sin, "cos_sin", b.f32, cos_sin.shape)
    rp = None if rows is None else _need(rows, "rows", b.f32, (T, rot_dim))
    ws = _status_ws(positions, ws, stream)
    if rows is None:
        rows = _new(stream, positions, (T, rot_dim), b.f32)
        rp = rows.data_ptr()
    stride = positions.stride(0) if n_axes > 1 else T
    status = b.rope_rows(n_axes, T, positions.data_ptr(), stride, codes, cs, max_pos, rot_dim, rp, ws.data_ptr(), ws.numel(),
                         _stream_of(stream, positions))
    if status:
        _m._check(status, "moe_rope_rows")
    return rows


def moe_kv_append_at(q, k, v, cache: KVCache, q_start, kv_len, page_table, rows, interleaved: bool = False, q_norm_weight=None,
                     k_norm_weight=None, eps: float = 1e-6, q_out=None, ws=None, stream=None):
    """moe_kv_append with the rotation of token t in rows[t] (of moe_rope_rows), wherever in the cache it goes."""
    if rows.dim() != 2 or rows.shape[0] != k.shape[0]:
        raise ValueError(f"rows: expected [{k.shape[0]}, rot_dim], got {tuple(rows.shape)}")
    return _append(q, k, v, cache, q_start, kv_len, page_table, rows, rows.shape[1], interleaved, q_norm_weight, k_norm_weight, eps, q_out,
                   ws, stream, True)


def moe_kv_append(q, k, v, cache: KVCache, q_start, kv_len, page_table, cos_sin=None, rot_dim: Optional[int] = None,
                  interleaved: bool = False, q_norm_weight=None, k_norm_weight=None, eps: float = 1e-6, q_out=None,
                  ws=None, stream=None):
    """Normalises (when weights are given) and rotates the new queries and keys, stores the new keys and values in the
    cache; returns the queries [T, Hq, D] (None when q is None).  q, k, v may be views of one projection's rows."""
    return _append(q, k, v, cache, q_start, kv_len, page_table, cos_sin, rot_dim, interleaved, q_norm_weight, k_norm_weight, eps, q_out,
                   ws, stream, False)


def _append(q, k, v, cache, q_start, kv_len, page_table, cos_sin, rot_dim, interleaved, q_norm_weight, k_norm_weight, eps, q_out, ws,
            stream, by_token):
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
    if by_token:
        status = b.append_at(_byref(d), qp, qs, kp, ks, vp, vs, starts, lens, table, cs, rot_dim, interleaved, qw, kw, eps, op,
                             _byref(kv), ws.data_ptr(), ws.numel(), _stream_of(stream, k))
    else:
        status = b.append(_byref(d), qp, qs, kp, ks, vp, vs, starts, lens, table, cs, max_pos, rot_dim, interleaved, qw, kw, eps,
                          op, _byref(kv), ws.data_ptr(), ws.numel(), _stream_of(stream, k))
    if status:
        _m._check(status, "moe_kv_append_at" if by_token else "moe_kv_append")
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
                         causal, _count(window), op, ws.data_ptr(), ws.numel(), _stream_of(stream, q))
    if status:
        _m._check(status, "moe_paged_attention")
    return out


def _prefix_struct(prefix, T: int):
    """moe_kv_prefix of (q_start [n+1], len [n], page_table [n, max_pages], max_q)."""
    b = _b()
    q_start, length, page_table, max_q = prefix
    table, n, max_pages = _table(page_table)
    return _m.moe_kv_prefix(n, max_pages, min(max_q, T), _need(q_start, "prefix q_start", b.i32, (n + 1,)),
                            _need(length, "prefix len", b.i32, (n,)), table)


def moe_paged_attention_shared_workspace(T: int, B: int, Hq: int, Hkv: int, D: int, max_q: int, n_prefixes: int = 0,
                                         max_prefix_q: int = 0, device="cuda"):
    """An initialised workspace for moe_paged_attention_shared calls of these sizes (n_prefixes = 0: without prefixes).  A call of
    fewer tokens, or of another max_q, may need a larger one."""
    p = _m.moe_kv_prefix(n_prefixes, 0, min(max_prefix_q, T), None, None, None) if n_prefixes else None
    return _shared_workspace(_m.moe_kv_desc(B, T, Hq, Hkv, D, 16, 0, 0), min(max_q, T), p, _b().torch.empty(0, device=device))


def _shared_workspace(desc, max_q: int, prefix, like, stream=None):
    b = _b()
    need = b.shared_size(_byref(desc), max_q, None if prefix is None else _byref(prefix))
    if need == 0:
        raise _m.MoEError(_m.MOE_ERR_UNSUPPORTED, "moe_paged_attention_shared_workspace_size")
    ws = _new(stream, like, (need,), b.u8)
    _m._check(_m.lib().moe_workspace_init(ws.data_ptr(), need, _stream_of(stream, ws)), "moe_workspace_init")
    return ws


def moe_paged_attention_shared(q, cache: KVCache, q_start, kv_len, page_table, max_q: int, prefix=None, scale: Optional[float] = None,
                               causal: bool = True, window: int = 0, out=None, lse=None, ws=None, stream=None):
    """moe_paged_attention of sequences that share prefixes, with the rows' denominators: returns (out [T, Hq, D] bf16,
    lse [T, Hq] fp32).

    prefix: None, or (q_start [n+1], len [n], page_table [n, max_pages], max_q): tokens q_start[i] .. q_start[i+1] - 1 see the
    len[i] tokens of prefix i before their sequence's own; max_q: at least the tokens of any one prefix's readers."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    T, Hq = q.shape[0], q.shape[1]
    max_q = min(max_q, T)
    qp, qs = _rows(q, "q", Hq, D)
    d = _m.moe_kv_desc(B, T, Hq, Hkv, D, page, n_pages, max_pages)
    starts, lens = _need(q_start, "q_start", b.i32, (B + 1,)), _need(kv_len, "kv_len", b.i32, (B,))
    p = None if prefix is None else _prefix_struct(prefix, T)
    op = None if out is None else _need(out, "out", b.bf16, (T, Hq, D))
    lp = None if lse is None else _need(lse, "lse", b.f32, (T, Hq))
    ws = _shared_workspace(d, max_q, p, q, stream) if ws is None else _status_ws(q, ws)
    if out is None:
        out = _new(stream, q, (T, Hq, D))
        op = out.data_ptr()
    if lse is None:
        lse = _new(stream, q, (T, Hq), b.f32)
        lp = lse.data_ptr()
    status = b.shared(_byref(d), qp, qs, starts, lens, table, _byref(kv), max_q, D ** -0.5 if scale is None else scale, causal,
                      _count(window), None if p is None else _byref(p), op, lp, ws.data_ptr(), ws.numel(), _stream_of(stream, q))
    if status:
        _m._check(status, "moe_paged_attention_shared")
    return out, lse


def moe_kv_weights(q, lse, cache: KVCache, q_start, kv_len, page_table, max_q: int, weight=None, out=None, scale: Optional[float] = None,
                   causal: bool = True, window: int = 0, ws=None, stream=None):
    """Adds what the new queries q [T, Hq, D] give to each cached token of their sequences, with the denominators lse [T, Hq] of
    moe_paged_attention_shared, to weight [n_pages, Hkv, page] fp32 (None: from zero on), in place or into out; returns that."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    T, Hq = q.shape[0], q.shape[1]
    max_q = min(max_q, T)
    qp, qs = _rows(q, "q", Hq, D)
    d = _m.moe_kv_desc(B, T, Hq, Hkv, D, page, n_pages, max_pages)
    starts, lens = _need(q_start, "q_start", b.i32, (B + 1,)), _need(kv_len, "kv_len", b.i32, (B,))
    lp, shape = _need(lse, "lse", b.f32, (T, Hq)), (n_pages, Hkv, page)
    wp = None if weight is None else _need(weight, "weight", b.f32, shape)
    op = wp if out is None else _need(out, "out", b.f32, shape)
    if op is None:
        raise ValueError("out: needed when there is no weight to add to")
    ws = _status_ws(q, ws, stream)
    status = b.weights(_byref(d), qp, qs, lp, starts, lens, table, _byref(kv), max_q, D ** -0.5 if scale is None else scale, causal,
                       _count(window), wp, op, ws.data_ptr(), ws.numel(), _stream_of(stream, q))
    if status:
        _m._check(status, "moe_kv_weights")
    return weight if out is None else out


def moe_kv_evict(cache: KVCache, weight, kv_len, page_table, keep, new_table, sink: int = 0, recent: int = 0, new_len=None, kept=None,
                 ws=None, stream=None):
    """Packs the keep[b] tokens of the largest weight [n_pages, Hkv, page] of each sequence and head, with their weights, into the
    pages of new_table; the first ``sink`` and last ``recent`` tokens stay before all others (of keep[b] below their number the first);
    returns (new_len [B], kept [B, Hkv, new_max_pages * page]: the tokens that stayed, then -1)."""
    b = _b()
    kv = cache._struct()
    n_pages, Hkv, page, D = cache[0].shape
    table, B, max_pages = _table(page_table)
    new, new_B, new_max = _table(new_table)
    if new_B != B:
        raise ValueError(f"new_table: expected [{B}, new_max_pages], got {tuple(new_table.shape)}")
    d = _m.moe_kv_desc(B, 0, Hkv, Hkv, D, page, n_pages, max_pages)
    wp = _need(weight, "weight", b.f32, (n_pages, Hkv, page))
    lens, keeps = _need(kv_len, "kv_len", b.i32, (B,)), _need(keep, "keep", b.i32, (B,))
    np_ = None if new_len is None else _need(new_len, "new_len", b.i32, (B,))
    kp = None if kept is None else _need(kept, "kept", b.i32, (B, Hkv, new_max * page))
    ws = _status_ws(weight, ws, stream)
    if new_len is None:
        new_len = _new(stream, weight, (B,), b.i32)
        np_ = new_len.data_ptr()
    if kept is None:
        kept = _new(stream, weight, (B, Hkv, new_max * page), b.i32)
        kp = kept.data_ptr()
    status = b.evict(_byref(d), wp, lens, table, keeps, _count(sink), _count(recent), new, new_max, _byref(kv), np_, kp,
                     ws.data_ptr(), ws.numel(), _stream_of(stream, weight))
    if status:
        _m._check(status, "moe_kv_evict")
    return new_len, kept


class AttentionLayer:
    """The attention of one decoder layer with its own cache and workspace: append, then attend.

    ``forward`` takes the rows of the merged projection [T, (Hq + 2 Hkv) * D] (query heads, key heads, value heads)
    and returns the attention output [T, Hq * D], the input of the output projection.  Pages are the caller's to hand
    out: page_table names them, and a page freed by one sequence may be given to another at any time.  Calls of one layer share its
    workspace and run one after another; ``status`` says what they found.

    Long conversations: ``rows`` (of ``rotation``) turns the tokens by given positions instead of their places in the cache; ``prefix``
    lets sequences share what another one stored; with ``track_weights`` every call adds the attention weights that the sequences' own
    cached tokens got to ``weight`` (not those of a prefix's tokens, whose readers' weights moe_kv_weights gives in a call of its own: see
    include/moe.h), and ``evict`` packs the tokens of the largest ones into new pages.  With weights, a page is in one row of
    ``page_table`` only; after an eviction a ``window`` counts the tokens that stayed."""

    def __init__(self, n_pages: int, Hq: int, Hkv: int, D: int = 128, page: int = 64, max_pos: int = 32768,
                 rot_dim: Optional[int] = None, rope_base: float = 1e6, interleaved: bool = False, q_norm_weight=None,
                 k_norm_weight=None, eps: float = 1e-6, scale: Optional[float] = None, window: int = 0, device="cuda",
                 track_weights: bool = False):
        if window < 0 or (scale is not None and not 0.0 < ctypes.c_float(scale).value < float("inf")):
            raise ValueError(f"expected window >= 0 and a scale that is positive and finite in fp32, got {window} and {scale}")
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.cache = KVCache.empty(n_pages, Hkv, page, D, device)
        rot_dim = D if rot_dim is None else rot_dim
        self.cos_sin = moe_rope_table(max_pos, rot_dim, rope_base, device=device) if rot_dim else None
        self.interleaved, self.q_norm_weight, self.k_norm_weight, self.eps = interleaved, q_norm_weight, k_norm_weight, eps
        self.scale, self.window = scale, window
        self.ws, self._outgrown = _status_ws(self.cache.k_codes, None), []
        self.weight = _b().torch.zeros((n_pages, Hkv, page), dtype=_b().f32, device=device) if track_weights else None

    def rotation(self, positions, axes=None, rows=None, stream=None):
        """The rows of ``forward`` for tokens at positions [n_axes, T] (int32), frequency f on axis axes[f] (the first one): once a
        step serves all layers of a model."""
        if self.cos_sin is None:
            raise ValueError("rotation: this layer rotates nothing")
        axes = [0] * (self.cos_sin.shape[1] // 2) if axes is None else axes
        return moe_rope_rows(positions, axes, self.cos_sin, rows, self.ws, stream)

    def forward(self, qkv, q_start, kv_len, page_table, max_q: int, out=None, stream=None, rows=None, prefix=None):
        """rows: None (a token's position is its place in the cache) or [T, rot_dim] of ``rotation``.  prefix: None, or as in
        moe_paged_attention_shared; the positions of tokens behind one go on from its end, so rows must be given."""
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
            _need_aligned("out", _need(out, "out", _b().bf16, out.shape))
        p = None
        if prefix is not None:
            if self.window or (rows is None and self.cos_sin is not None):
                raise ValueError("prefix: not with a window, and not without the rows of its readers' positions")
            p = _prefix_struct(prefix, T)
            if p.n < 1 or p.max_q * p.n < T or (p.max_q < 1 and T > 0):
                raise _m.MoEError(_m.MOE_ERR_INVALID_ARG, "AttentionLayer.forward: prefix")
            _need_aligned("prefix", p.q_start, p.len, p.page_table)
        if rows is not None:
            if self.cos_sin is None:
                raise ValueError("rows: this layer rotates nothing")
            _need(rows, "rows", _b().f32, (T, self.cos_sin.shape[1]))
        shared = p is not None or self.weight is not None
        n_pages, _, page, _ = self.cache.k_codes.shape
        d = _m.moe_kv_desc(B, T, self.Hq, self.Hkv, self.D, page, n_pages, page_table.shape[-1])
        ws = self._workspace_for(d, max_q, stream, p)
        if rows is None:
            rq = moe_kv_append(q, k, v, self.cache, q_start, kv_len, page_table, self.cos_sin, None, self.interleaved,
                               self.q_norm_weight, self.k_norm_weight, self.eps, ws=ws, stream=stream)
        else:
            rq = moe_kv_append_at(q, k, v, self.cache, q_start, kv_len, page_table, rows, self.interleaved, self.q_norm_weight,
                                  self.k_norm_weight, self.eps, ws=ws, stream=stream)
        if shared:
            o, lse = moe_paged_attention_shared(rq, self.cache, q_start, kv_len, page_table, max_q, prefix, self.scale, True,
                                                self.window, out, None, ws, stream)
        else:
            o = moe_paged_attention(rq, self.cache, q_start, kv_len, page_table, max_q, self.scale, True, self.window,
                                    out, ws, stream)
        if self.weight is not None:
            moe_kv_weights(rq, lse, self.cache, q_start, kv_len, page_table, max_q, self.weight, None, self.scale, True, self.window, ws,
                           stream)
        if ws is not self.ws:
            with _b().torch.cuda.stream(stream):
                self.ws[:_b().status_bytes].bitwise_or_(ws[:_b().status_bytes])
        return o.view(T, self.Hq * self.D)

    def evict(self, kv_len, page_table, keep, new_table, sink: int = 0, recent: int = 0, stream=None):
        """Packs the keep[b] tokens of the largest weights of each sequence into the pages of new_table (moe_kv_evict); returns
        (new_len, kept).  The old pages are free then, and the next token's place is new_len[b], its position what it was."""
        if self.weight is None:
            raise ValueError("evict: the layer has no weights (track_weights)")
        return moe_kv_evict(self.cache, self.weight, kv_len, page_table, keep, new_table, sink, recent, ws=self.ws, stream=stream)

    def _workspace_for(self, d, max_q: int, stream, prefix=None):
        """The layer's workspace, a larger one from now on if this call needs it.

        The smaller one is kept: a captured graph, or a call still running on another stream, goes on using it (there are few
        sizes).  A call that is being captured does not make the layer's workspace grow -- clearing the new one's status word would
        become a part of the graph, done again by every replay -- but has one of its own, whose status is added to the layer's."""
        b = _b()
        need = b.workspace_size(_byref(d), max_q) if prefix is None else b.shared_size(_byref(d), max_q, _byref(prefix))
        if self.ws.numel() >= need > 0:
            return self.ws
        with b.torch.cuda.stream(stream):
            ws = _workspace(d, max_q, self.ws, stream) if prefix is None else _shared_workspace(d, max_q, prefix, self.ws, stream)
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
