"""Attention over a paged 8-bit key/value cache: Python binding of the moe_kv_* and moe_paged_attention entry points.

Argument marshalling only, as in the rest of the package; ``include/moe.h`` states formats, limits and errors.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import moe_expert_layer_fwd_gb300 as _m


def _on(stream):
    """Allocations made for a call belong to the stream that the call runs on."""
    return contextlib.nullcontext() if stream is None else _m._torch().cuda.stream(stream)


def _need(t, what: str, dtype, shape=None):
    if t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return _m._ptr(t)


def _rows(t, what: str, heads: int, D: int):
    """(pointer, token stride) of a [T, heads, D] bf16 tensor whose heads are dense."""
    if t.dtype != _m._torch().bfloat16 or t.dim() != 3 or tuple(t.shape[1:]) != (heads, D):
        raise ValueError(f"{what}: expected a bfloat16 tensor [T, {heads}, {D}], got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if t.stride(2) != 1 or t.stride(1) != D:
        raise ValueError(f"{what}: the heads of a token must be dense, got strides {t.stride()}")
    stride = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), heads * D)
    return t.data_ptr(), stride


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
        u8 = _m._torch().uint8
        shape = self.k_codes.shape
        if len(shape) != 4:
            raise ValueError(f"k_codes: expected [n_pages, Hkv, page, D], got {tuple(shape)}")
        return _m.moe_kv_cache(_need(self.k_codes, "k_codes", u8), _need(self.v_codes, "v_codes", u8, shape),
                               _need(self.k_scale, "k_scale", u8, shape[:2]),
                               _need(self.v_scale, "v_scale", u8, shape[:2]))


def _desc(cache: KVCache, page_table, T: int, Hq: int) -> "_m.moe_kv_desc":
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected [B, max_pages], got {tuple(page_table.shape)}")
    n_pages, Hkv, page, D = cache.k_codes.shape
    return _m.moe_kv_desc(page_table.shape[0], T, Hq, Hkv, D, page, n_pages, page_table.shape[1])


def _status_ws(device, ws):
    return _m._ws(_m.lib().moe_status_bytes(), device, ws)


def moe_rope_table(max_pos: int, rot_dim: int = 128, base: float = 1e6, cos_sin=None, device="cuda", stream=None):
    """cos_sin [max_pos, rot_dim] fp32 of moe_kv_append: row p = cos(p f_i) | sin(p f_i), f_i = base^(-2i/rot_dim)."""
    torch = _m._torch()
    with _on(stream):
        if cos_sin is None:
            cos_sin = torch.empty((max_pos, rot_dim), dtype=torch.float32, device=device)
    _m._check(_m.lib().moe_rope_table(max_pos, rot_dim, base, _need(cos_sin, "cos_sin", torch.float32,
                                                                  (max_pos, rot_dim)), _m._stream(stream)),
              "moe_rope_table")
    return cos_sin


def moe_kv_append(q, k, v, cache: KVCache, q_start, kv_len, page_table, cos_sin=None, rot_dim: Optional[int] = None,
                  interleaved: bool = False, q_norm_weight=None, k_norm_weight=None, eps: float = 1e-6, q_out=None,
                  ws=None, stream=None):
    """Normalises (when weights are given) and rotates the new queries and keys, stores the new keys and values in the
    cache; returns the queries [T, Hq, D] (None when q is None).  q, k, v may be views of one projection's rows."""
    torch = _m._torch()
    i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32
    kv = cache._struct()
    Hkv, D = cache.k_codes.shape[1], cache.k_codes.shape[3]
    T, B = k.shape[0], page_table.shape[0]
    if v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("q, k and v must have the same number of tokens")
    if rot_dim is None:
        rot_dim = cos_sin.shape[1] if cos_sin is not None else 0
    Hq = q.shape[1] if q is not None else Hkv
    kp, ks = _rows(k, "k", Hkv, D)
    vp, vs = _rows(v, "v", Hkv, D)
    qp, qs = _rows(q, "q", Hq, D) if q is not None else (None, 0)
    with _on(stream):
        if q is not None and q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=bf16, device=k.device)
        ws = _status_ws(k.device, ws)
    d = _desc(cache, page_table, T, Hq)
    _m._check(_m.lib().moe_kv_append(
        ctypes.byref(d), qp, qs, kp, ks, vp, vs, _need(q_start, "q_start", i32, (B + 1,)),
        _need(kv_len, "kv_len", i32, (B,)), _need(page_table, "page_table", i32),
        _need(cos_sin, "cos_sin", f32, (cos_sin.shape[0], rot_dim)) if cos_sin is not None else None,
        cos_sin.shape[0] if cos_sin is not None else 0, rot_dim, int(interleaved),
        _need(q_norm_weight, "q_norm_weight", bf16, (D,)) if q_norm_weight is not None else None,
        _need(k_norm_weight, "k_norm_weight", bf16, (D,)) if k_norm_weight is not None else None, eps,
        _need(q_out, "q_out", bf16, (T, Hq, D)) if q_out is not None else None, ctypes.byref(kv), _m._ptr(ws),
        ws.numel(), _m._stream(stream)), "moe_kv_append")
    return q_out


def moe_kv_gather(cache: KVCache, start, out_start, page_table, n_rows: int, k=None, v=None, ws=None, stream=None):
    """Reads cached tokens back: returns (k, v) [n_rows, Hkv, D] bf16, where rows out_start[b] .. out_start[b+1] - 1
    are the tokens of sequence b from start[b] on."""
    torch = _m._torch()
    i32, bf16 = torch.int32, torch.bfloat16
    kv = cache._struct()
    Hkv, D = cache.k_codes.shape[1], cache.k_codes.shape[3]
    B = page_table.shape[0]
    shape = (n_rows, Hkv, D)
    with _on(stream):
        k = torch.empty(shape, dtype=bf16, device=page_table.device) if k is None else k
        v = torch.empty(shape, dtype=bf16, device=page_table.device) if v is None else v
        ws = _status_ws(page_table.device, ws)
    d = _desc(cache, page_table, 0, Hkv)
    _m._check(_m.lib().moe_kv_gather(
        ctypes.byref(d), _need(start, "start", i32, (B,)), _need(out_start, "out_start", i32, (B + 1,)),
        _need(page_table, "page_table", i32), ctypes.byref(kv), n_rows, _need(k, "k", bf16, shape),
        _need(v, "v", bf16, shape), _m._ptr(ws), ws.numel(), _m._stream(stream)), "moe_kv_gather")
    return k, v


def moe_paged_attention_workspace(T: int, B: int, Hq: int, Hkv: int, D: int, max_q: int, device="cuda"):
    """An initialised workspace for moe_paged_attention calls of these sizes (and for the cache calls of any size)."""
    torch = _m._torch()
    d = _m.moe_kv_desc(B, T, Hq, Hkv, D, 16, 0, 0)
    need = _m.lib().moe_paged_attention_workspace_size(ctypes.byref(d), max_q)
    if need == 0:
        raise _m.MoEError(_m.MOE_ERR_UNSUPPORTED, "moe_paged_attention_workspace_size")
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    _m.moe_workspace_init(ws)
    return ws


def moe_paged_attention(q, cache: KVCache, q_start, kv_len, page_table, max_q: int, scale: Optional[float] = None,
                        causal: bool = True, window: int = 0, out=None, ws=None, stream=None):
    """Softmax attention of the new queries q [T, Hq, D] over their sequences' cached tokens; returns [T, Hq, D] bf16.
    scale defaults to D ** -0.5; max_q: at least the new tokens of any one sequence."""
    torch = _m._torch()
    i32, bf16 = torch.int32, torch.bfloat16
    kv = cache._struct()
    D = cache.k_codes.shape[3]
    T, Hq = q.shape[0], q.shape[1]
    B = page_table.shape[0]
    qp, qs = _rows(q, "q", Hq, D)
    d = _desc(cache, page_table, T, Hq)
    with _on(stream):
        if out is None:
            out = torch.empty((T, Hq, D), dtype=bf16, device=q.device)
        need = _m.lib().moe_paged_attention_workspace_size(ctypes.byref(d), max_q)
        if ws is None or ws.numel() < need:
            ws = torch.empty(max(int(need), 256), dtype=torch.uint8, device=q.device)
            _m.moe_workspace_init(ws, stream)
    _m._check(_m.lib().moe_paged_attention(
        ctypes.byref(d), qp, qs, _need(q_start, "q_start", i32, (B + 1,)), _need(kv_len, "kv_len", i32, (B,)),
        _need(page_table, "page_table", i32), ctypes.byref(kv), max_q, D ** -0.5 if scale is None else scale,
        int(causal), window, _need(out, "out", bf16, (T, Hq, D)), _m._ptr(ws), ws.numel(), _m._stream(stream)),
        "moe_paged_attention")
    return out


class AttentionLayer:
    """The attention of one decoder layer with its own cache and workspace: append, then attend.

    ``forward`` takes the rows of the merged projection [T, (Hq + 2 Hkv) * D] (query heads, key heads, value heads)
    and returns the attention output [T, Hq * D], the input of the output projection.  Pages are the caller's to hand
    out: page_table names them, and a page freed by one sequence may be given to another at any time."""

    def __init__(self, n_pages: int, Hq: int, Hkv: int, D: int = 128, page: int = 64, max_pos: int = 32768,
                 rot_dim: Optional[int] = None, rope_base: float = 1e6, interleaved: bool = False, q_norm_weight=None,
                 k_norm_weight=None, eps: float = 1e-6, scale: Optional[float] = None, window: int = 0, device="cuda"):
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.cache = KVCache.empty(n_pages, Hkv, page, D, device)
        rot_dim = D if rot_dim is None else rot_dim
        self.cos_sin = moe_rope_table(max_pos, rot_dim, rope_base, device=device) if rot_dim else None
        self.interleaved, self.q_norm_weight, self.k_norm_weight, self.eps = interleaved, q_norm_weight, k_norm_weight, eps
        self.scale, self.window = scale, window
        self.ws = _status_ws(self.cache.k_codes.device, None)

    def forward(self, qkv, q_start, kv_len, page_table, max_q: int, out=None, stream=None):
        T = qkv.shape[0]
        q, k, v = qkv.view(T, self.Hq + 2 * self.Hkv, self.D).split([self.Hq, self.Hkv, self.Hkv], dim=1)
        d = _desc(self.cache, page_table, T, self.Hq)
        need = _m.lib().moe_paged_attention_workspace_size(ctypes.byref(d), max_q)
        if self.ws.numel() < need:
            with _on(stream):
                self.ws = _m._torch().empty(need, dtype=self.ws.dtype, device=self.ws.device)
                _m.moe_workspace_init(self.ws, stream)
        rq = moe_kv_append(q, k, v, self.cache, q_start, kv_len, page_table, self.cos_sin, None, self.interleaved,
                           self.q_norm_weight, self.k_norm_weight, self.eps, ws=self.ws, stream=stream)
        o = moe_paged_attention(rq, self.cache, q_start, kv_len, page_table, max_q, self.scale, True, self.window,
                                out.view(T, self.Hq, self.D) if out is not None else None, self.ws, stream)
        return o.view(T, self.Hq * self.D)
