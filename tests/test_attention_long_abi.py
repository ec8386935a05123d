"""Refusals of the entry points for long conversations: every check answers before anything is launched (CPU)."""
import ctypes

import pytest
import torch

import moe_expert_layer_fwd_gb300 as moe
from test_attention_abi import A, B_, BAD, C_, UNS, L, cache, desc  # noqa: F401

AXES = bytes([0, 1, 2, 0] * 16)


def rows(L, **kw):
    a = dict(n=3, T=5, pos=A + 4, stride=7, axes=AXES, cs=A, max_pos=100, rot=128, rows=B_, ws=A, bytes=256)
    a.update(kw)
    return L.moe_rope_rows(a["n"], a["T"], a["pos"], a["stride"], a["axes"], a["cs"], a["max_pos"], a["rot"], a["rows"], a["ws"],
                           a["bytes"], None)


def append_at(L, d=None, kv=None, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, start=A, lens=A, table=A, rows=A, rot=128, il=0, qn=A, kn=A, eps=1e-6, out=A, ws=A,
             n=256)
    a.update(kw)
    return L.moe_kv_append_at(ctypes.byref(d or desc()), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["start"], a["lens"],
                              a["table"], a["rows"], a["rot"], a["il"], a["qn"], a["kn"], a["eps"], a["out"], ctypes.byref(kv or cache()),
                              a["ws"], a["n"], None)


def prefix(**kw):
    f = dict(n=2, max_pages=4, max_q=3, q_start=A, len=A, page_table=A)
    f.update(kw)
    return moe.moe_kv_prefix(**f)


def shared(L, d=None, kv=None, p=None, none=False, **kw):
    d, p = d or desc(), None if none else ctypes.byref(p or prefix())
    a = dict(q=A, qs=1024, start=A, lens=A, table=A, max_q=2, scale=0.1, causal=1, window=0, out=A, lse=A + 4, ws=A)
    a["n"] = max(256, L.moe_paged_attention_shared_workspace_size(ctypes.byref(d), 2, p))
    a.update(kw)
    return L.moe_paged_attention_shared(ctypes.byref(d), a["q"], a["qs"], a["start"], a["lens"], a["table"], ctypes.byref(kv or cache()),
                                        a["max_q"], a["scale"], a["causal"], a["window"], p, a["out"], a["lse"], a["ws"], a["n"], None)


def weights(L, d=None, kv=None, **kw):
    a = dict(q=A, qs=1024, lse=A, start=A, lens=A, table=A, max_q=2, scale=0.1, causal=1, window=0, w=A, out=A, ws=A, n=256)
    a.update(kw)
    return L.moe_kv_weights(ctypes.byref(d or desc()), a["q"], a["qs"], a["lse"], a["start"], a["lens"], a["table"],
                            ctypes.byref(kv or cache()), a["max_q"], a["scale"], a["causal"], a["window"], a["w"], a["out"], a["ws"],
                            a["n"], None)


def evict(L, d=None, kv=None, **kw):
    a = dict(w=A, lens=A, table=A, keep=A, sink=1, recent=2, new=A, cols=3, new_len=A, kept=A, ws=A, n=256)
    a.update(kw)
    return L.moe_kv_evict(ctypes.byref(d or desc()), a["w"], a["lens"], a["table"], a["keep"], a["sink"], a["recent"], a["new"], a["cols"],
                          ctypes.byref(kv or cache()), a["new_len"], a["kept"], a["ws"], a["n"], None)


CALLS = [append_at, shared, weights, evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=7), BAD), (dict(D=64), UNS),
    (dict(D=0), BAD), (dict(page=48), UNS), (dict(page=256), UNS), (dict(page=0), BAD), (dict(n_pages=-1), BAD),
    (dict(max_pages=-1), BAD), (dict(B=0), BAD), (dict(Hq=2048), UNS), (dict(max_pages=1 << 26), UNS),
    (dict(n_pages=1 << 26), UNS), (dict(B=70000), UNS)])
def test_shapes_are_checked(L, call, kw, status):  # noqa: F811
    assert call(L, desc(**kw)) == status


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field", ["k_codes", "v_codes", "k_scale", "v_scale"])
def test_cache_pointers_are_checked(L, call, field):  # noqa: F811
    assert call(L, kv=cache(**{field: None})) == BAD
    if "codes" in field:
        assert call(L, kv=cache(**{field: A + 8})) == BAD
    assert call(L, kv=cache(k_codes=A, v_codes=A)) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), BAD), (dict(n=2), BAD), (dict(n=9), UNS), (dict(T=-1), BAD), (dict(stride=-1), BAD), (dict(axes=None), BAD),
    (dict(axes=bytes([3] * 64)), BAD), (dict(pos=None), BAD), (dict(pos=A + 2), BAD), (dict(cs=None), BAD), (dict(cs=A + 4), BAD),
    (dict(max_pos=-1), BAD), (dict(rot=0), BAD), (dict(rot=24), UNS), (dict(rot=144), UNS), (dict(rows=None), BAD), (dict(rows=A + 4), BAD),
    (dict(ws=None), BAD), (dict(bytes=128), moe.MOE_ERR_WORKSPACE), (dict(T=0, pos=None, rows=None), moe.MOE_OK)])
def test_rope_rows_arguments(L, kw, status):  # noqa: F811
    assert rows(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(out=None), BAD), (dict(k=A + 2), BAD), (dict(rows=None), BAD),
    (dict(rows=A + 4), BAD), (dict(start=None), BAD), (dict(lens=None), BAD), (dict(table=None), BAD), (dict(qs=1016), BAD),
    (dict(ks=248), BAD), (dict(rot=136), UNS), (dict(rot=24), UNS), (dict(rot=-16), BAD), (dict(eps=-1.0), BAD), (dict(ws=None), BAD),
    (dict(n=128), moe.MOE_ERR_WORKSPACE)])
def test_append_at_arguments(L, kw, status):  # noqa: F811
    assert append_at(L, **kw) == status


@pytest.mark.parametrize("none", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(q=A + 8), BAD), (dict(start=None), BAD), (dict(lens=None), BAD), (dict(table=None), BAD),
    (dict(out=None), BAD), (dict(lse=A + 2), BAD), (dict(max_q=0), BAD), (dict(max_q=4), BAD), (dict(max_q=1), BAD), (dict(max_q=-1), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(window=-1), BAD), (dict(window=3, causal=0), BAD), (dict(qs=1016), BAD),
    (dict(ws=None), BAD), (dict(n=1024), moe.MOE_ERR_WORKSPACE)])
def test_shared_arguments(L, none, kw, status):  # noqa: F811
    assert shared(L, none=none, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), BAD), (dict(n=70000), UNS), (dict(max_pages=-1), BAD), (dict(max_pages=1 << 26), UNS), (dict(max_q=0), BAD),
    (dict(max_q=1), BAD), (dict(max_q=4), BAD), (dict(q_start=None), BAD), (dict(len=None), BAD), (dict(page_table=None), BAD),
    (dict(page_table=A + 4), BAD)])
def test_prefixes_are_checked(L, kw, status):  # noqa: F811
    assert shared(L, p=prefix(**kw)) == status


def test_windows_and_prefixes_exclude_each_other(L):  # noqa: F811
    assert shared(L, window=3) == BAD
    assert shared(L, desc(B=0, T=0), p=prefix(max_q=0)) == moe.MOE_OK


def test_shared_workspace(L):  # noqa: F811
    size = lambda d, p, max_q=2: L.moe_paged_attention_shared_workspace_size(ctypes.byref(d), max_q, None if p is None else ctypes.byref(p))
    d = desc(T=300, B=300)
    assert size(d, None) == L.moe_paged_attention_workspace_size(ctypes.byref(d), 2)
    assert size(d, prefix(q_start=None, len=None, page_table=None, max_q=300)) >= 300 * 8 * 129 * 4 + \
        L.moe_paged_attention_workspace_size(ctypes.byref(d), 300)
    assert size(desc(D=64), prefix()) == 0 and size(d, prefix(n=0)) == 0 and size(d, prefix(max_q=-1)) == 0 and size(d, None, -1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(q=A + 8), BAD), (dict(lse=None), BAD), (dict(lse=A + 4), BAD), (dict(start=None), BAD), (dict(lens=None), BAD),
    (dict(table=None), BAD), (dict(out=None), BAD), (dict(out=A + 4), BAD), (dict(w=A + 4), BAD), (dict(max_q=0), BAD), (dict(max_q=4), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD), (dict(window=-1), BAD), (dict(window=3, causal=0), BAD), (dict(qs=1028), BAD),
    (dict(ws=None), BAD), (dict(n=128), moe.MOE_ERR_WORKSPACE)])
def test_weights_arguments(L, kw, status):  # noqa: F811
    assert weights(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), BAD), (dict(w=A + 4), BAD), (dict(lens=None), BAD), (dict(table=None), BAD), (dict(keep=None), BAD), (dict(sink=-1), BAD),
    (dict(recent=-1), BAD), (dict(new=None), BAD), (dict(cols=0), BAD), (dict(cols=1 << 25), UNS), (dict(new_len=None), BAD),
    (dict(kept=None), BAD), (dict(ws=None), BAD), (dict(n=128), moe.MOE_ERR_WORKSPACE)])
def test_evict_arguments(L, kw, status):  # noqa: F811
    assert evict(L, **kw) == status


def test_evict_of_no_sequence(L):  # noqa: F811
    assert evict(L, desc(B=0, T=0)) == moe.MOE_OK


def test_tensors_are_checked():
    """What the binding refuses: types, shapes and places of tensors."""
    t = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)
    with pytest.raises(ValueError):
        moe.moe_rope_rows(t(2, 5), [0] * 64, t(9, 128, dtype=torch.float32))          # not on a GPU
    with pytest.raises(ValueError):
        moe.moe_rope_rows(t(5), [0] * 64, t(9, 128, dtype=torch.float32))
    kv = moe.KVCache(t(3, 2, 16, 128, dtype=torch.uint8), t(3, 2, 16, 128, dtype=torch.uint8), t(3, 2, dtype=torch.uint8),
                     t(3, 2, dtype=torch.uint8))
    q = t(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_kv_evict(kv, t(3, 2, 16, dtype=torch.float32), t(1), t(1, 3), t(1), t(1, 2))
    with pytest.raises(ValueError):
        moe.moe_kv_weights(q, t(4, 8, dtype=torch.float32), kv, t(2), t(1), t(1, 3), 4)
    with pytest.raises(ValueError):
        moe.moe_paged_attention_shared(q, kv, t(2), t(1), t(1, 3), 4)
