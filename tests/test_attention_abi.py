"""Refusals of the attention entry points: every check answers before anything is launched (CPU)."""
import ctypes

import pytest

import moe_expert_layer_fwd_gb300 as moe

A, B_, C_ = 1 << 20, 1 << 21, 1 << 22   # aligned addresses that nothing reads
BAD = moe.MOE_ERR_INVALID_ARG
UNS = moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from moe_expert_layer_fwd_gb300 import build
    build.build()
    return moe.lib()


def desc(B=2, T=3, Hq=8, Hkv=2, D=128, page=64, n_pages=9, max_pages=4):
    return moe.moe_kv_desc(B, T, Hq, Hkv, D, page, n_pages, max_pages)


def cache(**kw):
    f = dict(k_codes=A, v_codes=B_, k_scale=A + 1, v_scale=B_ + 1)  # scales need no alignment
    f.update(kw)
    return moe.moe_kv_cache(**f)


def append(L, d=None, kv=None, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, start=A, lens=A, table=A, cs=A, max_pos=100, rot=128, il=0,
             qn=A, kn=A, eps=1e-6, out=A, ws=A, n=256)
    a.update(kw)
    return L.moe_kv_append(ctypes.byref(d or desc()), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["start"],
                           a["lens"], a["table"], a["cs"], a["max_pos"], a["rot"], a["il"], a["qn"], a["kn"], a["eps"],
                           a["out"], ctypes.byref(kv or cache()), a["ws"], a["n"], None)


def attend(L, d=None, kv=None, **kw):
    d = d or desc()
    a = dict(q=A, qs=1024, start=A, lens=A, table=A, max_q=2, scale=0.1, causal=1, window=0, out=A, ws=A,
             n=max(256, L.moe_paged_attention_workspace_size(ctypes.byref(d), 2)))
    a.update(kw)
    return L.moe_paged_attention(ctypes.byref(d), a["q"], a["qs"], a["start"], a["lens"], a["table"],
                                 ctypes.byref(kv or cache()), a["max_q"], a["scale"], a["causal"], a["window"],
                                 a["out"], a["ws"], a["n"], None)


def gather(L, d=None, kv=None, **kw):
    a = dict(start=A, ostart=A, table=A, rows=5, k=A, v=B_, ws=A, n=256)
    a.update(kw)
    return L.moe_kv_gather(ctypes.byref(d or desc()), a["start"], a["ostart"], a["table"], ctypes.byref(kv or cache()),
                           a["rows"], a["k"], a["v"], a["ws"], a["n"], None)


@pytest.mark.parametrize("call", [append, attend, gather])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=7), BAD), (dict(D=64), UNS),
    (dict(D=0), BAD), (dict(page=48), UNS), (dict(page=256), UNS), (dict(page=0), BAD), (dict(n_pages=-1), BAD),
    (dict(max_pages=-1), BAD), (dict(B=0), BAD), (dict(Hq=2048), UNS), (dict(max_pages=1 << 26), UNS),
    (dict(n_pages=1 << 26), UNS), (dict(B=70000), UNS)])
def test_shapes_are_checked(L, call, kw, status):
    assert call(L, desc(**kw)) == status


@pytest.mark.parametrize("call", [append, attend, gather])
@pytest.mark.parametrize("field", ["k_codes", "v_codes", "k_scale", "v_scale"])
def test_cache_pointers_are_checked(L, call, field):
    assert call(L, kv=cache(**{field: None})) == BAD
    if "codes" in field:
        assert call(L, kv=cache(**{field: A + 8})) == BAD
    assert call(L, kv=cache(k_codes=A, v_codes=A)) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(out=None), BAD), (dict(k=A + 2), BAD),
    (dict(q=A + 8), BAD), (dict(start=None), BAD), (dict(lens=None), BAD), (dict(table=None), BAD), (dict(cs=None), BAD),
    (dict(qs=1016), BAD), (dict(qs=1028), BAD), (dict(ks=248), BAD), (dict(vs=260), BAD), (dict(rot=136), UNS),
    (dict(rot=24), UNS), (dict(rot=-16), BAD), (dict(max_pos=-1), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(ws=None), BAD), (dict(n=128), moe.MOE_ERR_WORKSPACE),
    (dict(q=None, out=None), BAD), (dict(kn=A + 4), BAD)])
def test_append_arguments_are_checked(L, kw, status):
    assert append(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(q=A + 4), BAD), (dict(qs=1000), BAD), (dict(start=None), BAD),
    (dict(lens=None), BAD), (dict(table=None), BAD), (dict(max_q=-1), BAD), (dict(max_q=0), BAD), (dict(max_q=1), BAD),
    (dict(max_q=4), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD),
    (dict(scale=float("nan")), BAD), (dict(window=-1), BAD), (dict(window=5, causal=0), BAD), (dict(ws=None), BAD),
    (dict(n=128), moe.MOE_ERR_WORKSPACE)])
def test_attention_arguments_are_checked(L, kw, status):
    assert attend(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(start=None), BAD), (dict(ostart=None), BAD), (dict(table=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(rows=-1), BAD), (dict(k=A + 8), BAD), (dict(ws=None), BAD), (dict(n=16), moe.MOE_ERR_WORKSPACE)])
def test_gather_arguments_are_checked(L, kw, status):
    assert gather(L, **kw) == status


def test_empty_calls_do_nothing(L):
    assert append(L, desc(T=0)) == moe.MOE_OK and attend(L, desc(T=0)) == moe.MOE_OK
    assert gather(L, rows=0) == moe.MOE_OK and gather(L, desc(B=0, T=0), rows=0) == moe.MOE_OK
    assert L.moe_rope_table(0, 128, 1e4, None, None) == moe.MOE_OK


def test_rope_table_arguments_are_checked(L):
    assert L.moe_rope_table(4, 128, 1e4, None, None) == BAD
    assert L.moe_rope_table(4, 130, 1e4, A, None) == UNS and L.moe_rope_table(4, 24, 1e4, A, None) == UNS
    assert L.moe_rope_table(-1, 128, 1e4, A, None) == BAD and L.moe_rope_table(4, 0, 1e4, A, None) == BAD
    assert L.moe_rope_table(4, 128, 0.0, A, None) == BAD and L.moe_rope_table(4, 128, float("inf"), A, None) == BAD


def test_workspace_size(L):
    size = lambda max_q=1, **kw: L.moe_paged_attention_workspace_size(ctypes.byref(desc(**kw)), max_q)
    assert size() >= L.moe_status_bytes()
    assert size(D=64) == 0 and size(max_q=-1) == 0
    assert size(n_pages=0, max_pages=0, page=16) == size()     # the pool does not matter


def test_binding_checks_types_and_shapes():
    import torch
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype)
    kv = moe.KVCache(z(2, 1, 16, 128), z(2, 1, 16, 128), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        kv._struct()
    with pytest.raises(ValueError, match="uint8"):
        moe.KVCache(z(2, 1, 16, 128, dtype=torch.int8), *kv[1:])._struct()
    with pytest.raises(ValueError, match="n_pages"):
        moe.KVCache(z(2, 16, 128), *kv[1:])._struct()
