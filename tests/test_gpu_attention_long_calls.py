"""Calls of the long conversations' operators that their documentation allows and that differ from the usual ones in the kind of their
arguments (GPU).  Tolerances as in test_gpu_attention_long."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import attention_long as ol  # noqa: E402
from test_gpu_attention import D, Batch, bf16, env, f64  # noqa: E402,F401
from test_gpu_attention_long import Shared, check_shared, check_weights, denominators, i32  # noqa: E402


def test_axes_as_arrays(env):  # noqa: F811
    """Lists, arrays and tensors of the same numbers turn the tokens alike."""
    moe, torch = env
    table, axes = moe.moe_rope_table(100, 128, 1e4), [f % 3 for f in range(64)]
    pos = i32(np.random.default_rng(0).integers(0, 100, (3, 9)))
    want = moe.moe_rope_rows(pos, axes, table)
    layer = moe.AttentionLayer(2, 8, 2, max_pos=100, rope_base=1e4)
    for kind in (np.array(axes), np.array(axes, np.int32), np.array(axes, np.uint8), tuple(axes), torch.tensor(axes)):
        assert torch.equal(moe.moe_rope_rows(pos, kind, table), want)
        assert torch.equal(layer.rotation(pos, kind), want)


def layer_inputs(torch, T=5):
    x = torch.randn(T, 12 * D, device="cuda").to(torch.bfloat16)
    return x, i32([0, 2, 5]), i32([2, 3]), i32([[0, 1], [2, 3]])


def test_refused_prefixes_leave_the_cache_alone(env):  # noqa: F811
    """Starts, lengths and tables of prefixes that begin anywhere, tables wider than any: refused before a token is stored."""
    moe, torch = env
    x, starts, lens, table = layer_inputs(torch)
    start, length, pages = i32([7, 0, 2, 5]), i32([7, 9, 9]), i32([[0], [4], [5]])
    good = start[1:].clone(), length[1:].clone(), pages[1:].clone()
    wide = torch.zeros(2, 1 << 24, dtype=torch.int32, device="cuda")   # 2^31 tokens
    out = torch.zeros(5 * 8 * D + 8, dtype=torch.bfloat16, device="cuda")
    for bad in ((start[1:], good[1], good[2], 3), (good[0], length[1:], good[2], 3), (good[0], good[1], pages[1:], 3),
                (good[0], good[1], wide, 3), None):
        layer = moe.AttentionLayer(8, 8, 2, page=128, rot_dim=0)
        for t in layer.cache:
            t.fill_(3)
        kw = dict(prefix=bad) if bad else dict(out=out[1:1 + 5 * 8 * D].view(5, -1))
        with pytest.raises((ValueError, moe.MoEError)):
            layer.forward(x, starts, lens, table, 3, **kw)
        torch.cuda.synchronize()
        assert all((t == 3).all() for t in layer.cache)
        layer.forward(x, starts, lens, table, 3, prefix=(*good, 3))
        assert layer.status() == moe.MOE_OK


@pytest.mark.parametrize("new", [[2, 3], [200, 300], [0, 40]])
def test_prefixes_without_tokens_or_columns(env, new):  # noqa: F811
    """All prefixes empty, their table without a column: what the sequences give alone."""
    moe, torch = env
    T = sum(new)
    x, starts, lens = torch.randn(T, 12 * D, device="cuda").to(torch.bfloat16), i32([0, new[0], T]), i32(new)
    table = i32([list(range(20)), list(range(20, 40))])
    layer = moe.AttentionLayer(40, 8, 2, page=16, rot_dim=0, track_weights=True)
    want = layer.forward(x, starts, lens, table, max(new)).clone()
    weight = layer.weight.clone()
    got = layer.forward(x, starts, lens, table, max(new), prefix=(starts, i32([0, 0]), torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                                                                   max(new)))
    assert layer.status() == moe.MOE_OK
    # one rounding of each, and the weights' 2^-7 of the values that a row may weigh
    assert (got - want).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -7) * x.abs().max()
    assert (layer.weight - weight).abs().max() <= 2.0 ** -8 * T * 4


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 5])
def test_counts_of_more_than_32_bits(env, n):  # noqa: F811
    """A window, a sink or recent tokens beyond any length are all tokens, not the number's low bits."""
    moe, torch = env
    cache = moe.KVCache(*(torch.randint(0, 100, (4, 2, 16, D), dtype=torch.uint8, device="cuda") for _ in range(2)),
                        *(torch.full((4, 2), 127, dtype=torch.uint8, device="cuda") for _ in range(2)))
    q = torch.randn(1, 8, D, device="cuda").to(torch.bfloat16)
    w = torch.rand(4, 2, 16, device="cuda")
    lens, start, table, fresh = i32([20]), i32([0, 1]), i32([[0, 1]]), i32([[2]])
    assert torch.equal(moe.moe_paged_attention(q, cache, start, lens, table, 1, window=n), moe.moe_paged_attention(q, cache, start, lens, table, 1))
    out, lse = moe.moe_paged_attention_shared(q, cache, start, lens, table, 1)
    assert torch.equal(moe.moe_paged_attention_shared(q, cache, start, lens, table, 1, window=n)[0], out)
    assert torch.equal(moe.moe_kv_weights(q, lse, cache, start, lens, table, 1, w, w.clone(), window=n),
                       moe.moe_kv_weights(q, lse, cache, start, lens, table, 1, w, w.clone()))
    for kw in (dict(sink=n), dict(recent=n)):
        _, kept = moe.moe_kv_evict(cache, w, lens, table, i32([7]), fresh, **kw)
        assert kept[0, :, :7].tolist() == [list(range(7))] * 2      # all tokens alike: the first ones
    for call in (lambda: moe.moe_paged_attention(q, cache, start, lens, table, 1, window=-n),
                 lambda: moe.moe_kv_evict(cache, w, lens, table, i32([7]), fresh, recent=-n)):
        with pytest.raises(moe.MoEError):
            call()


@pytest.mark.parametrize("new,Hq", [(1, 2), (1, 8), (3, 8), (2, 24), (20, 8), (70, 16)])
@pytest.mark.parametrize("fresh", [False, True])
def test_weights_that_overflow(env, new, Hq, fresh):  # noqa: F811
    """A denominator so far below a row's scores that all its weights pass fp32 adds nothing, like one that is not there: the same bits,
    whatever max_q says."""
    moe, torch = env
    rng = np.random.default_rng(new + Hq)
    b = Batch(rng, [new, new], [300, 40], 2, 32).fill(rng).dev(env)
    q = bf16(rng, 2 * new, Hq, D).cuda()
    # scores lie within +-88 of zero by far, so e^(score + 200) is above fp32 and e^(score - 4) is not
    lse = torch.full((2 * new, Hq), 4.0, device="cuda")
    none = lse.clone()
    for t, h in ((0, 0), (2 * new - 1, Hq - 1)):
        lse[t, h], none[t, h] = -200.0, -float("inf")
    before = torch.rand(b.host["k_codes"].shape[:3], device="cuda")
    for max_q in (new, 2 * new):
        got, want = (moe.moe_kv_weights(q, x, b.cache, b.d_start, b.d_len, b.d_table, max_q, None if fresh else before, before.clone())
                     for x in (lse, none))
        assert torch.isfinite(got).all() and torch.equal(got, want)


@pytest.mark.parametrize("new,ctx", [([1] * 4, [0, 30, 129, 800]), ([1] * 40, [100 * i for i in range(40)]), ([7] * 10, [0, 5, 20, 9, 0, 1, 30, 2, 3, 4]),
                                     ([3, 1, 0, 6], [0, 60, 5, 300]), ([5] * 6, [700] * 6), ([100, 30], [0, 150]), ([300, 2], [900, 4000])])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (32, 4), (5, 5), (24, 2)])
def test_denominators_change_no_output(env, new, ctx, Hq, Hkv):  # noqa: F811
    """Without prefixes the rows are those of moe_paged_attention, bit for bit, in short tables too."""
    moe, torch = env
    rng = np.random.default_rng(len(new))
    for page in (16, 128):
        b = Batch(rng, new, ctx, Hkv, page).fill(rng, 1.0, 2.0).dev(env)
        q = bf16(rng, sum(new), Hq, D, mul=2.0).cuda()
        for kw in (dict(), dict(window=40), dict(causal=False)):
            want = moe.moe_paged_attention(q, b.cache, b.d_start, b.d_len, b.d_table, max(new), **kw)
            out, _ = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, b.d_table, max(new), **kw)
            assert torch.equal(out, want), kw


@pytest.mark.parametrize("new", [[1, 1, 1], [7, 5, 6], [90, 3, 200]])
def test_tracked_weights_change_no_output(env, new):  # noqa: F811
    moe, torch = env
    T = sum(new)
    layers = [moe.AttentionLayer(60, 32, 4, page=16, max_pos=512, track_weights=track) for track in (False, True)]
    starts, table = i32(np.cumsum([0] + new)), i32(np.random.default_rng(0).permutation(60).reshape(3, 20))
    for step in range(1, 3):
        x = torch.randn(T, 40 * D, device="cuda").to(torch.bfloat16)
        outs = [layer.forward(x, starts, i32([n * step for n in new]) if max(new) < 100 else i32(new), table, max(new)) for layer in layers]
        assert torch.equal(*outs)


@pytest.mark.parametrize("new,readers", [([1] * 12 + [150], [13]), ([1] * 3 + [150], [4]), ([1] * 12 + [150], [5, 8]), ([150, 0] + [1] * 9, [11]),
                                         ([40, 90, 0, 1, 1, 120], [2, 4])])
def test_long_and_short_sequences_behind_one_prefix(env, new, readers):  # noqa: F811
    """Both sides of the border between one pass and two, tight tables and tables much wider than their sequences."""
    moe, torch = env
    rng = np.random.default_rng(len(new))
    for wide in (0, 3000):
        b = Shared(rng, new, [int(x) for x in rng.integers(0, 200, len(new))], [700, 90][:len(readers)], readers, 2, 32)
        if wide:
            b.table, b.p_table = (np.concatenate([np.maximum(t, -1), np.full((len(t), wide), -1, np.int32)], 1) for t in (b.table, b.p_table))
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        for Hq in (8, 16):
            check_shared(env, b, bf16(rng, sum(new), Hq, D, mul=2.0))


@pytest.mark.parametrize("new", [[1] * 4, [30, 7], [200, 90]])
def test_tables_much_wider_than_their_sequences(env, new):  # noqa: F811
    """A server's tables are as wide as its longest context, whatever is in them."""
    moe, torch = env
    rng = np.random.default_rng(len(new))
    B = len(new)
    for wide in (0, 5, 2048):
        rng = np.random.default_rng(1)
        b = Shared(rng, new, [20, 0, 300, 11][:B], [100, 9], [1, B - 1], 2, 16)
        if wide:
            b.table, b.p_table = (np.concatenate([t, np.full((len(t), wide), -1, np.int32)], 1) for t in (b.table, b.p_table))
        b.dev(env)
        b.d_start, b.d_len, b.d_table = i32(b.q_start), i32(b.kv_len), i32(np.ascontiguousarray(b.table))
        q = bf16(rng, sum(new), 8, D, mul=2.0)
        check_shared(env, b, q)
        check_shared(env, b, q, prefix=False)
        check_weights(env, b, q, denominators(b, q))


@pytest.mark.parametrize("new,readers", [([1] * 4, [3, 1]), ([5, 0, 2, 3], [2, 2]), ([70, 30, 9], [1, 2])])
def test_weights_of_the_prefixes_tokens(env, new, readers):  # noqa: F811
    """What the readers give a prefix's tokens: the prefixes as the sequences, without a mask, from zero on.  With the sequences' own
    weights all rows add up."""
    moe, torch = env
    rng = np.random.default_rng(len(new))
    b = Shared(rng, new, [30, 0, 100, 4][:len(new)], [300, 77], readers, 2, 32)
    b.dev(env)
    b.d_start, b.d_len, b.d_table = i32(b.q_start), i32(b.kv_len), i32(np.ascontiguousarray(b.table))
    q, shape, ws = bf16(rng, sum(new), 8, D, mul=2.0).cuda(), b.host["k_codes"].shape[:3], moe.moe_kv_workspace()
    _, lse = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, b.d_table, max(new), b.prefix())
    start, length, table, most = b.prefix()
    own, of_prefix = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    moe.moe_kv_weights(q, lse, b.cache, b.d_start, b.d_len, b.d_table, max(new), own, ws=ws)
    moe.moe_kv_weights(q, lse, b.cache, start, length, table, most, None, of_prefix, causal=False, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    want, added, written = ol.weights(f64(q), lse.cpu().double().numpy(), b.host, b.p_start, b.p_len, b.p_table, D ** -0.5,
                                      np.zeros(shape), True, False)
    got = of_prefix.cpu().double().numpy()
    assert (np.abs(got - want) <= 2.0 ** -9 * added + 2.0 ** -22 * added).all() and (got[~written] == 0).all()
    total = (own + of_prefix).double().sum((0, 2))
    assert ((total - 4 * sum(new)).abs() <= 2.0 ** -9 * 4 * sum(new)).all()


@pytest.mark.parametrize("new", [[1] * 4, [30, 7], [200, 90]])
def test_denominators_are_optional(env, new):  # noqa: F811
    """lse = NULL at the C entry point: the same rows."""
    import ctypes
    moe, torch = env
    rng = np.random.default_rng(3)
    B, T = len(new), sum(new)
    b = Shared(rng, new, [20, 0, 300, 11][:B], [400, 9], [1, B - 1], 2, 16)
    b.dev(env)
    b.d_start, b.d_len, table = i32(b.q_start), i32(b.kv_len), i32(np.ascontiguousarray(b.table))
    q = bf16(rng, T, 8, D, mul=2.0).cuda()
    for prefix in (b.prefix(), None):
        want, _ = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, table, max(new), prefix)
        n, n_pages = table.shape[1], b.cache.k_codes.shape[0]
        d, kv = moe.moe_kv_desc(B, T, 8, 2, D, 16, n_pages, n), b.cache._struct()
        p = None if prefix is None else ctypes.byref(moe.moe_kv_prefix(2, prefix[2].shape[1], prefix[3], *(t.data_ptr() for t in prefix[:3])))
        need = moe.lib().moe_paged_attention_shared_workspace_size(ctypes.byref(d), max(new), p)
        ws, out = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
        assert moe.lib().moe_paged_attention_shared(ctypes.byref(d), q.data_ptr(), 8 * D, b.d_start.data_ptr(), b.d_len.data_ptr(), table.data_ptr(),
                                                    ctypes.byref(kv), max(new), D ** -0.5, 1, 0, p, out.data_ptr(), None, ws.data_ptr(), need,
                                                    torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
        assert torch.equal(out, want) and moe.moe_get_device_status(ws) == moe.MOE_OK


def test_tables_of_one_dimension_are_refused(env):  # noqa: F811
    moe, torch = env
    x, starts, lens, table = layer_inputs(torch)
    layer = moe.AttentionLayer(8, 8, 2, page=16)
    with pytest.raises(ValueError, match="page_table"):
        layer.forward(x, starts, lens, table[:, 0].contiguous(), 3)
