"""The long conversations' operators together, as AttentionLayer calls them: positions, shared prefixes, weights, eviction; their
graphs, streams, waits that run out, and what lies around their outputs (GPU).  Tolerances as in test_gpu_attention_long."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import attention as oa  # noqa: E402
from oracle import attention_long as ol  # noqa: E402
from test_gpu_attention import D, Batch, bf16, env, f64  # noqa: E402,F401
from test_gpu_attention_long import Shared, check_shared, check_weights, denominators, i32  # noqa: E402

HQ, HKV, PAGE = 8, 2, 16
NAMES = ("k_codes", "v_codes", "k_scale", "v_scale")


def host_cache(cache):
    return {n: getattr(cache, n).cpu().numpy().copy() for n in NAMES}


def test_conversation(env):  # noqa: F811
    """Prompts of text and images, decoding, an eviction, and on with it: outputs and weights against the oracle at every step."""
    moe, torch = env
    rng = np.random.default_rng(0)
    layer = moe.AttentionLayer(64, HQ, HKV, page=PAGE, max_pos=4096, track_weights=True)
    axes = [f % 3 for f in range(64)]
    pool = [int(p) for p in rng.permutation(64)]
    table = np.array(pool[:24], np.int32).reshape(2, 12)
    lens, pos = [0, 0], [5, 900]
    for step, new in enumerate(([70, 33], [1, 1], [1, 0], [4, 3], "evict", [1, 1], [1, 1], [30, 2])):
        if new == "evict":
            keep, fresh = [40, 90], np.array(pool[24:36], np.int32).reshape(2, 6)
            host, weight = host_cache(layer.cache), layer.weight.cpu().numpy()
            new_len, kept = layer.evict(i32(lens), i32(table), i32(keep), i32(fresh), 2, 8)
            ref_len, ref_kept = ol.evict(host, weight, lens, table, keep, fresh, 2, 8)
            assert layer.status() == moe.MOE_OK and np.array_equal(kept.cpu().numpy(), ref_kept)
            assert new_len.tolist() == ref_len.tolist() == [40, min(90, lens[1])]
            assert np.array_equal(layer.weight.cpu().numpy(), weight)
            lens, table = ref_len.tolist(), fresh
            continue
        T, lens = sum(new), [a + n for a, n in zip(lens, new)]
        starts = np.cumsum([0] + new).astype(np.int32)
        p = np.concatenate([np.stack([at + np.arange(n) // 7, at + np.arange(n) % 7, at + np.arange(n)]) for at, n in zip(pos, new)], 1)
        pos = [a + n for a, n in zip(pos, new)]
        x = bf16(rng, T, HQ + 2 * HKV, D, mul=2.0)
        before, weight = host_cache(layer.cache), layer.weight.cpu().numpy()
        rows = layer.rotation(i32(p), axes)
        out = layer.forward(x.view(T, -1).cuda(), i32(starts), i32(lens), i32(table), max(new), rows=rows)
        assert layer.status() == moe.MOE_OK
        # the queries as moe_kv_append_at gives them, the cache as the layer left it
        other = moe.KVCache(*(torch.from_numpy(before[n].copy()).cuda() for n in NAMES))
        q, k, v = x.cuda().split([HQ, HKV, HKV], dim=1)
        rq = moe.moe_kv_append_at(q, k, v, other, i32(starts), i32(lens), i32(table), rows)
        assert all(torch.equal(a, b) for a, b in zip(other, layer.cache))
        turned = oa.norm_rotate(f64(x)[:, :HQ], np.arange(T), ol.rope_rows(p, axes, layer.cos_sin.cpu().numpy()), D, False)
        assert (np.abs(f64(rq) - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -18 * np.abs(turned).max(-1, keepdims=True)).all()
        host = host_cache(layer.cache)
        ref, spread, lse = ol.shared_attention(f64(rq), host, starts, lens, table, D ** -0.5)
        assert (np.abs(f64(out).reshape(T, HQ, D) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread).all(), step
        want, added, written = ol.weights(f64(rq), lse, host, starts, lens, table, D ** -0.5, weight)
        got = layer.weight.cpu().double().numpy()
        # 2^-9 of what was added for the scores, 2^-10 for the denominators' logarithms (the kernel has its own)
        assert (np.abs(got - want) <= (2.0 ** -9 + 2.0 ** -9) * added + 2.0 ** -22 * (want + added)).all()
        assert (got[~written] == weight[~written]).all()


def test_prefix_through_the_layer(env):  # noqa: F811
    """Sequences behind a prefix that another one stored, and the same sequences whole."""
    moe, torch = env
    rng = np.random.default_rng(1)
    layer = moe.AttentionLayer(64, HQ, HKV, page=PAGE, max_pos=512, track_weights=True)
    P, B = 6 * PAGE, 3
    ids = rng.permutation(64)
    head, own = ids[:6].reshape(1, 6).astype(np.int32), ids[6:6 + 4 * B].reshape(B, 4).astype(np.int32)
    layer.forward(bf16(rng, P, (HQ + 2 * HKV) * D).cuda(), i32([0, P]), i32([P]), i32(head), P)
    lens = [0] * B
    for new in ([9, 0, 20], [1, 1, 1], [1, 1, 1]):
        first, lens, T = list(lens), [a + n for a, n in zip(lens, new)], sum(new)
        starts = np.cumsum([0] + new)
        pos = np.concatenate([P + np.arange(a, a + n) for a, n in zip(first, new)])
        x = bf16(rng, T, (HQ + 2 * HKV) * D).cuda()
        before = host_cache(layer.cache)
        out = layer.forward(x, i32(starts), i32(lens), i32(own), max(new), rows=layer.rotation(i32(pos[None])),
                            prefix=(i32([0, T]), i32([P]), i32(head), T))
        assert layer.status() == moe.MOE_OK
        # the same tokens behind a table that has the prefix's pages before their own
        whole = moe.AttentionLayer(64, HQ, HKV, page=PAGE, max_pos=512)
        for n, t in zip(NAMES, whole.cache):
            t.copy_(torch.from_numpy(before[n]))
        joined = np.concatenate([np.repeat(head, B, 0), own], 1)
        ref = whole.forward(x, i32(starts), i32([P + n for n in lens]), i32(joined), max(new))
        assert all(torch.equal(a, b) for a, b in zip(whole.cache, layer.cache))
        q, k, v = x.view(T, -1, D).split([HQ, HKV, HKV], dim=1)
        rq = moe.moe_kv_append(q, k, v, whole.cache, i32(starts), i32([P + n for n in lens]), i32(joined), whole.cos_sin)
        exact, spread, _ = ol.shared_attention(f64(rq), host_cache(layer.cache), starts, [P + n for n in lens], joined, D ** -0.5)
        for o in (out, ref):
            assert (np.abs(f64(o).reshape(T, HQ, D) - exact) <= 2.0 ** -8 * np.abs(exact) + 2.0 ** -7 * spread).all()
    # what the prefix got is nobody's; the sequences' own weights add up to less than their rows
    w = layer.weight.double()
    for b in range(B):
        total = w[own[b].tolist()].sum((0, 2))
        assert (total < 4 * (lens[b])).all() and (total > 0).all()


def test_refused_calls_leave_the_cache_alone(env):  # noqa: F811
    moe, torch = env
    rng = np.random.default_rng(2)
    x, starts, lens, table = bf16(rng, 5, (HQ + 2 * HKV) * D).cuda(), i32([0, 2, 5]), i32([2, 3]), i32([[0, 1], [2, 3]])
    prefix = i32([0, 2, 5]), i32([9, 9]), i32([[4], [5]]), 3
    for kw, f in ((dict(), dict(prefix=prefix)), (dict(window=5, rot_dim=0), dict(prefix=prefix)),
                  (dict(rot_dim=0), dict(prefix=prefix[:3] + (0,))), (dict(rot_dim=0), dict(prefix=prefix[:3] + (2,))),
                  (dict(rot_dim=0), dict(prefix=(prefix[0][:2],) + prefix[1:])), (dict(rot_dim=0), dict(rows=torch.zeros(5, 128, device="cuda"))),
                  (dict(), dict(rows=torch.zeros(4, 128, device="cuda"))), (dict(rot_dim=64), dict(rows=torch.zeros(5, 128, device="cuda")))):
        layer = moe.AttentionLayer(8, HQ, HKV, page=PAGE, max_pos=64, **kw)
        for t in layer.cache:
            t.fill_(3)
        with pytest.raises((ValueError, moe.MoEError)):
            layer.forward(x, starts, lens, table, 3, **f)
        torch.cuda.synchronize()
        assert all((t == 3).all() for t in layer.cache)
    with pytest.raises(ValueError):
        layer.evict(lens, table, lens, table)
    with pytest.raises(ValueError):
        moe.AttentionLayer(8, HQ, HKV, rot_dim=0).rotation(i32([[0]]))


@pytest.mark.parametrize("new,heads", [(1, 8), (30, 16)])
def test_graphs_follow_lengths_and_tables(env, new, heads):  # noqa: F811
    """One captured step (rotation, append, shared attention, weights) and one captured eviction, replayed with other lengths, tables
    and numbers, beside eager calls; two graphs that share one workspace run one after another."""
    moe, torch = env
    rng = np.random.default_rng(new)
    layers = [moe.AttentionLayer(80, heads, HKV, page=PAGE, max_pos=512, track_weights=True) for _ in range(2)]
    P = 50
    ids = rng.permutation(80)
    head, own, fresh = ids[:4].reshape(1, 4), ids[4:44].reshape(2, 20), ids[44:64].reshape(2, 10)
    for layer in layers:
        layer.forward(bf16(np.random.default_rng(5), P, (heads + 2 * HKV) * D).cuda(), i32([0, P]), i32([P]), i32(head), P)
    T = 2 * new
    x, pos = torch.zeros(T, (heads + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda"), i32(np.zeros((1, T)))
    lens, table, keep, new_table = i32([new, new]), i32(own), i32([5, 7]), i32(fresh)
    p = (i32([0, T]), i32([P]), i32(head), T)

    def step(layer):
        return layer.forward(x, i32_start, lens, table, new, rows=layer.rotation(pos), prefix=p)

    i32_start = i32([0, new, T])
    step(layers[0])
    graphs = []
    for f in (lambda: step(layers[0]), lambda: layers[0].evict(lens, table, keep, new_table, 1, 2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for layer in layers:      # (the prompt and the step before the captures left theirs)
        layer.weight.zero_()
    for t, u in zip(layers[0].cache, layers[1].cache):
        u.copy_(t)
    at = [0, 0]
    for turn in range(4):
        at = [a + new for a in at]
        lens.copy_(i32(at))
        x.copy_(bf16(rng, *x.shape))
        pos.copy_(i32(np.concatenate([P + np.arange(a - new, a) for a in at])[None]))
        graphs[0][0].replay()
        eager = step(layers[1])
        assert torch.equal(graphs[0][1], eager)
        if turn == 2:
            graphs[1][0].replay()
            n, kept = layers[1].evict(lens, table, keep, new_table, 1, 2)
            assert torch.equal(graphs[1][1][0], n) and torch.equal(graphs[1][1][1], kept)
            at = n.tolist()
            old = table.clone()
            table.copy_(torch.cat([new_table, old[:, 10:]], 1))
        assert all(torch.equal(a, b) for a, b in zip((*layers[0].cache, layers[0].weight), (*layers[1].cache, layers[1].weight)))
    assert layers[0].status() == layers[1].status() == moe.MOE_OK


def test_streams(env):  # noqa: F811
    """Calls on a stream of their own, behind work that keeps it busy: inputs that are written there, outputs that are read there."""
    moe, torch = env
    rng = np.random.default_rng(3)
    for new in ([1] * 4, [40, 1, 30, 2]):
        b = Shared(rng, new, [30, 0, 200, 11], [150, 70], [2, 2], 2, 32)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        table, prefix = i32(np.ascontiguousarray(b.table)), b.prefix()
        q = bf16(rng, sum(new), 8, D).cuda()
        want, want_lse = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, table, max(new), prefix)
        want_w = moe.moe_kv_weights(q, want_lse, b.cache, b.d_start, b.d_len, table, max(new), out=torch.zeros_like(
            torch.empty(b.host["k_codes"].shape[:3], device="cuda")))
        late, w = torch.zeros_like(q), torch.zeros_like(want_w)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20000000)
            late.copy_(q)
        out, lse = moe.moe_paged_attention_shared(late, b.cache, b.d_start, b.d_len, table, max(new), prefix, stream=s)
        moe.moe_kv_weights(late, lse, b.cache, b.d_start, b.d_len, table, max(new), out=w, stream=s)
        with torch.cuda.stream(s):
            got = out.clone(), lse.clone(), w.clone()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], want_lse) and torch.equal(got[2], want_w)


@pytest.mark.parametrize("new,Hq", [(1, 8), (1, 32), (2, 16), (20, 8), (40, 16)])
def test_waits_that_run_out_end_the_kernels(env, new, Hq):  # noqa: F811
    """The copies are withheld: each call ends and reports it, and the next ones on the same context are correct.  (The limit stays far
    above what a copy takes: those in flight are waited for with it, too.)"""
    moe, torch = env
    rng = np.random.default_rng(7 + new + Hq)
    L = moe.lib()
    b = Shared(rng, [new] * 3, [700, 90, 2000], [600, 40], [1, 2], 2, 32)
    b.dev(env)
    b.d_start, b.d_len, b.d_table = i32(b.q_start), i32(b.kv_len), i32(np.ascontiguousarray(b.table))
    q = bf16(rng, 3 * new, Hq, D)
    lse = torch.zeros(3 * new, Hq, device="cuda")
    w = torch.zeros(b.host["k_codes"].shape[:3], device="cuda")
    try:
        assert L.moe_debug_set(4, 1) == moe.MOE_OK and L.moe_debug_set(1, 3000000) == moe.MOE_OK
        for call in (lambda ws: moe.moe_paged_attention_shared(q.cuda(), b.cache, b.d_start, b.d_len, b.d_table, new, b.prefix(), ws=ws),
                     lambda ws: moe.moe_kv_weights(q.cuda(), lse, b.cache, b.d_start, b.d_len, b.d_table, new, w, ws=ws)):
            ws = moe.moe_paged_attention_shared_workspace(3 * new, 3, Hq, 2, D, new, 2, b.max_p)
            call(ws)
            assert moe.moe_get_device_status(ws) == moe.MOE_ERR_TIMEOUT
    finally:
        L.moe_debug_set(4, 0)
        L.moe_debug_set(1, 0)
    check_shared(env, b, q)
    check_weights(env, b, q, denominators(b, q))


GUARD = 4096


def guarded(torch, shape, dtype, fill):
    n, g = int(np.prod(shape)), GUARD // torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n + 2 * g,), fill, dtype=dtype, device="cuda")
    return buf, buf[g:g + n].view(*shape), lambda: bool((buf[:g] == fill).all()) and bool((buf[g + n:] == fill).all())


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 0, 4], [50, 70, 9]])
def test_guards_around_every_output(env, new):  # noqa: F811
    """Each output, the workspace among them, is the middle of a larger buffer that stays as it was."""
    moe, torch = env
    rng = np.random.default_rng(sum(new))
    T, B = sum(new), 3
    b = Shared(rng, new, [30, 100, 300], [150], [B], 2, 16)
    b.dev(env)
    b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
    table, prefix, shape = i32(np.ascontiguousarray(b.table)), b.prefix(), b.host["k_codes"].shape[:3]
    q = bf16(rng, T, 8, D).cuda()
    p = moe.moe_kv_prefix(1, 0, T, None, None, None)
    import ctypes
    need = moe.lib().moe_paged_attention_shared_workspace_size(ctypes.byref(moe.moe_kv_desc(B, T, 8, 2, D, 16, 0, 0)), max(new), ctypes.byref(p))
    checks = []

    def out(shape, dtype, fill):
        _, t, intact = guarded(torch, shape, dtype, fill)
        checks.append(intact)
        return t

    ws = out((need,), torch.uint8, 0)
    o, lse = out((T, 8, D), torch.bfloat16, 7.0), out((T, 8), torch.float32, 7.0)
    moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, table, max(new), prefix, out=o, lse=lse, ws=ws)
    w = out(shape, torch.float32, 7.0)
    moe.moe_kv_weights(q, lse, b.cache, b.d_start, b.d_len, table, max(new), None, w, ws=ws)
    m = [20, 130, 17]
    used = [-(-x // 16) for x in m]
    free = Batch(rng, [0] * 6, b.total + m, 2, 16).fill(rng, upto=b.total + [0] * 3).dev(env)
    fresh = np.full((3, max(used)), -1, np.int32)
    for s in range(3):
        fresh[s, :used[s]] = free.table[3 + s, :used[s]]
    weight = out(free.host["k_codes"].shape[:3], torch.float32, 7.0)
    n, kept = out((3,), torch.int32, 7), out((3, 2, max(used) * 16), torch.int32, 7)
    cache = moe.KVCache(*(out(getattr(free.cache, x).shape, torch.uint8, 7) for x in NAMES))
    for t, x in zip(cache, NAMES):
        t.copy_(getattr(free.cache, x))
    moe.moe_kv_evict(cache, weight, i32(b.total), i32(np.ascontiguousarray(free.table[:3])), i32(m), i32(fresh), 1, 2, n, kept, ws=ws)
    rows = out((T, 128), torch.float32, 7.0)
    table128 = moe.moe_rope_table(64)
    moe.moe_rope_rows(i32(np.zeros((1, T))), [0] * 64, table128, rows, ws=ws)
    x = bf16(rng, T, 2, D).cuda()
    rq = out((T, 8, D), torch.bfloat16, 7.0)
    moe.moe_kv_append_at(q, x, x, b.cache, b.d_start, b.d_len, table, rows, q_out=rq, ws=ws)
    torch.cuda.synchronize()
    assert all(f() for f in checks) and moe.moe_get_device_status(ws) == moe.MOE_OK


def test_long_caches_pass_32_bits(env):  # noqa: F811
    """The last pages of a pool whose codes pass 2^32 bytes."""
    moe, torch = env
    Hkv, page = 8, 128
    n_pages = 40000            # 5.2 GB of keys, 5.2 GB of values, 0.16 GB of weights
    cache = moe.KVCache(*(torch.full((n_pages, Hkv, page, D), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2)),
                        *(torch.full((n_pages, Hkv), 127, dtype=torch.uint8, device="cuda") for _ in range(2)))
    w = torch.zeros(n_pages, Hkv, page, device="cuda")
    table, fresh = i32([[n_pages - 1, 3, n_pages - 2]]), i32([[n_pages - 3]])
    cache.k_codes[n_pages - 2, :, 5] = 0xB8           # one key against the query, the others for it
    q = torch.full((1, 16, D), 0.125, dtype=torch.bfloat16, device="cuda")
    lens, start = i32([300]), i32([0, 1])
    out, lse = moe.moe_paged_attention_shared(q, cache, start, lens, table, 1)
    moe.moe_kv_weights(q, lse, cache, start, lens, table, 1, w)
    z = np.full(300, 16.0)
    z[261] = -16.0
    p = np.exp(z * D ** -0.5)
    p /= p.sum()
    got = w[[n_pages - 1, 3, n_pages - 2]].transpose(0, 1).reshape(Hkv, -1)[:, :300].cpu().double().numpy()
    assert (np.abs(got - 2 * p) <= 2.0 ** -9 * 2 * p).all() and (out == 1).all()
    w[n_pages - 2, :, 7] = 5.0
    n, kept = moe.moe_kv_evict(cache, w, lens, table, i32([2]), fresh, 0, 1)
    assert kept[0, :, :2].tolist() == [[263, 299]] * Hkv and (w[n_pages - 3, :, 0] == 5.0).all()
    assert torch.equal(cache.k_codes[n_pages - 3, :, :2], cache.k_codes[n_pages - 2, :, [7, 43]])


def test_calls_at_once(env):  # noqa: F811
    """Shared attention and weights on two streams at the same time, workspaces of their own: what each gives alone.  And one stream's calls
    right behind one another in one workspace, each of whose passes overlap."""
    moe, torch = env
    rng = np.random.default_rng(4)
    work = []
    for new, own, prefix, readers, Hq in (([1] * 12, [50 * i for i in range(12)], [3000], [12], 16),
                                          ([5, 0, 3, 6], [900, 10, 0, 44], [500, 70], [2, 2], 16), ([90, 150], [30, 400], [700], [2], 8)):
        b = Shared(rng, new, own, prefix, readers, 2, 32)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        q = bf16(rng, sum(new), Hq, D).cuda()
        ws = moe.moe_paged_attention_shared_workspace(sum(new), len(new), Hq, 2, D, max(new), len(prefix), b.max_p)
        work.append((b, q, i32(np.ascontiguousarray(b.table)), b.prefix(), ws, torch.zeros(b.host["k_codes"].shape[:3], device="cuda")))

    def call(b, q, table, prefix, ws, w, stream=None):
        out, lse = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, table, max(b.new), prefix, ws=ws, stream=stream)
        return out, lse, moe.moe_kv_weights(q, lse, b.cache, b.d_start, b.d_len, table, max(b.new), None, w, ws=ws, stream=stream)

    want = [[t.clone() for t in call(*x)] for x in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for turn in range(20):
        got = [[call(*x, stream=s) for _ in range(3)][-1] for x, s in zip(work, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), turn
    assert all(moe.moe_get_device_status(x[4]) == moe.MOE_OK for x in work)
