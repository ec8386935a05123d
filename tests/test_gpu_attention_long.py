"""Positions on several axes, shared prefixes, accumulated weights and eviction against the float64 oracle (GPU).

Tolerances.  Output of moe_paged_attention_shared: as moe_paged_attention's, 2^-8 |out| for its one rounding and
2^-7 sum_j p_j |v_j| for the weights, whose sums pass between its two passes in fp32.  Scores: fp32 sums of 128 products
(2^-12 at a score's size of up to 20) of queries in two E4M3 halves, exact but for elements below 2^-9 of a row's largest, which are off by
at most 2^-17 of that one: less than 2^-11 together, for 128 elements of keys and queries of a few units and a scale of 128^-1/2.
So a denominator's logarithm is within 2^-10, and a weight exp(score - lse) with lse given within 2^-9 of itself; the sums of
positive fp32 numbers add less than 2^-16.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import attention as oa  # noqa: E402
from oracle import attention_long as ol  # noqa: E402
from test_gpu_attention import D, Batch, bf16, env, f64, same_cache  # noqa: E402,F401


def i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ positions
@pytest.mark.parametrize("n_axes,rot", [(1, 128), (3, 128), (4, 64), (2, 32), (8, 16), (3, 96)])
@pytest.mark.parametrize("T", [1, 2, 37, 1000])
def test_rope_rows(env, n_axes, rot, T):
    moe, torch = env
    rng = np.random.default_rng(n_axes * 100 + T)
    table = moe.moe_rope_table(500, rot, 1e4)
    pos = rng.integers(0, 500, (n_axes, T + 3)).astype(np.int32)
    d_pos = i32(pos)[:, 1:T + 1]        # the axes' tokens in rows further apart, none of them aligned
    for axes in ([f % n_axes for f in range(rot // 2)], [f * n_axes // (rot // 2) for f in range(rot // 2)], [n_axes - 1] * (rot // 2)):
        ws = moe.moe_kv_workspace()
        rows = moe.moe_rope_rows(d_pos, axes, table, ws=ws)
        assert np.array_equal(rows.cpu().numpy(), ol.rope_rows(pos[:, 1:T + 1], axes, table.cpu().numpy()).astype(np.float32))
        assert moe.moe_get_device_status(ws) == moe.MOE_OK


def test_rope_rows_of_one_row_for_all_axes(env):
    """Text alone: one row of positions, expanded."""
    moe, torch = env
    table, pos = moe.moe_rope_table(500, 64), i32([[7, 8, 9, 400]])
    rows = moe.moe_rope_rows(pos.expand(3, -1), [f % 3 for f in range(32)], table)
    assert torch.equal(rows, table[pos[0].long()])


def test_rope_rows_outside_the_table(env):
    moe, torch = env
    table, axes = moe.moe_rope_table(64, 32), [0] * 8 + [1] * 8
    pos = i32([[3, 64, 5, -1], [63, 4, 1 << 30, 0]])
    ws = moe.moe_kv_workspace()
    rows = moe.moe_rope_rows(pos, axes, table, ws=ws).cpu().numpy().reshape(4, 2, 16)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    bad = np.array([[False, False], [True, False], [False, True], [True, False]])
    assert np.array_equal(np.isnan(rows), np.broadcast_to(np.repeat(bad, 8, 1)[:, None], rows.shape))
    assert moe.moe_rope_rows(pos[:, :0], axes, table).shape == (0, 32)


RAGGED = dict(new=[3, 0, 1, 40, 17], ctx=[0, 9, 31, 5, 64])


@pytest.mark.parametrize("Hq,Hkv,rot,interleaved,norm", [(8, 2, 128, False, True), (3, 1, 64, True, False), (20, 4, 96, False, False),
                                                         (12, 12, 32, True, True), (5, 5, 0, False, True)])
def test_append_at_the_slots_is_append(env, Hq, Hkv, rot, interleaved, norm):
    """The same bits when every token's position is its place."""
    moe, torch = env
    rng = np.random.default_rng(Hq)
    T = sum(RAGGED["new"])
    q, k, v = bf16(rng, T, Hq + 2 * Hkv, D, mul=3.0).cuda().split([Hq, Hkv, Hkv], dim=1)
    w = bf16(rng, D).cuda() if norm else None
    table = moe.moe_rope_table(128, rot, 1e4) if rot else None
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(RAGGED["new"], RAGGED["ctx"])])
    rows = moe.moe_rope_rows(i32(pos[None]), [0] * (rot // 2), table) if rot else torch.empty(T, 0, device="cuda")
    got = []
    for at in (False, True):
        r = np.random.default_rng(3)
        b = Batch(r, **RAGGED, Hkv=Hkv, page=32).fill(r, upto=RAGGED["ctx"]).dev(env)
        args = (q, k, v, b.cache, b.d_start, b.d_len, b.d_table)
        kw = dict(interleaved=interleaved, q_norm_weight=w, k_norm_weight=w, ws=b.ws)
        out = moe.moe_kv_append_at(*args, rows, **kw) if at else moe.moe_kv_append(*args, table, **kw)
        assert moe.moe_get_device_status(b.ws) == moe.MOE_OK
        got.append((out, *b.cache))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*got))


@pytest.mark.parametrize("page", [16, 128])
def test_append_at(env, page):
    """Positions on three axes, far from the slots and beyond any length."""
    moe, torch = env
    rng = np.random.default_rng(page)
    Hq, Hkv, rot = 6, 2, 128
    b = Batch(rng, **RAGGED, Hkv=Hkv, page=page).fill(rng, upto=RAGGED["ctx"]).dev(env)
    T = sum(b.new)
    x = bf16(rng, T, Hq + 2 * Hkv, D, mul=3.0)
    table, axes = moe.moe_rope_table(20000, rot, 1e6), [(0, 1, 2)[f % 3] for f in range(64)]
    pos = rng.integers(0, 20000, (3, T)).astype(np.int32)
    rows = moe.moe_rope_rows(i32(pos), axes, table)
    q, k, v = x.cuda().split([Hq, Hkv, Hkv], dim=1)
    out = moe.moe_kv_append_at(q, k, v, b.cache, b.d_start, b.d_len, b.d_table, rows, ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == moe.MOE_OK
    ref_rows = ol.rope_rows(pos, axes, table.cpu().numpy())
    turned = oa.norm_rotate(f64(x), np.arange(T), ref_rows, rot, False)
    size = np.abs(turned[:, :Hq]).max(-1, keepdims=True)
    assert (np.abs(f64(out) - turned[:, :Hq]) <= 2.0 ** -8 * np.abs(turned[:, :Hq]) + 2.0 ** -18 * size).all()
    oa.append(turned[:, Hq:Hq + Hkv], f64(x)[:, Hq + Hkv:], b.host, b.q_start, b.kv_len, b.table)
    for name, codes, scale in same_cache(b):
        for s in range(len(b.new)):
            for i in range(b.ctx[s], b.total[s]):
                p, at = b.table[s, i // page], i % page
                assert (scale[p] == b.host[name + "_scale"][p]).all()
                # within one rounding of the unrounded value
                y = turned[b.q_start[s] + i - b.ctx[s], Hq:Hq + Hkv] if name == "k" else f64(x)[b.q_start[s] + i - b.ctx[s], Hq + Hkv:]
                unit = 2.0 ** (scale[p].astype(int) - 127)[:, None]
                off = np.abs(oa.values(codes[p, :, at], 0) * unit - y)
                assert (off <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * unit) + 2.0 ** -18 * np.abs(y).max(-1, keepdims=True)).all()


# ------------------------------------------------------------------------------------------------ shared prefixes
class Shared(Batch):
    """A batch whose pool also holds prefixes: `readers` cuts the sequences into their groups."""

    def __init__(self, rng, new, ctx, prefix, readers, Hkv, page):
        super().__init__(rng, list(new) + [0] * len(prefix), list(ctx) + list(prefix), Hkv, page)
        self.fill(rng, 1.0, 2.0)
        B = len(new)
        self.new, self.ctx, self.total = list(new), list(ctx), self.total[:B]
        self.p_table, self.table = self.table[B:], self.table[:B]
        self.p_len = np.array(prefix, np.int32)
        self.kv_len, self.q_start = self.kv_len[:B], self.q_start[:B + 1]
        cuts = np.concatenate([[0], np.cumsum(readers)])
        assert cuts[-1] == B
        self.p_start = self.q_start[cuts].astype(np.int32)
        self.max_p = int(np.diff(self.p_start).max())

    def prefix(self):
        return i32(self.p_start), i32(self.p_len), i32(np.ascontiguousarray(self.p_table)), self.max_p


def check_shared(env, b, q, prefix=True, status=0, window=0, causal=True, **kw):
    moe, torch = env
    p = b.prefix() if prefix else None
    ws = moe.moe_paged_attention_shared_workspace(q.shape[0], len(b.new), q.shape[1], b.Hkv, D, max(b.new), len(b.p_len) if prefix else 0,
                                                  b.max_p if prefix else 0)
    out, lse = moe.moe_paged_attention_shared(q.cuda(), b.cache, b.d_start, b.d_len, i32(np.ascontiguousarray(b.table)), max(b.new), p, ws=ws,
                                              window=window, causal=causal, **kw)
    assert moe.moe_get_device_status(ws) == status
    ref, spread, ref_lse = ol.shared_attention(f64(q), b.host, b.q_start, b.kv_len, b.table, D ** -0.5,
                                               (b.p_start, b.p_len, b.p_table) if prefix else None, causal, window)
    got, got_lse = f64(out), lse.cpu().double().numpy()
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and (np.abs(got_lse[~empty] - ref_lse[~empty]) <= 2.0 ** -10).all()
    return out, lse


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 2), (4, 4), (10, 2), (7, 1), (24, 2)])
@pytest.mark.parametrize("new,ctx,prefix,readers", [
    ([1], [0], [1], [1]),                                                        # the first token behind a token
    ([1] * 5, [0, 3, 16, 100, 140], [333], [5]),                                 # decoding, one prefix
    ([1] * 6, [0, 3, 16, 700, 140, 2], [128, 0, 1, 700], [2, 3, 0, 1]),          # some without tokens, some without readers
    ([2, 0, 5, 1], [0, 9, 100, 64], [50, 300], [2, 2]),                          # a sequence that brings nothing
    ([40, 3, 130], [0, 200, 31], [129, 600], [1, 2]),                            # chunks
])
def test_shared(env, Hq, Hkv, new, ctx, prefix, readers):
    moe, torch = env
    rng = np.random.default_rng(Hq + len(new))
    for page in (16, 64):
        b = Shared(rng, new, ctx, prefix, readers, Hkv, page)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        check_shared(env, b, bf16(rng, sum(new), Hq, D, mul=2.0))


@pytest.mark.parametrize("page", [32, 128])
def test_shared_long_prefix(env, page):
    """Prefixes that many blocks share out, with many readers (the prefix pass has full tiles) and with few."""
    rng = np.random.default_rng(page)
    for new, ctx, prefix, readers in (([1] * 40, [5 * i for i in range(40)], [3000], [40]), ([1] * 3, [10, 0, 300], [5000, 2001], [1, 2])):
        b = Shared(rng, new, ctx, prefix, readers, 2, page)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        check_shared(env, b, bf16(rng, sum(new), 16, D, mul=1.5))


@pytest.mark.parametrize("new,ctx", [([1] * 4, [0, 30, 129, 800]), ([3, 1, 0, 6], [0, 60, 5, 300]), ([100, 30], [0, 150]), ([260], [500])])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0)])
def test_denominators_without_prefix(env, new, ctx, causal, window):
    rng = np.random.default_rng(len(new))
    b = Batch(rng, new, ctx, 2, 32).fill(rng, 1.0, 2.0).dev(env)
    check_shared(env, b, bf16(rng, sum(new), 8, D, mul=2.0), prefix=False, causal=causal, window=window)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 40, 3]])
def test_rows_that_see_nothing(env, new):
    """Own tokens that are none, before position 0, on pages without values: the prefix alone, or nothing at all."""
    rng = np.random.default_rng(5)
    for prefix in ([0], [77]):
        b = Shared(rng, new, [0, 10, 200], prefix, [3], 2, 16)
        b.kv_len = np.array([0, max(0, new[1] - 25), b.kv_len[2]], np.int32)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        out, lse = check_shared(env, b, bf16(rng, sum(new), 6, D))
        if not prefix[0]:
            assert (out[:new[0]] == 0).all() and (lse[:new[0]] == -np.inf).all()


def test_prefix_and_own_far_apart(env):
    """One of the two parts takes all of the softmax, and value scales of the two differ by many powers of two."""
    moe, torch = env
    for new in ([1] * 3, [70] * 3):
        rng = np.random.default_rng(31)
        b = Shared(rng, new, [40, 0, 300], [200], [3], 1, 16)
        b.host["v_scale"][b.p_table[0, :13]] = 100
        for j, s in enumerate((90, 127, 140)):
            b.host["v_scale"][b.table[j][b.table[j] >= 0]] = s
        b.host["k_scale"][b.table[0][b.table[0] >= 0]] += 3
        b.host["k_scale"][b.table[1][b.table[1] >= 0]] -= 20
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        check_shared(env, b, bf16(rng, sum(new), 8, D, mul=2.0))


def test_shared_contradictions_set_the_status(env):
    moe, torch = env
    rng = np.random.default_rng(7)
    for new in ([1] * 4, [30] * 4):
        for fault in ("page", "length", "start", "end"):
            b = Shared(rng, new, [20, 0, 3, 40], [100, 60], [2, 2], 2, 16)
            b.dev(env)
            b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
            start, length, table, most = b.prefix()
            if fault == "page":
                table[0, 3] = 1 << 20
            elif fault == "length":
                length[1] = 1 << 20
            elif fault == "start":
                start[1] = -3
            else:
                start[2] = start[2] - 1
            ws = moe.moe_paged_attention_shared_workspace(sum(new), 4, 8, 2, D, max(new), 2, sum(new))
            moe.moe_paged_attention_shared(bf16(rng, sum(new), 8, D).cuda(), b.cache, b.d_start, b.d_len, i32(np.ascontiguousarray(b.table)),
                                           max(new), (start, length, table, sum(new)), ws=ws)
            assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK, fault


# ------------------------------------------------------------------------------------------------ weights
def check_weights(env, b, q, lse, fresh=False, causal=True, window=0, in_place=False, status=0, max_q=None):
    moe, torch = env
    rng = np.random.default_rng(1)
    before = rng.exponential(size=(b.host["k_codes"].shape[:3])).astype(np.float32)
    w = torch.from_numpy(before).cuda()
    out = w if in_place else torch.full_like(w, -7.0)
    ws = moe.moe_kv_workspace()
    got = moe.moe_kv_weights(q.cuda(), lse, b.cache, b.d_start, b.d_len, b.d_table, max(b.new) if max_q is None else max_q,
                             None if fresh else w, out, causal=causal, window=window, ws=ws)
    assert got is out and moe.moe_get_device_status(ws) == status
    ref, added, written = ol.weights(f64(q), lse.cpu().double().numpy(), b.host, b.q_start, b.kv_len, b.table, D ** -0.5, before,
                                     fresh, causal, window)
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - ref) <= 2.0 ** -9 * added + 2.0 ** -22 * (ref + added)) & written
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    assert (got[~written] == (before[~written] if in_place else -7.0)).all()
    return out


def denominators(b, q, causal=True, window=0):
    import torch
    return torch.from_numpy(ol.shared_attention(f64(q), b.host, b.q_start, b.kv_len, b.table, D ** -0.5, None, causal, window)[2]).float().cuda()


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 2), (4, 4), (10, 2), (7, 1), (24, 2)])
@pytest.mark.parametrize("new,ctx", [([1] * 9, [0, 1, 15, 16, 127, 128, 129, 300, 700]), ([2, 0, 5, 3, 1], [0, 40, 130, 255, 64]),
                                     ([33, 0, 150, 1], [100, 7, 0, 300]), ([70], [700])])
def test_weights(env, Hq, Hkv, new, ctx):
    rng = np.random.default_rng(Hq + len(new))
    for page, causal, window, fresh in ((16, True, 0, False), (64, True, 50, False), (128, False, 0, True), (32, True, 1, True)):
        b = Batch(rng, new, ctx, Hkv, page).fill(rng).dev(env)
        q = bf16(rng, sum(new), Hq, D, mul=2.0)
        lse = denominators(b, q, causal, window)
        out = check_weights(env, b, q, lse, fresh, causal, window)
        again = check_weights(env, b, q, lse, fresh, causal, window, in_place=True)
        seen = out != -7.0
        assert bool((out[seen] == again[seen]).all())   # the same bits, in place or not
        # whatever the kernel that max_q chooses
        check_weights(env, b, q, lse, fresh, causal, window, max_q=sum(new))


def test_weights_long(env):
    """More tiles than blocks, several groups of tiles a block, and runs that begin inside a sequence."""
    rng = np.random.default_rng(3)
    for new, ctx, Hq, Hkv in (([1, 1], [20000, 5000], 8, 4), ([12, 1], [6000, 3000], 16, 2)):
        b = Batch(rng, new, ctx, Hkv, 128).fill(rng).dev(env)
        q = bf16(rng, sum(new), Hq, D, mul=2.0)
        check_weights(env, b, q, denominators(b, q))


@pytest.mark.parametrize("scale", [D ** -0.5, 1e-10])
def test_weights_chunks_of_the_kernel_for_few_rows(env, scale):
    """More rows than max_q says -- it has to cover the tokens in the mean only -- and a scale so small that the other kernel leaves them
    to this one."""
    moe, torch = env
    rng = np.random.default_rng(6)
    for new, ctx, Hq, Hkv in (([20, 0, 0, 0], [300, 5, 0, 70], 8, 4), ([30, 1, 0, 0, 0, 1, 0, 0], [900, 5, 0, 70, 1, 0, 2, 300], 4, 2)):
        b = Batch(rng, new, ctx, Hkv, 32).fill(rng).dev(env)
        q = bf16(rng, sum(new), Hq, D, mul=2.0)
        lse = torch.from_numpy(ol.shared_attention(f64(q), b.host, b.q_start, b.kv_len, b.table, scale)[2]).float().cuda()
        before = rng.exponential(size=b.host["k_codes"].shape[:3]).astype(np.float32)
        for max_q in (-(-sum(new) // len(new)), max(new)):
            for window in (0, 50):
                w, ws = torch.from_numpy(before.copy()).cuda(), moe.moe_kv_workspace()
                moe.moe_kv_weights(q.cuda(), lse, b.cache, b.d_start, b.d_len, b.d_table, max_q, w, scale=scale, window=window, ws=ws)
                assert moe.moe_get_device_status(ws) == moe.MOE_OK
                ref, added, written = ol.weights(f64(q), lse.cpu().double().numpy(), b.host, b.q_start, b.kv_len, b.table, scale, before,
                                                 False, True, window)
                got = w.cpu().double().numpy()
                assert (np.abs(got - ref) <= 2.0 ** -9 * added + 2.0 ** -22 * (ref + added)).all()


def test_weights_sum_to_the_rows(env):
    """With the attention's own denominators, all weights of a head add up to its rows."""
    moe, torch = env
    rng = np.random.default_rng(4)
    for new, ctx in (([1] * 4, [0, 200, 1000, 77]), ([50, 9], [300, 0])):
        b = Batch(rng, new, ctx, 2, 16).fill(rng).dev(env)
        q = bf16(rng, sum(new), 8, D, mul=2.0).cuda()
        _, lse = moe.moe_paged_attention_shared(q, b.cache, b.d_start, b.d_len, b.d_table, max(new))
        w = torch.zeros(b.host["k_codes"].shape[:3], device="cuda")
        moe.moe_kv_weights(q, lse, b.cache, b.d_start, b.d_len, b.d_table, max(new), w)
        for s, n in enumerate(new):
            pages = [p for p in b.table[s] if p >= 0]
            assert (w[pages].double().sum((0, 2)) - 4 * n).abs().max() <= 2.0 ** -9 * 4 * n


@pytest.mark.parametrize("new", [1, 2, 20])
def test_weights_of_numbers_that_are_none(env, new):
    """A row without a denominator or with a NaN adds nothing; a NaN key gets nothing; bytes behind the end are not read."""
    moe, torch = env
    rng = np.random.default_rng(new)
    b = Batch(rng, [new, new], [100, 40], 2, 32).fill(rng)
    b.host["k_codes"][b.table[0, 1], 1, 5] = 0x7F
    b.dev(env)
    q = bf16(rng, 2 * new, 8, D)
    lse = torch.full((2 * new, 8), 4.0, device="cuda")
    lse[0, 0], lse[new - 1, 1], lse[2 * new - 1, 2] = -float("inf"), float("nan"), float("inf")
    q[0, 4, 7] = float("nan")
    q[new, 5, 8] = float("inf")
    check_weights(env, b, q, lse)


def test_weights_lengths_below_the_new_tokens(env):
    rng = np.random.default_rng(8)
    for new in ([1, 1, 1], [90, 40, 3]):
        b = Batch(rng, new, [0, 10, 200], 2, 16).fill(rng).dev(env)
        b.kv_len[0], b.kv_len[1] = 0, max(0, new[1] - 25)
        b.d_len = i32(b.kv_len)
        q = bf16(rng, sum(new), 6, D)
        for window in (0, 7, 2 ** 31 - 1):
            check_weights(env, b, q, denominators(b, q, True, window), window=window)


def test_weights_contradictions_set_the_status(env):
    moe, torch = env
    rng = np.random.default_rng(9)
    for new in (1, 30):
        b = Batch(rng, [new, new], [100, 20], 2, 16).fill(rng).dev(env)
        q = bf16(rng, 2 * new, 4, D)
        lse = torch.zeros(2 * new, 4, device="cuda")
        b.table[0, 2] = 1 << 20
        b.d_table = i32(b.table)
        check_weights(env, b, q, lse, status=moe.MOE_ERR_DEVICE_CHECK)
        b.d_len[1] = -1
        w = torch.full(b.host["k_codes"].shape[:3], 3.0, device="cuda")
        ws = moe.moe_kv_workspace()
        moe.moe_kv_weights(q.cuda(), lse, b.cache, b.d_start, b.d_len, b.d_table, new, w, ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
        assert (w[[p for p in b.table[1] if p >= 0]] == 3.0).all()


# ------------------------------------------------------------------------------------------------ eviction
def check_evict(env, rng, lengths, keep, Hkv, page, sink=0, recent=0, weight=None, extra_cols=1, slack=1):
    moe, torch = env
    B = len(lengths)
    m = [min(a, b) for a, b in zip(lengths, keep)]
    both = Batch(rng, [0] * (2 * B), list(lengths) + m, Hkv, page, extra_cols=extra_cols)
    n_pages = both.host["k_codes"].shape[0]
    both.host["k_scale"][:] = rng.integers(110, 130, (n_pages, Hkv))
    both.host["v_scale"][:] = rng.integers(60, 200, (n_pages, Hkv))
    cols = max(1, max(-(-x // page) for x in m)) + slack
    both.table[B:][both.table[B:] < 0] = -1
    table, new_table = np.ascontiguousarray(both.table[:B]), np.full((B, cols), -1, np.int32)
    for b in range(B):
        used = -(-m[b] // page)
        new_table[b, :used] = both.table[B + b, :used]
    both.dev(env)
    if weight is None:
        weight = rng.exponential(size=(n_pages, Hkv, page)) ** 3
        weight = np.where(rng.random(weight.shape) < 0.4, np.floor(weight * 8) / 8, weight).astype(np.float32)   # ties, zeros
    else:
        weight = weight(n_pages)
    w, ws = torch.from_numpy(weight.copy()).cuda(), moe.moe_kv_workspace()
    new_len, kept = moe.moe_kv_evict(both.cache, w, i32(lengths), i32(table), i32(keep), i32(new_table), sink, recent, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    ref_len, ref_kept = ol.evict(both.host, weight, lengths, table, keep, new_table, sink, recent)
    assert (new_len.cpu().numpy() == ref_len).all()
    kept = kept.cpu().numpy()
    assert np.array_equal(kept, ref_kept), np.argwhere(kept != ref_kept)[:5]
    assert np.array_equal(w.cpu().numpy().view(np.uint32), weight.view(np.uint32))
    for name, codes, scale in same_cache(both):
        assert np.array_equal(scale, both.host[name + "_scale"])
        want = both.host[name + "_codes"]
        assert np.array_equal(oa.values(codes, 0), oa.values(want, 0), equal_nan=True)
    return kept


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 10), (0, 33), (50, 0), (1000, 1000)])
def test_evict(env, page, sink, recent):
    rng = np.random.default_rng(page + sink)
    check_evict(env, rng, [700, 1, 0, 16, 129, 64, 300], [200, 1, 5, 3, 128, 0, 1000], 3, page, sink, recent)


def test_evict_equal_weights(env):
    """All the same, all zero, NaN and negative numbers (zeros), infinities: the first tokens stay."""
    rng = np.random.default_rng(2)
    same = lambda v: lambda n: np.full((n, 2, 32), v, np.float32)
    for v in (0.0, 1.0, np.nan, -3.0, np.inf, 1e-42):
        kept = check_evict(env, rng, [500, 100], [130, 33], 2, 32, weight=same(v))
        assert (kept[0, :, :130] == np.arange(130)).all()
    odd = lambda n: rng.choice(np.array([0.0, -1.0, np.nan, np.inf, 1e-42, 3e38, 1.0], np.float32), size=(n, 2, 32))
    check_evict(env, rng, [500, 100], [130, 33], 2, 32, weight=odd, sink=3, recent=7)


@pytest.mark.parametrize("length,keep,cols", [(20000, 3000, 1), (40000, 100, 1), (5000, 4999, 2000), (3, 2, 6000)])
def test_evict_over_several_blocks(env, length, keep, cols):
    """A cluster shares a sequence: long ones, and tables much wider than their sequences (blocks without tokens)."""
    rng = np.random.default_rng(length)
    check_evict(env, rng, [length], [keep], 1, 64, 4, 100, extra_cols=cols)
    check_evict(env, rng, [length, 50], [keep, 7], 2, 64, 0, 0, extra_cols=cols)


def test_evict_more_than_shared_memory_holds(env):
    """450,000 tokens: the eight blocks keep a part of their pieces and read the rest again."""
    moe, torch = env
    n, page, m = 450000, 128, 700
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(0)
    order = torch.randperm(pages + 6, device="cuda", generator=g).to(torch.int32)
    cache = moe.KVCache(*(torch.randint(0, 127, (pages + 6, 1, page, D), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2)),
                        *(torch.full((pages + 6, 1), 127, dtype=torch.uint8, device="cuda") for _ in range(2)))
    w = torch.rand(pages + 6, 1, page, device="cuda", generator=g)
    w = torch.where(w > 0.999, 0.999, w)    # equals at the top, more than there is room for when 300 stay
    flat = w[order[:pages].long()].reshape(-1)[:n].cpu().numpy()
    rank = flat.copy()
    rank[:2] = rank[n - 5:] = np.inf
    best = np.lexsort((np.arange(n), -rank))
    rows = cache.k_codes[order[:pages].long(), 0].reshape(-1, D)
    ws = moe.moe_kv_workspace()
    for keep in (m, 300):
        new_len, kept = moe.moe_kv_evict(cache, w, i32([n]), order[None, :pages].contiguous(), i32([keep]), order[None, pages:].contiguous(), 2, 5,
                                         ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK and new_len.item() == keep
        want = np.sort(best[:keep])
        assert (kept[0, 0, :keep].cpu().numpy() == want).all() and (kept[0, 0, keep:] == -1).all()
        assert torch.equal(cache.k_codes[order[pages:].long(), 0].reshape(-1, D)[:keep], rows[torch.from_numpy(want).cuda()])


def test_evict_contradictions_set_the_status(env):
    moe, torch = env
    for fault in ("keep", "length", "room", "page", "new page"):
        rng = np.random.default_rng(6)
        b = Batch(rng, [0] * 4, [100, 60, 40, 30], 2, 16).fill(rng).dev(env)
        lengths, keep, table, new = [100, 60], [40, 30], b.table[:2].copy(), b.table[2:, :3].copy()
        if fault == "keep":
            keep[0] = -1
        elif fault == "length":
            lengths[0] = 1 << 20
        elif fault == "room":
            keep[0] = 49
        elif fault == "page":
            table[0, 0] = -2
        else:
            new[0, 1] = 1 << 20
        w = torch.rand(b.host["k_codes"].shape[:3], device="cuda")
        before = [x.clone() for x in b.cache]
        ws = moe.moe_kv_workspace()
        new_len, kept = moe.moe_kv_evict(b.cache, w, i32(lengths), i32(table), i32(keep), i32(new), ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK, fault
        left_out = fault in ("keep", "length", "room")
        assert new_len.tolist() == [-1 if left_out else 40, 30]
        if left_out:
            assert (kept[0] == -1).all()
            assert torch.equal(b.cache.k_codes[b.table[2, :3]], before[0][b.table[2, :3]])
        if fault == "page":     # what lay on it counts as nothing, and stays last
            assert (kept[0, :, :40] >= 16).all()


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 2), (10, 2), (24, 2)])
@pytest.mark.parametrize("new,ctx,prefix,readers", [
    ([70], [0], [1], [1]), ([90, 40, 60], [0, 200, 31], [129, 600], [1, 2]), ([200, 30], [100, 5], [0, 77], [1, 1]),
    ([130, 0, 100, 80], [5, 9, 300, 0], [128, 500, 3], [0, 3, 1]), ([64, 300], [1000, 3], [1500], [2])])
def test_shared_many_rows(env, Hq, Hkv, new, ctx, prefix, readers):
    """Sequences of many tokens, whose rows go over their prefix and their own keys in one pass: prefixes that end within a tile, at its
    end, within 16 keys of it, that have no tokens; sequences without tokens, and shorter than what they bring."""
    rng = np.random.default_rng(Hq + len(new))
    for page in (16, 128):
        b = Shared(rng, new, ctx, prefix, readers, Hkv, page)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        q = bf16(rng, sum(new), Hq, D, mul=2.0)
        check_shared(env, b, q)
        check_shared(env, b, q, causal=False)
        b.kv_len = np.maximum(0, b.kv_len - 90).astype(np.int32)
        b.d_len = i32(b.kv_len)
        check_shared(env, b, q)


def test_shared_many_rows_contradictions(env):
    """A sequence over the border of two prefixes, a length beyond the table, a page outside the pool."""
    moe, torch = env
    rng = np.random.default_rng(7)
    new = [80, 90, 100]
    for fault in ("border", "length", "page", "end"):
        b = Shared(rng, new, [20, 0, 300], [100, 60], [1, 2], 2, 16)
        b.dev(env)
        b.d_start, b.d_len = i32(b.q_start), i32(b.kv_len)
        start, length, table, most = b.prefix()
        if fault == "border":
            start[1] = 100
        elif fault == "length":
            length[1] = 1 << 20
        elif fault == "page":
            table[0, 3] = 1 << 20
        else:
            start[2] = 260
        q = bf16(rng, sum(new), 8, D)
        ws = moe.moe_paged_attention_shared_workspace(sum(new), 3, 8, 2, D, max(new), 2, sum(new))
        out, lse = moe.moe_paged_attention_shared(q.cuda(), b.cache, b.d_start, b.d_len, i32(np.ascontiguousarray(b.table)), max(new),
                                                  (start, length, table, sum(new)), ws=ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK, fault
