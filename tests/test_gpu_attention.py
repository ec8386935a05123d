"""The attention operators against the float64 oracle (GPU).

Tolerances.  Roundings are off by at most half a step: bf16 2^-8 and E4M3 2^-4 of the value (2^-10 of the page's scale
for E4M3 subnormals).  moe_kv_append rounds once, after fp32 arithmetic of relative error below 2^-18 of the pair's size.
moe_paged_attention rounds its output once (2^-8 |out|); a weight p_j enters the product with V as a number of at least
8 significant bits (2^-8 p_j, or 2^-18 of the largest weight), the scores are fp32 sums of 128 products (their error, times
a score's size of up to 20, stays under 2^-12): 2^-7 sum_j p_j |v_j| covers these with the order of the sums.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import attention as oa  # noqa: E402
from oracle import bf16_to_f64  # noqa: E402

D = 128


@pytest.fixture(scope="module")
def env():
    import torch

    from moe_expert_layer_fwd_gb300 import build
    build.build()
    import moe_expert_layer_fwd_gb300 as moe
    return moe, torch


def bf16(rng, *shape, mul=1.0):
    import torch
    return torch.from_numpy((rng.normal(size=shape) * mul).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    import torch
    return bf16_to_f64(t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16))


class Batch:
    """Lengths, shuffled pages and a cache of random codes (any byte, so NaN codes and stale scales are among them)."""

    def __init__(self, rng, new, ctx, Hkv, page, spare=2, extra_cols=1):
        self.new, self.ctx, self.page, self.Hkv = new, ctx, page, Hkv
        self.total = [a + b for a, b in zip(new, ctx)]
        used = [-(-t // page) for t in self.total]
        n = sum(used) + spare
        ids = rng.permutation(n)
        self.table = np.full((len(new), max(used + [0]) + extra_cols), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u
        self.q_start = np.cumsum([0] + new).astype(np.int32)
        self.kv_len = np.array(self.total, np.int32)
        self.host = dict(k_codes=rng.integers(0, 256, (n, Hkv, page, D)).astype(np.uint8),
                         v_codes=rng.integers(0, 256, (n, Hkv, page, D)).astype(np.uint8),
                         k_scale=rng.integers(0, 256, (n, Hkv)).astype(np.uint8),
                         v_scale=rng.integers(0, 256, (n, Hkv)).astype(np.uint8))

    def fill(self, rng, k_mul=1.0, v_mul=1.0, upto=None):
        """Stores the tokens before the new ones (upto: all of them, or only the context) through the oracle."""
        lens = self.total if upto is None else upto
        t = sum(lens)
        k, v = rng.normal(size=(t, self.Hkv, D)) * k_mul, rng.normal(size=(t, self.Hkv, D)) * v_mul
        oa.append(k, v, self.host, np.cumsum([0] + list(lens)), lens, self.table)
        return self

    def dev(self, env):
        moe, torch = env
        cuda = lambda a: torch.from_numpy(a).cuda()
        self.cache = moe.KVCache(*(cuda(self.host[n].copy()) for n in ("k_codes", "v_codes", "k_scale", "v_scale")))
        self.d_start, self.d_len, self.d_table = cuda(self.q_start), cuda(self.kv_len), cuda(self.table)
        self.ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        return self


def same_cache(b):
    """The device cache holds the oracle's codes and scales wherever a sequence has tokens."""
    for name in ("k", "v"):
        codes = getattr(b.cache, name + "_codes").cpu().numpy()
        scale = getattr(b.cache, name + "_scale").cpu().numpy()
        yield name, codes, scale


RAGGED = dict(new=[3, 0, 1, 40, 17], ctx=[0, 9, 31, 5, 64])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,rot,interleaved,norm", [(8, 2, 128, False, True), (3, 1, 64, True, False),
                                                         (20, 4, 96, False, False), (12, 12, 32, True, True),
                                                         (5, 5, 0, False, True), (16, 2, 16, False, False)])
def test_append(env, page, Hq, Hkv, rot, interleaved, norm):
    moe, torch = env
    rng = np.random.default_rng(page * 1000 + Hq)
    b = Batch(rng, **RAGGED, Hkv=Hkv, page=page).fill(rng, upto=RAGGED["ctx"]).dev(env)
    T = sum(b.new)
    qkv = bf16(rng, T, Hq + 2 * Hkv, D, mul=3.0)
    wq, wk = bf16(rng, D), bf16(rng, D)
    table = moe.moe_rope_table(128, rot, 1e4) if rot else None
    q, k, v = qkv.cuda().split([Hq, Hkv, Hkv], dim=1)
    out = moe.moe_kv_append(q, k, v, b.cache, b.d_start, b.d_len, b.d_table, table, interleaved=interleaved,
                            q_norm_weight=wq.cuda() if norm else None, k_norm_weight=wk.cuda() if norm else None, ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == moe.MOE_OK
    pos = np.concatenate([np.arange(c, c + n) for n, c in zip(b.new, b.ctx)])
    cs = table.cpu().numpy() if rot else np.zeros((128, 0), np.float32)
    x = f64(qkv)
    turn = lambda y, w: oa.norm_rotate(y, pos, cs, rot, interleaved, f64(w) if norm else None)
    ref_q, ref_k, ref_v = turn(x[:, :Hq], wq), turn(x[:, Hq:Hq + Hkv], wk), x[:, Hq + Hkv:]
    size = np.abs(ref_q).max(-1, keepdims=True)
    assert (np.abs(f64(out) - ref_q) <= 2.0 ** -8 * np.abs(ref_q) + 2.0 ** -18 * size).all()
    before = {n: a.copy() for n, a in b.host.items()}
    oa.append(ref_k, ref_v, b.host, b.q_start, b.kv_len, b.table)
    for name, codes, scale in same_cache(b):
        want = b.host[name + "_scale"]
        touched = np.zeros_like(want, dtype=bool)
        for s in range(len(b.new)):
            for j in range(b.ctx[s] // page, -(-b.total[s] // page)) if b.new[s] else ():
                p = b.table[s, j]
                touched[p] = True
                lo = max(0, b.ctx[s] - j * page)
                hi = min(page, b.total[s] - j * page)
                assert (scale[p] == want[p]).all()
                # earlier tokens: exactly the oracle's; new ones: within one rounding of the unrounded value
                assert (oa.values(codes[p, :, :lo], 0) == oa.values(b.host[name + "_codes"][p, :, :lo], 0)).all()
                t = b.q_start[s] + j * page + lo - b.ctx[s]
                y = (ref_k if name == "k" else ref_v)[t:t + hi - lo].transpose(1, 0, 2)
                unit = 2.0 ** (want[p].astype(int) - 127)[:, None, None]
                got = oa.values(codes[p, :, lo:hi], 0) * unit
                size = np.abs(y).max(-1, keepdims=True)
                assert (np.abs(got - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * unit) + 2.0 ** -18 * size).all()
                # bytes behind the last token are left alone
                assert (codes[p, :, hi:] == before[name + "_codes"][p, :, hi:]).all()
        assert (codes[~touched.any(1)] == before[name + "_codes"][~touched.any(1)]).all()
        assert (scale[~touched] == before[name + "_scale"][~touched]).all()


def test_append_again_changes_nothing(env):
    moe, torch = env
    rng = np.random.default_rng(5)
    b = Batch(rng, **RAGGED, Hkv=2, page=32).fill(rng, 0.1, 0.1, upto=RAGGED["ctx"]).dev(env)
    T = sum(b.new)
    k, v, table = bf16(rng, T, 2, D).cuda(), bf16(rng, T, 2, D).cuda(), moe.moe_rope_table(128)
    call = lambda: moe.moe_kv_append(None, k, v, b.cache, b.d_start, b.d_len, b.d_table, table, ws=b.ws)
    assert call() is None
    first = [t.clone() for t in b.cache]
    call()
    assert all(torch.equal(x, y) for x, y in zip(first, b.cache))


def test_append_extremes(env):
    """Zero, tiny, huge and infinite rows set the scales they should; a NaN becomes a NaN key row and a zero value."""
    moe, torch = env
    rng = np.random.default_rng(6)
    b = Batch(rng, [16, 16, 16, 16], [0, 0, 0, 0], 1, 16).dev(env)
    k, v = bf16(rng, 64, 1, D), bf16(rng, 64, 1, D)
    k[:16], v[:16] = 0, 1e-30
    k[16:32] = k[16:32] * 1e38
    v[20, 0, 3] = float("inf")
    v[21, 0, 4] = -float("inf")
    v[33, 0, 7] = float("nan")
    k[35, 0, 1] = float("nan")
    moe.moe_kv_append(None, k.cuda(), v.cuda(), b.cache, b.d_start, b.d_len, b.d_table, None, ws=b.ws)
    k64, v64 = f64(k), f64(v)
    oa.append(k64, v64, b.host, b.q_start, b.kv_len, b.table)
    used = b.table[:, 0]
    for name, codes, scale in same_cache(b):
        assert (scale[used] == b.host[name + "_scale"][used]).all()
        same = oa.values(codes[used], 0), oa.values(b.host[name + "_codes"][used], 0)
        assert np.array_equal(*same, equal_nan=True)
    assert (b.cache.k_codes[used[2], 0, 1].cpu() == 0x7F).all() and (b.cache.v_codes[used[2], 0, 1, 7].cpu() & 0x7F == 0)


def test_append_contradictions_set_the_status(env):
    moe, torch = env
    rng = np.random.default_rng(7)
    for fault in ("page", "length", "position", "order"):
        b = Batch(rng, [4, 4], [20, 0], 2, 16).fill(rng, upto=[20, 0]).dev(env)
        if fault == "page":
            b.d_table[0, 1] = 1 << 20
        elif fault == "length":
            b.d_len[0] = 2          # fewer tokens than it brings
        elif fault == "order":
            b.d_start[1] = 9
        x = bf16(rng, 8, 2, D).cuda()
        before = b.cache.k_codes.clone()
        table = moe.moe_rope_table(22 if fault == "position" else 64)
        moe.moe_kv_append(x, x, x, b.cache, b.d_start, b.d_len, b.d_table, table, ws=b.ws)
        assert moe.moe_get_device_status(b.ws) == moe.MOE_ERR_DEVICE_CHECK, fault
        keep = [p for p in range(before.shape[0]) if p not in b.table[0, :2].tolist() + b.table[1, :1].tolist()]
        assert torch.equal(b.cache.k_codes[keep], before[keep])


def test_gather(env):
    moe, torch = env
    rng = np.random.default_rng(8)
    for page, Hkv in ((16, 1), (32, 3), (64, 4), (128, 2)):
        b = Batch(rng, [0] * 4, [7, 150, 64, 33], Hkv, page).fill(rng, 3.0, 0.01).dev(env)
        start, count = [0, 13, 63, 33], [7, 137, 1, 0]
        out_start = torch.tensor(np.cumsum([0] + count), dtype=torch.int32, device="cuda")
        k, v = moe.moe_kv_gather(b.cache, torch.tensor(start, dtype=torch.int32, device="cuda"), out_start, b.d_table,
                                 sum(count), ws=b.ws)
        assert moe.moe_get_device_status(b.ws) == moe.MOE_OK
        for name, got in (("k", k), ("v", v)):
            ref = np.concatenate([oa.read(b.host, name, s, x, x + n, b.table) for s, (x, n) in enumerate(zip(start, count))])
            assert np.array_equal(f64(got), ref, equal_nan=True)
    b.d_table[1, 0] = -5
    k, v = moe.moe_kv_gather(b.cache, torch.tensor(start, dtype=torch.int32, device="cuda"), out_start, b.d_table, sum(count), ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    assert (k[7:7 + 115] == 0).all() and torch.equal(v[7 + 115:].cpu(), v.cpu()[7 + 115:])


def attend(env, b, q, status=0, **kw):
    moe, torch = env
    qd = q.cuda()
    kw.setdefault("max_q", max(b.new))
    ws = moe.moe_paged_attention_workspace(q.shape[0], len(b.new), q.shape[1], b.Hkv, D, kw["max_q"])
    out = moe.moe_paged_attention(qd, b.cache, b.d_start, b.d_len, b.d_table, ws=ws, **kw)
    assert moe.moe_get_device_status(ws) == status
    return out


def check(env, b, q, scale=D ** -0.5, causal=True, window=0, **kw):
    out = attend(env, b, q, scale=scale, causal=causal, window=window, **kw)
    ref, spread = oa.attention(f64(q), b.host, b.q_start, b.kv_len, b.table, scale, causal, window)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return out


HEADS = [(8, 1), (16, 2), (4, 4), (10, 2), (7, 1), (24, 2)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_decode(env, page, Hq, Hkv):
    rng = np.random.default_rng(page + 7 * Hq)
    total = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300, 700, 33]
    b = Batch(rng, [1] * len(total), [t - 1 for t in total], Hkv, page).fill(rng, 1.0, 2.0).dev(env)
    check(env, b, bf16(rng, len(total), Hq, D, mul=2.0))


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("new,ctx", [([2, 0, 5, 3, 1], [0, 40, 130, 255, 64]), ([4, 4], [500, 3]), ([8], [121])])
def test_several_tokens(env, Hq, Hkv, new, ctx):
    rng = np.random.default_rng(11 * Hq + len(new))
    b = Batch(rng, new, ctx, Hkv, 32).fill(rng).dev(env)
    q = bf16(rng, sum(new), Hq, D, mul=2.0)
    for causal, window in ((True, 0), (True, 1), (True, 50), (False, 0)):
        check(env, b, q, causal=causal, window=window)


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("new,ctx", [([130], [0]), ([33, 0, 150, 1], [100, 7, 0, 300]), ([257, 70], [3, 129])])
def test_prefill(env, Hq, Hkv, new, ctx):
    rng = np.random.default_rng(13 * Hq + len(new))
    b = Batch(rng, new, ctx, Hkv, 64).fill(rng, 1.0, 0.3).dev(env)
    q = bf16(rng, sum(new), Hq, D, mul=2.0)
    for causal, window in ((True, 0), (True, 100), (False, 0)):
        check(env, b, q, causal=causal, window=window)


@pytest.mark.parametrize("page", [16, 32, 128])
def test_prefill_pages(env, page):
    rng = np.random.default_rng(page)
    b = Batch(rng, [140, 60], [37, 210], 2, page).fill(rng).dev(env)
    check(env, b, bf16(rng, 200, 8, D))


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 40, 3]])
def test_lengths_that_leave_rows_empty(env, new):
    """A sequence without tokens, and one whose first new tokens lie before its start (more new tokens than tokens)."""
    moe, torch = env
    rng = np.random.default_rng(17)
    b = Batch(rng, new, [0, 10, 200], 2, 16).fill(rng).dev(env)
    b.kv_len[0] = 0
    b.kv_len[1] = max(0, new[1] - 25)
    b.d_len = torch.from_numpy(b.kv_len).cuda()
    out = check(env, b, bf16(rng, sum(new), 6, D))
    assert (out[:new[0]] == 0).all()


@pytest.mark.parametrize("new", [1, 3, 150])
def test_masked_numbers_do_not_reach_the_output(env, new):
    """Keys and values that a row does not see may be NaN or huge: behind the end of a page (random bytes everywhere in
    these tests), before the window, and -- through the append -- in later tokens of the same call."""
    moe, torch = env
    rng = np.random.default_rng(19 + new)
    b = Batch(rng, [new] * 2, [100, 300], 2, 32).fill(rng, upto=[100, 300]).dev(env)
    k, v = bf16(rng, 2 * new, 2, D), bf16(rng, 2 * new, 2, D)
    k[new - 1, 0, 5] = float("nan")
    v[2 * new - 1, 1, 9] = float("nan")
    moe.moe_kv_append(None, k.cuda(), v.cuda(), b.cache, b.d_start, b.d_len, b.d_table, None, ws=b.ws)
    oa.append(f64(k), f64(v), b.host, b.q_start, b.kv_len, b.table)
    q = bf16(rng, 2 * new, 8, D)
    out = check(env, b, q)
    assert torch.isnan(out[new - 1, :4]).all() and not torch.isnan(out[new - 1, 4:]).any()
    assert torch.isnan(out[2 * new - 1, 4:]).all() and not torch.isnan(out[:new - 1]).any()
    # NaN before the window
    b = Batch(rng, [new] * 2, [100, 300], 2, 32).fill(rng).dev(env)
    for name in ("k_codes", "v_codes"):
        for s in range(2):
            b.host[name][b.table[s, 1], :, :7] = 0x7F
            b.host[name][b.table[s, 2], :, 3] = 0xFF
    b.dev(env)
    check(env, b, q, window=25)


def test_scales_of_pages_far_apart(env):
    """Pages whose scales differ by many powers of two, among them pages of zeros."""
    for new in (1, 140):
        rng = np.random.default_rng(23 + new)
        b = Batch(rng, [new], [600], 1, 16).fill(rng)
        for j in range(0, 30):
            b.host["v_scale"][b.table[0, j]] = 127 + rng.integers(-30, 10)
            b.host["k_scale"][b.table[0, j]] = 127 - 8 - rng.integers(0, 30)
        b.host["v_codes"][b.table[0, 5]] = 0
        b.host["v_scale"][b.table[0, 5]] = 63
        b.dev(env)
        check(env, b, bf16(rng, new, 8, D))


def test_large_and_small_queries(env):
    rng = np.random.default_rng(29)
    for new in ([1] * 5, [40] * 5):
        b = Batch(rng, new, [200] * 5, 2, 64).fill(rng).dev(env)
        q = bf16(rng, sum(new), 8, D)
        for s, mul in enumerate((0.0, 1e-20, 1e3, 1e-4, 1.0)):
            q[sum(new[:s]):sum(new[:s + 1])] *= mul
        q[sum(new[:4]), 3, 100] = 40.0            # one element far above the rest of its row
        check(env, b, q, scale=1e-3)
        check(env, b, q * 0.01, scale=3.0)


def test_one_key_has_all_the_weight(env):
    rng = np.random.default_rng(31)
    for new in (1, 130):
        b = Batch(rng, [new], [500], 1, 64).fill(rng, k_mul=4.0).dev(env)
        out = check(env, b, bf16(rng, new, 4, D, mul=20.0))
        assert not out.isnan().any()


@pytest.mark.parametrize("new", [[1, 1, 1], [50, 70, 2]])
def test_bad_pages_and_lengths_set_the_status(env, new):
    moe, torch = env
    rng = np.random.default_rng(37)
    b = Batch(rng, new, [300, 60, 80], 2, 32).fill(rng).dev(env)
    q = bf16(rng, sum(new), 8, D)
    b.table[0, 3] = 1 << 20
    b.table[2, 1] = -7
    b.d_table = torch.from_numpy(b.table).cuda()
    check(env, b, q, status=moe.MOE_ERR_DEVICE_CHECK)      # tokens on such a page are not seen
    b = Batch(rng, new, [300, 60, 80], 2, 32).fill(rng).dev(env)
    b.d_len[1] = 1 << 30
    out = attend(env, b, q, status=moe.MOE_ERR_DEVICE_CHECK)
    ref, spread = oa.attention(f64(q), b.host, b.q_start, b.kv_len, b.table, D ** -0.5)
    rows = np.r_[0:new[0], new[0] + new[1]:sum(new)]
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread)[rows].all()


def test_strides_stream_and_reuse(env):
    """Queries inside a wider row, on a stream of their own, twice in one workspace: the same bits each time."""
    moe, torch = env
    rng = np.random.default_rng(41)
    for new in ([1] * 6, [45, 1, 90]):
        ctx = [int(x) for x in rng.integers(0, 900, len(new))]
        b = Batch(rng, new, ctx, 2, 64).fill(rng).dev(env)
        wide = bf16(rng, sum(new), 14, D).cuda()
        q = wide[:, 3:11]
        plain = attend(env, b, q.contiguous().cpu())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = moe.moe_paged_attention_workspace(sum(new), len(new), 8, 2, D, max(new))
        torch.cuda.synchronize()
        one = moe.moe_paged_attention(q, b.cache, b.d_start, b.d_len, b.d_table, max_q=max(new), ws=ws, stream=s)
        two = moe.moe_paged_attention(q, b.cache, b.d_start, b.d_len, b.d_table, max_q=max(new), ws=ws, stream=s)
        s.synchronize()
        assert torch.equal(one, plain) and torch.equal(two, plain)


def test_graph_follows_the_lengths(env):
    """A captured append + attention replays over lengths and a page table that change between replays."""
    moe, torch = env
    rng = np.random.default_rng(43)
    layer = moe.AttentionLayer(24, 8, 2, page=16, max_pos=256)
    table = torch.from_numpy(rng.permutation(24).reshape(2, 12).astype(np.int32)).cuda()
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    qkv = torch.zeros(2, 12 * D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.forward(qkv, start, lens, table, 1)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.forward(qkv, start, lens, table, 1)
    other = moe.AttentionLayer(24, 8, 2, page=16, max_pos=256)
    for step in range(40):
        lens.fill_(step + 1)
        qkv.copy_(bf16(rng, 2, 12 * D))
        g.replay()
        assert torch.equal(out, other.forward(qkv, start, lens, table, 1))
    assert moe.moe_get_device_status(layer.ws) == moe.MOE_OK


def test_layer_workspace_grows_behind_a_graph(env):
    """A decode graph captured before a prompt made the layer's workspace grow still has its own: replays give the same
    bits, and write nothing into memory that was allocated since.  The prompt runs on a stream of its own."""
    moe, torch = env
    rng = np.random.default_rng(53)
    layers = [moe.AttentionLayer(80, 8, 2, page=16, max_pos=1024) for _ in range(2)]
    table = torch.from_numpy(rng.permutation(80).reshape(1, 80).astype(np.int32)).cuda()
    start, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [1]))
    qkv = torch.zeros(1, 12 * D, dtype=torch.bfloat16, device="cuda")
    prompt, p_start, p_len = bf16(rng, 700, 12 * D).cuda(), *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                                                             ([0, 700], [700]))
    for layer in layers:
        layer.forward(qkv, start, lens, table, 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layers[0].forward(qkv, start, lens, table, 1)
    small = layers[0].ws.numel()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one = layers[0].forward(prompt, p_start, p_len, table, 700, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert layers[0].ws.numel() > small
    assert torch.equal(one, layers[1].forward(prompt, p_start, p_len, table, 700))
    since = [torch.full((small,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for step in range(4):
        lens.fill_(701 + step)
        qkv.copy_(bf16(rng, 1, 12 * D))
        g.replay()
        assert torch.equal(out, layers[1].forward(qkv, start, lens, table, 1))
    assert all(bool((t == 7).all()) for t in since)
    assert all(moe.moe_get_device_status(layer.ws) == moe.MOE_OK for layer in layers)


def test_cache_beyond_2_31_bytes(env):
    """Pages whose codes start past 2^31 bytes of the pool."""
    moe, torch = env
    rng = np.random.default_rng(47)
    n_pages, Hkv, page = 70000, 2, 128
    kv = moe.KVCache.empty(n_pages, Hkv, page)
    for new in (1, 140):
        small = Batch(rng, [new], [290], Hkv, page, spare=0, extra_cols=0)
        small.fill(rng).dev(env)
        used = small.table[0]
        far = n_pages - 1 - np.arange(len(used))
        for big, t in zip(kv, small.cache):
            big[torch.from_numpy(far).cuda()] = t[torch.from_numpy(used).cuda().long()]
        small.cache, small.d_table = kv, torch.from_numpy(far[None].astype(np.int32)).cuda()
        check(env, small, bf16(rng, new, 8, D))
        k, _ = moe.moe_kv_gather(kv, torch.tensor([0], dtype=torch.int32, device="cuda"),
                                 torch.tensor([0, 290], dtype=torch.int32, device="cuda"), small.d_table, 290)
        assert np.array_equal(f64(k), oa.read(small.host, "k", 0, 0, 290, small.table))


def test_long_cache_is_split_and_joined(env):
    """One sequence of many tiles over few heads: every part of the split contributes its share."""
    rng = np.random.default_rng(53)
    for new in (1, 40):
        b = Batch(rng, [new, new], [20000, 3000], 1, 128).fill(rng).dev(env)
        check(env, b, bf16(rng, 2 * new, 2, D, mul=3.0))


@pytest.mark.parametrize("new", [1, 4, 60])
def test_wait_limit_is_reported_and_recoverable(env, new):
    """The values' copies are withheld: the waits for them run out, the kernel records it and returns, and the next call on the
    same context is correct."""
    moe, torch = env
    rng = np.random.default_rng(59)
    b = Batch(rng, [new] * 3, [400, 90, 1500], 2, 64).fill(rng).dev(env)
    q = bf16(rng, 3 * new, 8, D)
    L = moe.lib()
    try:
        assert L.moe_debug_set(1, 20_000_000) == moe.MOE_OK and L.moe_debug_set(4, 1) == moe.MOE_OK
        attend(env, b, q, status=moe.MOE_ERR_TIMEOUT)
    finally:
        L.moe_debug_set(4, 0)
        L.moe_debug_set(1, 0)
    check(env, b, q)


def test_guards_around_every_output(env):
    """Outputs in the middle of larger buffers, whose 4 KB before and after stay as they were."""
    moe, torch = env
    rng = np.random.default_rng(61)

    def guarded(*shape, dtype=torch.bfloat16):
        n = int(np.prod(shape))
        g = 4096 // torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * g,), 77, dtype=dtype, device="cuda")
        return buf[g:g + n].view(*shape), lambda: bool((buf[:g] == 77).all()) and bool((buf[g + n:] == 77).all())

    for new in ([1, 1], [3, 5], [45, 200]):
        T = sum(new)
        b = Batch(rng, new, [70, 13], 2, 16).fill(rng, upto=[70, 13]).dev(env)
        fields, intact = [], []
        for x in b.cache:
            y, ok = guarded(*x.shape, dtype=torch.uint8)
            y.copy_(x)
            fields.append(y)
            intact.append(ok)
        b.cache = moe.KVCache(*fields)
        k, v, q = bf16(rng, T, 2, D), bf16(rng, T, 2, D), bf16(rng, T, 8, D)
        rq, ok = guarded(T, 8, D)
        intact.append(ok)
        moe.moe_kv_append(q.cuda(), k.cuda(), v.cuda(), b.cache, b.d_start, b.d_len, b.d_table, None, q_out=rq, ws=b.ws)
        oa.append(f64(k), f64(v), b.host, b.q_start, b.kv_len, b.table)
        out, ok = guarded(T, 8, D)
        intact.append(ok)
        ws, ok = guarded(moe.lib().moe_paged_attention_workspace_size(
            moe.ctypes.byref(moe.moe_kv_desc(2, T, 8, 2, D, 16, 0, 0)), max(new)), dtype=torch.uint8)
        intact.append(ok)
        moe.moe_workspace_init(ws)
        moe.moe_paged_attention(rq, b.cache, b.d_start, b.d_len, b.d_table, max_q=max(new), out=out, ws=ws)
        n = sum(b.total)
        gk, ok = guarded(n, 2, D)
        intact.append(ok)
        gv, ok = guarded(n, 2, D)
        intact.append(ok)
        start = torch.zeros(2, dtype=torch.int32, device="cuda")
        ends = torch.tensor([0, b.total[0], n], dtype=torch.int32, device="cuda")
        moe.moe_kv_gather(b.cache, start, ends, b.d_table, n, k=gk, v=gv, ws=b.ws)
        torch.cuda.synchronize()
        assert all(ok() for ok in intact)
        ref, spread = oa.attention(f64(q), b.host, b.q_start, b.kv_len, b.table, D ** -0.5)
        assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread).all()


@pytest.mark.parametrize("B", [1, 33, 300])
def test_many_sequences(env, B):
    """More sequences than one step of the searches and scans covers, some of them without new tokens or without any."""
    rng = np.random.default_rng(67 + B)
    for most in (1, 40):
        new = [int(x) for x in rng.integers(0, most + 1, B)]
        new[0] = most
        ctx = [int(x) for x in rng.integers(0, 150, B)]
        b = Batch(rng, new, ctx, 1, 16).fill(rng).dev(env)
        check(env, b, bf16(rng, sum(new), 4, D), max_q=most)


def test_decoder_layer_example(env):
    """Decoding token by token ends in the state that the whole sequences give at once, up to the layer's bf16 roundings (and the
    8-bit cache's second rounding where a page's scale grew: half an E4M3 step of single keys and values, averaged over the
    sequence).  Every expert is chosen, so that no near tie of the router turns a rounding into another choice."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.run(prompt=100, steps=20, batch=3, k=16, say=lambda *_: None) < 5e-2
