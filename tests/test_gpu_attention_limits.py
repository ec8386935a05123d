"""What the attention operators leave out, and what they say about it: positions beyond the table of angles, pages that are not in
the pool, starts and lengths that do not fit together (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import D, Batch, bf16, env, f64  # noqa: E402,F401
from oracle import attention as oa  # noqa: E402

SENTINEL = 77.0


def append(env, b, q, k, v, table, status):  # noqa: F811
    """moe_kv_append into b.cache; q_out was full of sentinels."""
    moe, torch = env
    out = torch.full(q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
    b.ws.zero_()
    moe.moe_kv_append(q.cuda(), k.cuda(), v.cuda(), b.cache, b.d_start, b.d_len, b.d_table, table, q_out=out, ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == status
    return out


def codes_are(b, host):
    """Keys and values of the device's cache are the given ones, byte for byte (NaN codes aside)."""
    for name, got in zip(("k_codes", "v_codes", "k_scale", "v_scale"), b.cache):
        got, want = got.cpu().numpy(), host[name]
        if "codes" in name:
            assert np.array_equal(oa.values(got, 0), oa.values(want, 0), equal_nan=True), name
        else:
            assert (got == want).all(), name


def turned(env, x, pos, rot, max_pos):  # noqa: F811
    """(table, x rotated in 64 bits): angles of 0 and quarter turns only, so that rounding has no part in the codes."""
    moe, torch = env
    p = np.arange(max_pos)[:, None] + np.zeros(rot // 2, int)[None]
    cos, sin = np.array([1, 0, -1, 0])[p % 4], np.array([0, 1, 0, -1])[p % 4]
    cs = np.concatenate([cos, sin], 1).astype(np.float32)
    inside = pos < max_pos
    y = np.full(x.shape, np.nan)
    y[inside] = oa.norm_rotate(x[inside], pos[inside], cs, rot, False)
    return torch.from_numpy(cs).cuda(), y


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("max_pos", [37, 32, 28, 20])
def test_tokens_beyond_the_table_of_angles(env, page, max_pos):  # noqa: F811
    """A chunk that passes the table's end inside a page, at a page's end, before its first token: the tokens before that end
    are stored as if they were the chunk, their queries rotated, the others left out; the other sequence has all of its own."""
    moe, torch = env
    rng = np.random.default_rng(page + max_pos)
    b = Batch(rng, [30, 9], [20, 0], 2, page).fill(rng, upto=[20, 0]).dev(env)
    x = bf16(rng, 39, 8, D, mul=3.0)
    pos = np.concatenate([np.arange(20, 50), np.arange(9)])
    table, y = turned(env, f64(x), pos, 128, max_pos)
    out = append(env, b, x[:, :4], x[:, 4:6], x[:, 6:], table, moe.MOE_ERR_DEVICE_CHECK)
    inside = pos < max_pos
    assert np.array_equal(f64(out)[inside], y[inside, :4]) and (f64(out)[~inside] == SENTINEL).all()
    kept = [int(inside[:30].sum()), int(inside[30:].sum())]
    rows = np.r_[0:kept[0], 30:30 + kept[1]]
    oa.append(y[rows, 4:6], f64(x)[rows, 6:], b.host, [0, kept[0], sum(kept)], [20 + kept[0], kept[1]], b.table)
    codes_are(b, b.host)


@pytest.mark.parametrize("bad", [1 << 20, -7])
def test_append_on_a_page_that_is_not_there(env, bad):  # noqa: F811
    """The tokens of that page are not stored; those of the pages around it are, and all queries are rotated."""
    moe, torch = env
    rng = np.random.default_rng(3)
    b = Batch(rng, [40, 5], [10, 0], 2, 16).fill(rng, upto=[10, 0]).dev(env)
    x = bf16(rng, 45, 8, D)
    pos = np.concatenate([np.arange(10, 50), np.arange(5)])
    table, y = turned(env, f64(x), pos, 128, 64)
    b.d_table[0, 1] = bad
    out = append(env, b, x[:, :4], x[:, 4:6], x[:, 6:], table, moe.MOE_ERR_DEVICE_CHECK)
    assert np.array_equal(f64(out), y[:, :4])
    lost = b.table[0, 1]
    before = {n: a[lost].copy() for n, a in b.host.items()}
    oa.append(y[:, 4:6], f64(x)[:, 6:], b.host, b.q_start, b.kv_len, b.table)
    for n, a in before.items():
        b.host[n][lost] = a
    codes_are(b, b.host)


def test_append_of_more_new_tokens_than_tokens(env):  # noqa: F811
    """A length below the sequence's new tokens: none of them is stored, queries before position 0 are left out."""
    moe, torch = env
    rng = np.random.default_rng(4)
    b = Batch(rng, [6, 5], [20, 3], 2, 16).fill(rng, upto=[20, 3]).dev(env)
    x = bf16(rng, 11, 8, D)
    b.d_len[0] = 4
    pos = np.concatenate([np.arange(-2, 4), np.arange(3, 8)])
    table, y = turned(env, f64(x), pos.clip(0), 128, 64)
    out = append(env, b, x[:, :4], x[:, 4:6], x[:, 6:], table, moe.MOE_ERR_DEVICE_CHECK)
    assert (f64(out)[:2] == SENTINEL).all() and np.array_equal(f64(out)[2:], y[2:, :4])
    oa.append(y[6:, 4:6], f64(x)[6:, 6:], b.host, [0, 0, 5], [20, 8], b.table)
    codes_are(b, b.host)


def rows_ok(got, ref, spread, rows):
    return (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread)[rows].all()


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 5], [90, 40, 60], [300, 20, 1]])
@pytest.mark.parametrize("window", [0, 9, 2 ** 31 - 1])
def test_attention_of_more_new_tokens_than_tokens(env, new, window):  # noqa: F811
    """A new token before position 0 sees nothing: its rows are zeros.  That is no error (a token that is the first of
    nothing), and the others' rows are right, whatever the window."""
    moe, torch = env
    rng = np.random.default_rng(5 + new[0])
    b = Batch(rng, new, [30, 10, 200], 2, 32).fill(rng).dev(env)
    b.kv_len[0], b.kv_len[1] = new[0] // 2, 0
    b.d_len = torch.from_numpy(b.kv_len).cuda()
    q = bf16(rng, sum(new), 4, D)
    ws = moe.moe_paged_attention_workspace(sum(new), 3, 4, 2, D, max(new))
    out = moe.moe_paged_attention(q.cuda(), b.cache, b.d_start, b.d_len, b.d_table, max_q=max(new), window=window, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    ref, spread = oa.attention(f64(q), b.host, b.q_start, b.kv_len, b.table, D ** -0.5, True, window)
    assert rows_ok(out, ref, spread, slice(None))
    assert (out[:new[0] - new[0] // 2] == 0).all() and (out[new[0]:new[0] + new[1]] == 0).all()


@pytest.mark.parametrize("new", [[2, 1, 1], [70, 20, 60], [200, 5, 3]])
@pytest.mark.parametrize("end", ["first", "last"])
def test_starts_that_leave_tokens_out(env, new, end):  # noqa: F811
    """Tokens before the first start or behind the last one belong to no sequence: the status says so, for the attention as
    for an append with queries or without."""
    moe, torch = env
    rng = np.random.default_rng(6)
    T = sum(new)
    b = Batch(rng, new, [30, 10, 200], 2, 32).fill(rng).dev(env)
    q = bf16(rng, T, 4, D)
    b.d_start[0 if end == "first" else 3] += 1 if end == "first" else -1
    b.d_len[0 if end == "first" else 2] -= 1
    ws = moe.moe_paged_attention_workspace(T, 3, 4, 2, D, max(new))
    out = torch.full(q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
    moe.moe_paged_attention(q.cuda(), b.cache, b.d_start, b.d_len, b.d_table, max_q=max(new), out=out, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    start, lens = b.d_start.cpu().numpy(), b.d_len.cpu().numpy()
    ref, spread = oa.attention(f64(q), b.host, start, lens, b.table, D ** -0.5)
    assert rows_ok(out, ref, spread, slice(start[0], start[3]))
    assert (out[:start[0]] == SENTINEL).all() and (out[start[3]:] == SENTINEL).all()
    k = bf16(rng, T, 2, D).cuda()
    for queries in (q.cuda(), None):
        b.ws.zero_()
        moe.moe_kv_append(queries, k, k, b.cache, b.d_start, b.d_len, b.d_table, None, ws=b.ws)
        assert moe.moe_get_device_status(b.ws) == moe.MOE_ERR_DEVICE_CHECK


def test_gather_around_a_page_that_is_not_there(env):  # noqa: F811
    """The rows of that page are zeros, keys and values alike, and all others are the cached tokens."""
    moe, torch = env
    rng = np.random.default_rng(8)
    b = Batch(rng, [0] * 3, [40, 150, 64], 3, 32).fill(rng, 3.0, 0.01).dev(env)
    start, count = [3, 13, 0], [37, 137, 64]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    b.d_table[1, 2] = 1 << 20
    b.table[1, 2] = 1 << 20
    k, v = moe.moe_kv_gather(b.cache, i32(start), i32(np.cumsum([0] + count)), b.d_table, sum(count), ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    for name, got in (("k", k), ("v", v)):
        ref = np.concatenate([oa.read(b.host, name, s, x, x + n, b.table) for s, (x, n) in enumerate(zip(start, count))])
        lost = slice(37 + 64 - 13, 37 + 96 - 13)
        assert np.isnan(ref[lost]).all()
        ref[lost] = 0.0
        assert np.array_equal(f64(got), ref)


def test_gather_of_rows_that_no_sequence_has(env):  # noqa: F811
    """Rows behind the last end are zeros, and reported."""
    moe, torch = env
    rng = np.random.default_rng(9)
    b = Batch(rng, [0], [12], 2, 16).fill(rng).dev(env)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = moe.moe_kv_gather(b.cache, i32([0]), i32([0, 5]), b.d_table, 9, ws=b.ws)
    assert moe.moe_get_device_status(b.ws) == moe.MOE_ERR_DEVICE_CHECK
    assert np.array_equal(f64(k)[:5], oa.read(b.host, "k", 0, 0, 5, b.table)) and (k[5:] == 0).all() and (v[5:] == 0).all()
