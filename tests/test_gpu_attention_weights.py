"""Attention where one key has nearly all of the softmax and thousands of others share the rest (GPU).

The tolerance is that of the other attention tests: one bf16 rounding of the output (2^-8 |out|) and 2^-7 sum_j p_j |v_j|, which
is twice what weights of 8 significant bits can be off by.  With the dominant key's value zero the output is the others'
share alone, and the sum on the right is as small.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import D, Batch, env, f64  # noqa: E402,F401
from oracle import attention as oa  # noqa: E402

GAPS = (8, 10, 12, 14, 16)   # natural logarithms


def dominated(rng, keys, place, new, Hq, sequences):
    """(batch, queries): `sequences` sequences that share one cache of 2 heads.  One key has element 0 alone, the others all but
    that, so that a query's element 0 sets the one key's score and its other elements the rest's.  Its value is zero in the first head.
    Sequence s has the gap GAPS[s % 5]; the others' scores are N(0, 0.5) or, in every other five, all equal."""
    b = Batch(rng, [new], [keys - new], 2, 64)
    at = {"first": 0, "middle": keys // 2 + 3, "last": keys - 1}[place]
    k, v = rng.normal(size=(keys, 2, D)), rng.normal(size=(keys, 2, D)) + 1.0
    k[:, :, 0] = 0.0
    k[at] = 0.0
    k[at, :, 0] = 8.0
    v[at, 0] = 0.0
    oa.append(k, v, b.host, [0, keys], [keys], b.table)
    b.new, b.ctx, b.total = [new] * sequences, [keys - new] * sequences, [keys] * sequences
    b.table = np.repeat(b.table, sequences, 0)
    b.q_start = (np.arange(sequences + 1) * new).astype(np.int32)
    b.kv_len = np.full(sequences, keys, np.int32)
    q = rng.normal(size=(sequences, new, Hq, D)) * 0.5
    s = np.arange(sequences)
    q[s // 5 % 2 == 1] = 0.0
    q[..., 0] = (np.array(GAPS)[s % 5] * D ** 0.5 / 8.0)[:, None, None]
    import torch
    return b, torch.from_numpy(q.reshape(sequences * new, Hq, D).astype(np.float32)).to(torch.bfloat16)


def reference(b, q, sequences):
    """{sequence: (out, tolerance)} in 64 bits, from the codes."""
    new, keys, ref = b.new[0], b.total[0], {}
    k, v = (np.concatenate([oa.values(b.host[n + "_codes"][p], b.host[n + "_scale"][p].astype(int)[:, None, None] - 127)
                            for p in b.table[0, :-(-keys // 64)]], 1)[:, :keys] for n in "kv")        # [heads, keys, D]
    for s in sequences:
        x = f64(q[s * new:(s + 1) * new])
        x = x.reshape(new, 2, -1, D).transpose(1, 2, 0, 3)                                             # [heads, group, new, D]
        z = x @ k.transpose(0, 2, 1)[:, None] * D ** -0.5
        z[..., np.arange(keys)[None] > np.arange(keys - new, keys)[:, None]] = -np.inf
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        rows = lambda y: y.transpose(2, 0, 1, 3).reshape(new, -1, D)
        out, spread = rows(p @ v[:, None]), rows(p @ np.abs(v)[:, None])
        ref[s] = out, 2.0 ** -8 * np.abs(out) + 2.0 ** -7 * spread
    return ref


def off(out, ref, new):
    """The largest error, in units of the tolerance, of the sequences that there is a reference of."""
    out = f64(out).reshape(-1, new, *out.shape[1:])
    assert not np.isnan(out).any()
    return max(float((np.abs(out[s] - r) / np.maximum(tol, 1e-300)).max()) for s, (r, tol) in ref.items() if s < len(out))


def attention(env, b, q, sequences, max_q):  # noqa: F811
    moe, torch = env
    new = b.new[0]
    ws = moe.moe_paged_attention_workspace(sequences * new, sequences, q.shape[1], 2, D, max_q)
    out = moe.moe_paged_attention(q[:sequences * new].cuda(), b.cache, b.d_start[:sequences + 1], b.d_len[:sequences],
                                  b.d_table[:sequences], max_q=max_q, ws=ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    return out


@pytest.mark.parametrize("keys", [1000, 8000, 40000])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("Hq,new", [(4, 1), (32, 1), (16, 2)])
def test_small_weights_beside_a_dominant_key(env, keys, place, Hq, new):  # noqa: F811
    """By the kernel of few rows, over rows that are split into short runs and rows that a block has to itself, and by the one
    of many rows."""
    rng = np.random.default_rng(keys + 7 * Hq + len(place))
    b, q = dominated(rng, keys, place, new, Hq, 300)
    b.dev(env)
    ref = reference(b, q, (0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 151, 297))
    for sequences, max_q in ((10, new), (300, new), (10, 10), (300, 40)):    # 10 rows of 2 heads: the kernel of many rows
        assert off(attention(env, b, q, sequences, max_q), ref, new) <= 1.0, (sequences, max_q)


def test_pages_of_far_apart_values_beside_a_dominant_key(env):  # noqa: F811
    """The same where the dominant key's page has values 2^6 times larger, or smaller."""
    rng = np.random.default_rng(5)
    for up in (6, -6):
        b, q = dominated(rng, 4000, "middle", 1, 8, 300)
        b.host["v_scale"][b.table[0, 2003 // 64]] += np.uint8(up % 256)
        b.dev(env)
        ref = reference(b, q, range(10))
        for sequences, max_q in ((10, 1), (300, 1), (10, 10), (300, 40)):
            assert off(attention(env, b, q, sequences, max_q), ref, 1) <= 1.0, (up, sequences, max_q)


@pytest.mark.parametrize("large", ["first", "last"])
def test_zeros_beside_large_values(env, large):  # noqa: F811
    """A page of values up to 2^44 among pages of zeros, whose scale is 2^-64, all keys' scores being much the same: the keys of the zeros
    take their share of the denominator although their terms of the sum are 2^100 times smaller than the others'."""
    rng = np.random.default_rng(7)
    for new, Hq, limits in ((1, 4, (1, 20)), (2, 16, (2, 20)), (140, 4, (140,))):
        b, q = dominated(rng, 1000, "middle", new, Hq, 20)
        q[..., 0] = 0.0
        n = -(-1000 // 64)
        p = b.table[0, 0 if large == "first" else n - 2]
        rest = [x for x in b.table[0, :n] if x != p]
        b.host["v_codes"][rest], b.host["v_scale"][rest], b.host["v_scale"][p] = 0, 63, 127 + 36
        b.dev(env)
        ref = reference(b, q, range(4))
        for max_q in limits:
            assert off(attention(env, b, q, 20, max_q), ref, new) <= 1.0, (new, Hq, max_q)
