"""The oracle of the long conversations' operators against closed forms and brute force (CPU)."""
import numpy as np
import pytest

from oracle import attention as oa
from oracle import attention_long as ol

D = 128


def cache_of(rng, lengths, Hkv=2, page=16):
    used = [-(-n // page) for n in lengths]
    n, ids = sum(used) + 1, rng.permutation(sum(used) + 1)
    table = np.full((len(lengths), max(used + [1])), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    cache = {x: np.zeros((n, Hkv, page, D), np.uint8) for x in ("k_codes", "v_codes")}
    cache.update({x: np.full((n, Hkv), 63, np.uint8) for x in ("k_scale", "v_scale")})
    oa.append(rng.normal(size=(sum(lengths), Hkv, D)), rng.normal(size=(sum(lengths), Hkv, D)), cache,
              np.cumsum([0] + list(lengths)), lengths, table)
    return cache, table


def test_rows_of_one_axis_are_rows_of_the_table():
    table = oa.rope_table(40, 32, 1e4)
    pos = np.array([[3, 39, 0, 7], [1, 1, 2, 30]])
    assert np.array_equal(ol.rope_rows(pos[:1], [0] * 16, table), table[pos[0]])
    rows = ol.rope_rows(pos, [0] * 4 + [1] * 12, table)
    assert np.allclose(rows[1, 3], np.cos(39 * 1e4 ** (-6 / 32))) and np.allclose(rows[1, 16 + 4], np.sin(1e4 ** (-8 / 32)))


@pytest.mark.parametrize("cut", [0, 16, 48, 64])
def test_a_prefix_is_the_first_part_of_a_sequence(cut):
    """Any cut at a page's end gives the whole sequence's attention."""
    rng = np.random.default_rng(cut)
    cache, table = cache_of(rng, [70])
    q, start = rng.normal(size=(3, 4, D)), np.array([0, 3])
    ref, spread = oa.attention(q, cache, start, [70], table, 0.1)
    prefix = (start, [cut], table[:, :cut // 16])
    out, spread2, lse = ol.shared_attention(q, cache, start, [70 - cut], table[:, cut // 16:], 0.1, prefix)
    assert np.allclose(out, ref) and np.allclose(spread, spread2)
    k = oa.read(cache, "k", 0, 0, 70, table)
    assert np.isclose(lse[2, 3], np.log(np.exp(k[:, 1] @ q[2, 3] * 0.1).sum()))
    assert np.isclose(lse[0, 0], np.log(np.exp(k[:68, 0] @ q[0, 0] * 0.1).sum()))


def test_weights_add_up_to_the_rows():
    rng = np.random.default_rng(1)
    cache, table = cache_of(rng, [70, 5])
    q, start, lens = rng.normal(size=(5, 4, D)), np.array([0, 3, 5]), [70, 5]
    for window in (0, 6):
        lse = ol.shared_attention(q, cache, start, lens, table, 0.1, None, True, window)[2]
        old = np.full((cache["k_codes"].shape[0], 2, 16), 10.0)
        out, added, written = ol.weights(q, lse, cache, start, lens, table, 0.1, old, False, True, window)
        assert np.isclose(added[table[0, :5]].sum((0, 2)), 6).all() and np.isclose(added[table[1, 0]].sum(1), 4).all()
        assert (out[~written] == 10).all() and written[table[1, 0], :, :5].all() and not written[table[1, 0], :, 5:].any()
        assert (out[table[0, 4], :, 3:6] < 7).all() and (out[table[0, 4], :, 2] >= 10).all()    # new tokens start at zero
        assert written[table[0, 0]].all() == (window == 0)
    fresh = ol.weights(q, lse, cache, start, lens, table, 0.1, old, True, True, 6)[0]
    assert np.allclose(fresh[written], added[written])


def test_evict_by_hand():
    rng = np.random.default_rng(2)
    cache, table = cache_of(rng, [20, 33])
    weight = np.zeros((cache["k_codes"].shape[0], 2, 16), np.float32)
    weight[table[0, 0], 0, [3, 5, 9]] = 2.0, 7.0, 2.0
    weight[table[0, 1], 1, 1] = np.nan
    weight[table[0, 0], 1, [4, 6]] = 1.0
    before = {x: a.copy() for x, a in cache.items()}
    new = table[1:, :1].copy()
    n, kept = ol.evict(cache, weight, [20], table[:1], [5], new, 1, 2)
    assert n[0] == 5 and kept[0, 0, :6].tolist() == [0, 3, 5, 18, 19, -1] and kept[0, 1, :5].tolist() == [0, 4, 6, 18, 19]
    assert weight[new[0, 0], 0, :5].tolist() == [0, 2, 7, 0, 0]
    top = max(before["k_scale"][table[0, 0], 0], before["k_scale"][table[0, 1], 0])
    assert cache["k_scale"][new[0, 0], 0] == top
    got, want = oa.read(cache, "k", 0, 0, 5, new), oa.read(before, "k", 0, 0, 20, table[:1])
    # rounded at most once more, by half of the smallest step
    assert (np.abs(got[:, 0] - want[[0, 3, 5, 18, 19], 0]) <= 2.0 ** -10 * 2.0 ** (int(top) - 127)).all()
    n, kept = ol.evict(cache, weight, [20], table[:1], [50], table[1:, :2], 0, 0)
    assert n[0] == 20 and kept[0, 0, :20].tolist() == list(range(20))
