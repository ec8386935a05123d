"""The attention oracle against hand-worked values, torch's float8 type and closed forms (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as oa


def test_scale_exponent_is_the_smallest_power_that_fits():
    for amax, e in [(0.0, -64), (448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.76, -7), (1e-30, -64), (3e38, 120)]:
        assert oa.scale_exponent(amax) == e
    for amax in np.random.default_rng(0).lognormal(0, 20, 200):
        e = oa.scale_exponent(amax)
        assert amax <= 448 * 2.0 ** e and (e == -64 or amax > 448 * 2.0 ** (e - 1))


def test_codes_are_those_of_float8_e4m3fn():
    x = np.random.default_rng(1).normal(0, 60, 4000).clip(-448, 448).astype(np.float32)
    x[:16] = 2.0 ** -np.arange(16)
    ours = oa.quantise(x, 0)
    theirs = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ours == theirs).all()
    assert np.allclose(oa.values(ours, 3), torch.from_numpy(theirs).view(torch.float8_e4m3fn).float().numpy() * 8)


def test_rotation_by_hand():
    x = np.zeros((1, 1, 32))
    x[0, 0, 0], x[0, 0, 8], x[0, 0, 20] = 3.0, 4.0, 7.0
    table = oa.rope_table(5, 16, 100.0)
    y = oa.norm_rotate(x, np.array([2]), table, 16, False)
    assert y[0, 0, 0] == pytest.approx(3 * math.cos(2) - 4 * math.sin(2))
    assert y[0, 0, 8] == pytest.approx(3 * math.sin(2) + 4 * math.cos(2))
    assert y[0, 0, 20] == 7.0
    z = oa.norm_rotate(x, np.array([3]), table, 16, True)   # pair (8, 9) is pair 4: angle 3 * 100^(-8/16) = 0.3
    assert z[0, 0, 8] == pytest.approx(4 * math.cos(0.3)) and z[0, 0, 9] == pytest.approx(4 * math.sin(0.3))


def _cache(n, Hkv, page, D):
    return dict(k_codes=np.zeros((n, Hkv, page, D), np.uint8), v_codes=np.zeros((n, Hkv, page, D), np.uint8),
                k_scale=np.zeros((n, Hkv), np.uint8), v_scale=np.zeros((n, Hkv), np.uint8))


def test_append_in_pieces_equals_append_at_once_when_the_scale_is_known():
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(40, 2, 32)), rng.normal(size=(40, 2, 32))
    k[[0, 16, 32]] *= 8                      # the first token of a page has its largest values: the scale never grows
    v[[0, 16, 32]] *= 8
    table = np.array([[2, 0, 1]])
    whole, parts = _cache(3, 2, 16, 32), _cache(3, 2, 16, 32)
    oa.append(k, v, whole, [0, 40], [40], table)
    at = 0
    for n in (1, 15, 7, 17):
        oa.append(k[at:at + n], v[at:at + n], parts, [0, n], [at + n], table)
        at += n
    assert all((whole[x] == parts[x]).all() for x in whole)


def test_growing_scale_rounds_earlier_codes_again():
    c = _cache(1, 1, 16, 16)
    one = np.full((1, 1, 16), 1.0)
    oa.append(one, one, c, [0, 1], [1], np.array([[0]]))
    assert c["k_scale"][0, 0] == 127 - 8     # 1 <= 448 * 2^-8 = 1.75
    oa.append(one * 100, one * 100, c, [0, 1], [2], np.array([[0]]))
    assert c["k_scale"][0, 0] == 127 - 2     # 100 <= 448 / 4 = 112
    assert (oa.read(c, "k", 0, 0, 1, np.array([[0]])) == 1.0).all()
    assert np.abs(oa.read(c, "k", 0, 1, 2, np.array([[0]])) - 100).max() <= 100 * 2.0 ** -4


def test_attention_matches_torch_in_float64():
    rng = np.random.default_rng(3)
    c = _cache(4, 2, 16, 32)
    n, total = 5, 40
    table = np.array([[3, 1, 2]])
    oa.append(rng.normal(size=(total, 2, 32)), rng.normal(size=(total, 2, 32)), c, [0, total], [total], table)
    q = rng.normal(size=(n, 4, 32))
    out, _ = oa.attention(q, c, [0, n], [total], table, 0.3)
    k = torch.from_numpy(oa.read(c, "k", 0, 0, total, table)).repeat_interleave(2, 1).transpose(0, 1)
    v = torch.from_numpy(oa.read(c, "v", 0, 0, total, table)).repeat_interleave(2, 1).transpose(0, 1)
    mask = torch.arange(total)[None] <= torch.arange(total - n, total)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).transpose(0, 1)[None], k[None], v[None],
                                                           attn_mask=mask, scale=0.3)[0].transpose(0, 1)
    assert np.abs(out - ref.numpy()).max() < 1e-12


def test_rows_that_see_nothing_are_zero():
    c = _cache(1, 1, 16, 16)
    out, _ = oa.attention(np.ones((2, 1, 16)), c, [0, 2], [0], np.array([[0]]), 1.0)
    assert (out == 0).all()
