"""Arguments of the long conversations' binding that are converted or checked on the host (CPU)."""
import array

import numpy as np
import pytest
import torch

from moe_expert_layer_fwd_gb300 import attention

AXES = [f % 3 for f in range(64)]


@pytest.mark.parametrize("make", [list, tuple, bytes, bytearray, lambda a: memoryview(bytes(a)), lambda a: array.array("i", a), torch.tensor,
                                  *(lambda a, t=t: np.array(a, t) for t in (np.uint8, np.int8, np.int32, np.int64, np.uint16)),
                                  lambda a: np.array(a, np.int32)[::-1][::-1], lambda a: np.repeat(np.array(a), 2)[::2]])
def test_axes_of_any_kind_of_sequence(make):
    """One byte a frequency, whatever holds the numbers (an array's own bytes are not its elements)."""
    assert attention._axis_bytes(make(AXES), 3, 128) == bytes(AXES)


@pytest.mark.parametrize("axes", [AXES[:-1], AXES + [0], [3] + AXES[1:], [-1] + AXES[1:], [300] + AXES[1:], np.array(AXES) + 1,
                                  np.array(AXES).reshape(32, 2), np.array(AXES) - 1, [0.0] + AXES[1:], np.array(AXES, float)])
def test_axes_that_are_none(axes):
    with pytest.raises((ValueError, TypeError)):
        attention._axis_bytes(axes, 3, 128)


def test_axes_of_no_frequency():
    assert attention._axis_bytes([], 1, 0) == b""


def test_layer_numbers():
    """Scales that are none in fp32, and windows below zero, are refused when the layer is made."""
    import moe_expert_layer_fwd_gb300 as moe
    for kw in (dict(window=-1), dict(window=-1 << 32), dict(scale=1e-60), dict(scale=1e60), dict(scale=0.0),
               dict(scale=float("nan"))):
        with pytest.raises(ValueError, match="window"):
            moe.AttentionLayer(4, 8, 2, device="cpu", **kw)


def test_prefix_tables_without_columns():
    """NULL for a table that has no columns, not for one that has; what comes behind that check still refuses."""
    from test_attention_abi import A, BAD
    from test_attention_long_abi import prefix, shared
    import moe_expert_layer_fwd_gb300 as moe
    L = moe.lib()
    empty = prefix(max_pages=0, page_table=None)
    assert shared(L, p=empty, n=256) == moe.MOE_ERR_WORKSPACE and shared(L, p=empty, out=None) == BAD
    assert shared(L, p=prefix(page_table=None)) == BAD and shared(L, p=prefix(max_pages=0, page_table=A + 4)) == BAD
    assert shared(L, p=empty, table=None) == BAD


def test_counts_beyond_an_int():
    """All tokens, not the low bits; negative ones stay negative and are refused."""
    assert [attention._count(n) for n in (0, 5, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 5)] == [0, 5] + [(1 << 31) - 1] * 4
    assert attention._count(-1) == attention._count(-1 << 40) == -1


@pytest.mark.parametrize("new,Hq,Hkv,joined", [
    ([1] * 63 + [1100], 64, 8, False), ([1] * 63 + [4000], 64, 8, False), ([1] * 15 + [1100], 64, 8, False), ([1, 4000], 64, 8, True),
    ([1] * 15 + [4000], 32, 4, True), ([17] * 16, 32, 4, True), ([16] * 16, 32, 4, False), ([200] * 8 + [1] * 16, 32, 4, True),
    ([200] * 8 + [1] * 40, 32, 4, False), ([20, 250, 100, 180], 32, 4, True), ([129], 1, 1, True), ([128], 1, 1, False), ([1] * 64, 64, 8, False)])
def test_batches_of_long_and_short_sequences_share_their_prefix(new, Hq, Hkv, joined):
    """Decoding sequences beside a chunk of tokens keep the reading that all share, which needs room for its rows; batches of much the same
    lengths go over their prefixes by themselves."""
    import ctypes
    import moe_expert_layer_fwd_gb300 as moe
    L, T = moe.lib(), sum(new)
    d = moe.moe_kv_desc(len(new), T, Hq, Hkv, 128, 64, 1000, 100)
    size = lambda p: L.moe_paged_attention_shared_workspace_size(ctypes.byref(d), max(new), p)
    alone, behind = size(None), size(ctypes.byref(moe.moe_kv_prefix(1, 200, T, None, None, None)))
    assert behind == alone if joined else behind >= alone + 2 * T * Hq * 129 * 4
