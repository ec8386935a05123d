"""Calls of the long conversations' operators that their documentation allows and that differ from the usual ones in the kind of their
arguments (GPU).  Tolerances as in test_gpu_attention_long."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import D, env  # noqa: E402,F401
from test_gpu_attention_long import i32  # noqa: E402


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
