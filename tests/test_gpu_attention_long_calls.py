"""Calls of the long conversations' operators that their documentation allows and that differ from the usual ones in the kind of their
arguments (GPU).  Tolerances as in test_gpu_attention_long."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import env  # noqa: E402,F401
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
