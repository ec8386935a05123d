"""What the attention operators leave out, and what they say about it: positions beyond the table of angles, pages that are not in
the pool, starts and lengths that do not fit together (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import D, Batch, bf16, env, f64  # noqa: E402,F401
from oracle import attention as oa  # noqa: E402


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
