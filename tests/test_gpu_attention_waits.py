"""Waits that run out in the attention kernels (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import Batch, attend, bf16, check, env  # noqa: E402,F401


@pytest.mark.parametrize("new,Hq", [(1, 8), (1, 32), (2, 16), (20, 8)])
def test_waits_that_run_out_end_the_kernel(env, new, Hq):  # noqa: F811
    """The values' copies are withheld: the limit runs out for some warps of a block while others are on their way to the
    same barriers, in tiles with masked keys (whose values the softmax warps wait for themselves) and without, in rows that are
    split over blocks and rows that are not.  Each call ends and reports it; the next ones on the same context are correct.
    (The limit stays far above what a copy takes: those in flight are waited for with it, too.)"""
    moe, torch = env
    rng = np.random.default_rng(71 + new + Hq)
    L = moe.lib()
    for ctx in ([700, 90, 2048 - new], [640 - new] * 3, [5000, 1, 64], [300, 129, 2]):
        b = Batch(rng, [new] * 3, ctx, 2, 32).fill(rng).dev(env)
        q = bf16(rng, 3 * new, Hq, 128)
        try:
            assert L.moe_debug_set(4, 1) == moe.MOE_OK
            for limit_ms in (2, 3, 5):
                for causal in (True, False):
                    assert L.moe_debug_set(1, limit_ms * 1000000) == moe.MOE_OK
                    attend(env, b, q, status=moe.MOE_ERR_TIMEOUT, causal=causal)
        finally:
            L.moe_debug_set(4, 0)
            L.moe_debug_set(1, 0)
        check(env, b, q)
