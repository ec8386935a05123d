"""moe_rope_table against the oracle's angles in 64 bits (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from oracle import attention as oa  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    from moe_expert_layer_fwd_gb300 import build
    build.build()
    import moe_expert_layer_fwd_gb300 as m
    return m


def close(got, pos, rot, base):
    """A cosine or sine of an angle x: one rounding to fp32 (2^-24) and the angle's own error in double, a few 2^-53 of x."""
    angle = pos[:, None].astype(np.longdouble) * np.array(
        [np.longdouble(base) ** (np.longdouble(-2 * i) / rot) for i in range(rot // 2)])[None]
    ref = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float64)
    tol = 2.0 ** -24 * np.abs(ref) + np.concatenate([angle, angle], 1).astype(np.float64) * 2.0 ** -50 + 2.0 ** -40
    return (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("rot", [16, 32, 64, 96, 128])
@pytest.mark.parametrize("base", [1e4, 1e6, 500.0])
def test_table(moe, rot, base):
    got = moe.moe_rope_table(300, rot, base).double().cpu().numpy()
    assert got.shape == (300, rot)
    assert np.abs(got - oa.rope_table(300, rot, base)).max() <= 2.0 ** -24 + 2.0 ** -40
    assert close(got, np.arange(300), rot, base)


@pytest.mark.parametrize("rot,base", [(128, 1e6), (64, 1e4)])
def test_far_positions(moe, rot, base):
    """Far out the angle has lost most of fp32's bits; the table has not."""
    n = 1 << 20
    import torch
    t = moe.moe_rope_table(n, rot, base)
    pos = np.unique(np.r_[0:9, 99_990:100_010, 131_072, 500_001, n - 9:n])
    assert close(t[torch.from_numpy(pos).cuda()].double().cpu().numpy(), pos, rot, base)


def test_one_row_and_a_given_table(moe):
    import torch
    t = torch.full((3, 32), 9.0, device="cuda")
    assert moe.moe_rope_table(3, 32, 1e4, cos_sin=t) is t
    assert np.abs(t.double().cpu().numpy() - oa.rope_table(3, 32, 1e4)).max() <= 2.0 ** -24 + 2.0 ** -40
    one = moe.moe_rope_table(1, 128)
    assert (one[0, :64] == 1).all() and (one[0, 64:] == 0).all()
