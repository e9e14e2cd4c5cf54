"""GPU checks of the operators around the recurrence at values and views that the
other suites pass over: decays of exactly one, infinities beside a rotation,
gates far from zero, slices of a longer buffer of positions."""
import numpy as np
import pytest

from test_gpu_around import _down, _nan, _pdn, _up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_normed_gain_slope_at_a_decay_of_one(dtype, T):
    """sqrt(1 - a^2) falls ever steeper towards a = 1, where its derivative by
    log_a is -inf whichever zero log_a is: dlog_a is -inf times the sign of x G."""
    pdn = _pdn()
    rng = np.random.default_rng(400)
    D = 16
    x = rng.choice([-1.0, 2.0], (1, T, D)).astype(np.float32)
    la = np.full((1, T, D), -0.25, np.float32)
    at = T // 2
    la[:, at, ::2], la[:, at, 1::2] = 0.0, -0.0
    sign = rng.choice([-1.0, 1.0], (1, 1, D)).astype(np.float32)
    dh = np.broadcast_to(sign, x.shape).copy()       # every G of a channel has its sign
    xd, lad = _up(x, dtype), _up(la, dtype)
    dx, dla = _nan(x.shape, dtype), _nan(x.shape, dtype)
    pdn.pdn_scan_bwd(xd, lad, _up(dh, dtype), dx, dla, gain=pdn.PDN_GAIN_NORM)
    got = _down(dla)
    np.testing.assert_array_equal(got[:, at], -np.inf * (x * dh)[:, at])
    assert np.isfinite(np.delete(got, at, 1)).all()
    dx = _down(dx)
    assert (dx[:, at] == 0).all() and np.isfinite(dx).all()
    h = _nan(x.shape, dtype)
    pdn.pdn_scan_fwd(xd, lad, h, gain=pdn.PDN_GAIN_NORM)
    h = _down(h)
    np.testing.assert_array_equal(h[:, at], h[:, at - 1] if at else 0 * h[:, 0])
