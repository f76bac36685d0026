"""Pins of oracle/norm_q4_ref.py, CPU only: closed forms, and the norm's gradients against central
differences of its forward in float64."""
import numpy as np

from oracle import norm_q4_ref as ref


def test_norm_of_equal_elements():
    # every element c: y = c / |c| · w without eps
    y, r = ref.rms_fwd(np.full((2, 8), -3.0), np.arange(8.0), np.full((2, 8), 1.0), 0.0)
    np.testing.assert_allclose(y, np.broadcast_to(-np.arange(8.0), (2, 8)), rtol=1e-15)
    assert (r == -2).all()


def test_norm_gradient():
    r = np.random.default_rng(1)
    x, w, dy, dr = (r.normal(size=s) for s in ((3, 11), 11, (3, 11), (3, 11)))

    def loss():
        y, s = ref.rms_fwd(x, w, None, 1e-3)
        return (y * dy).sum() + (s * dr).sum()
    dx, dw = ref.rms_bwd(dy, x, w, dr, 1e-3)
    for a, g in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + 1e-5
            up = loss()
            a[i] = keep - 1e-5
            down = loss()
            a[i] = keep
            assert abs((up - down) / 2e-5 - g[i]) < 1e-7


def test_codes_in_their_places():
    wq = np.array([[0x10, 0x32], [0xfe, 0xdc]], np.uint8)
    s = np.array([[2.0, 0.5], [1.0, 4.0]])
    z = np.array([[1, 0], [15, 2]], np.uint8)
    want = np.array([[(0 - 1) * 2, (1 - 1) * 2, 2 * 0.5, 3 * 0.5], [14 - 15, 0, (12 - 2) * 4, (13 - 2) * 4]])
    np.testing.assert_array_equal(ref.q4_weights(wq, s, z, 2), want)
    np.testing.assert_array_equal(ref.q4_weights(wq, s, None, 2)[0], [-16, -14, -3, -2.5])
    np.testing.assert_array_equal(ref.q4_mv(np.ones((1, 4)), wq, s, z, 2, np.array([3.0])), [3 * want.sum(1)])
