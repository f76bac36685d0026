"""The float64 oracles of the gated recurrence, the layer norm and the 4-bit values against
differences, sums and hand-worked values."""
import numpy as np
import pytest

from oracle import gr_ref, ln_mx4_ref as ref


def differences(loss, arrays, grads, step, tol):
    for a, g in zip(arrays, grads):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + step
            up = loss()
            a[i] = keep - step
            down = loss()
            a[i] = keep
            assert abs((up - down) / (2 * step) - g[i]) < tol, (i, (up - down) / (2 * step), g[i])


@pytest.mark.parametrize("marks", ["none", "lengths", "reset", "both"])
def test_recurrence_gradients_are_differences(marks):
    r0 = np.random.default_rng(1)
    B, T, D = 2, 6, 3
    x, r, i, dy = (r0.normal(size=(B, T, D)) for _ in range(4))
    lam, h0, dh = r0.normal(size=D), r0.normal(size=(B, D)), r0.normal(size=(B, D))
    kw = {}
    if marks in ("lengths", "both"):
        kw["lengths"] = [4, 0]
    if marks in ("reset", "both"):
        kw["reset"] = r0.random((B, T)) < 0.4
    g = gr_ref.bwd(x, r, i, lam, dy, h0, dh, 2.0, **kw)

    def loss():
        y, h = gr_ref.fwd(x, r, i, lam, h0, 2.0, **kw)
        return (y * dy).sum() + (h[:, -1] * dh).sum()
    differences(loss, (x, r, i, lam, h0), [g[n] for n in ("dx", "dr", "di", "dlam", "dh0")], 1e-5, 1e-7)


def test_recurrence_by_hand():
    """lam with c softplus(lam) = 2 ln 2 and r = 0: a = 1/2, s = sqrt(3)/2; i = 0 halves x."""
    lam = np.log(np.expm1(np.array([2 * np.log(2.0) / 8])))
    x = np.array([2.0, 4.0, 0.0]).reshape(1, 3, 1)
    z = np.zeros_like(x)
    y, h = gr_ref.fwd(x, z, z, lam, np.array([[8.0]]))
    s = np.sqrt(3) / 2
    np.testing.assert_allclose(y[0, :, 0], [4 + s, 2 + s / 2 + 2 * s, 1 + s / 4 + s], rtol=1e-14)
    y, h = gr_ref.fwd(x, z, z, lam, np.array([[8.0]]), reset=np.array([[0, 1, 0]]))
    np.testing.assert_allclose(y[0, :, 0], [4 + s, 2.0, 1.0], rtol=1e-14)


def test_layer_norm():
    r0 = np.random.default_rng(2)
    x, res, dy, dr = (r0.normal(size=(3, 7)) for _ in range(4))
    w, b = r0.normal(size=7), r0.normal(size=7)
    y, r = ref.ln_fwd(x, w, b, res, 1e-3)
    n = (y - b) / w
    assert abs(n.mean(-1)).max() < 1e-14
    dx, dw, db = ref.ln_bwd(dy, r, w, dr, 1e-3)

    def loss():
        y, r = ref.ln_fwd(x, w, b, res, 1e-3)
        return (y * dy).sum() + (r * dr).sum()
    differences(loss, (x, res, w, b), (dx, dx, dw, db), 1e-5, 1e-7)


def test_four_bit_values():
    """Every half step between two codes and its neighbours, in blocks whose largest value is 6 or
    7.5 times the power of two."""
    x = np.zeros((1, 32))
    x[0, :14] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -0.75, -0.25, 0.2500001, 4.999]
    code, e = ref.mx4_quant(x)
    assert e[0, 0] == 127                       # 4 <= 6 < 8
    want = [6, 4, 4, 2, 2, 1, 1, 0, -4, -4, -1, 0, 0.5, 4]
    assert ref.mx4_values(code, e)[0, :14].tolist() == want
    code, e = ref.mx4_quant(x * 1.25)           # 7.5 stays in the same block: past 6 to 6
    assert e[0, 0] == 127 and ref.mx4_values(code, e)[0, 0] == 6
    code, e = ref.mx4_quant(x * 2.0 ** -140)    # the smallest exponent
    assert e[0, 0] == 1 and not ref.mx4_values(code, e)[0].any()
    x[0, 31] = np.inf
    code, e = ref.mx4_quant(x)
    assert e[0, 0] == 255 and np.isnan(ref.mx4_values(code, e)).all()
    c = np.arange(16)
    assert (ref.unpack(ref.pack(c)) == c).all()
