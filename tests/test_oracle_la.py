"""Pins of the linear-attention oracle (oracle/la_ref.py), CPU only.

The forward against the closed double sum, the gradients against central differences of the
forward in float64, the resume identity, and the meaning of a -inf decay and of lengths.
"""
import numpy as np
import pytest

from oracle import la_ref


def _case(seed, B=2, T=7, H=4, Hk=2, dk=3, dv=5, decay="token", s0=True):
    r = np.random.default_rng(seed)
    q, k = r.normal(size=(2, B, T, Hk, dk))
    v = r.normal(size=(B, T, H, dv))
    g = {"token": -r.uniform(0, 2, size=(B, T, H)), "head": -r.uniform(0, 2, size=H),
         "none": None}[decay]
    return q, k, v, g, r.normal(size=(B, H, dk, dv)) if s0 else None


def test_forward_is_the_double_sum():
    q, k, v, g, s0 = _case(1)
    o, s = la_ref.fwd(q, k, v, g, s0, 0.7)
    B, T, H, dv = v.shape
    for b in range(B):
        for h in range(H):
            u = h // 2
            for t in range(T):
                want = np.exp(g[b, :t + 1, h].sum()) * (q[b, t, u] @ s0[b, h])
                for i in range(t + 1):
                    want = want + np.exp(g[b, i + 1:t + 1, h].sum()) * (q[b, t, u] @ k[b, i, u]) * v[b, i, h]
                # float64 sums of at most 8 terms: 1e-12 is far above their rounding
                np.testing.assert_allclose(o[b, t, h], 0.7 * want, rtol=1e-12, atol=1e-12)


def test_resume():
    q, k, v, g, s0 = _case(2)
    o, s = la_ref.fwd(q, k, v, g, s0)
    o1, s1 = la_ref.fwd(q[:, :3], k[:, :3], v[:, :3], g[:, :3], s0)
    o2, s2 = la_ref.fwd(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:], s1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(s2, s, rtol=1e-13, atol=1e-13)


def test_infinite_decay_cuts():
    q, k, v, g, s0 = _case(3)
    g[:, 4] = -np.inf
    o, s = la_ref.fwd(q, k, v, g, s0)
    o2, s2 = la_ref.fwd(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], None)
    np.testing.assert_allclose(o[:, 4:], o2, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(s, s2, rtol=1e-13, atol=1e-13)


def test_lengths_hide_what_is_behind():
    q, k, v, g, s0 = _case(4)
    n = np.array([0, 5])
    o, s = la_ref.fwd(q, k, v, g, s0, lengths=n)
    q[0], v[1, 5:], g[1, 6] = np.nan, np.inf, np.nan
    o2, s2 = la_ref.fwd(q, k, v, g, s0, lengths=n)
    np.testing.assert_array_equal(o, o2)
    np.testing.assert_array_equal(s, s2)
    np.testing.assert_array_equal(s[0], s0[0])
    assert not o[0].any() and not o[1, 5:].any()


@pytest.mark.parametrize("lengths", [None, [7, 4], [0, 1]])
@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("s0", [True, False])
def test_gradients_are_the_differences(decay, s0, lengths):
    q, k, v, g, s = _case(5, decay=decay, s0=s0)
    r = np.random.default_rng(6)
    do = r.normal(size=v.shape)
    ds = r.normal(size=(2, 4, 3, 5))
    ins = dict(dq=q, dk=k, dv=v, dg=g, ds0=s)
    n = None if lengths is None else np.array(lengths)

    def loss():
        o, sf = la_ref.fwd(q, k, v, g, s, 0.6, n)
        return (o * do).sum() + (sf * ds).sum()
    got = la_ref.bwd(q, k, v, do, g, s, ds, 0.6, n)
    eps = 1e-5
    for name, x in ins.items():
        if x is None:
            assert got[name] is None
            continue
        assert got[name].shape == x.shape
        for i in r.choice(x.size, min(x.size, 12), replace=False):
            at = np.unravel_index(i, x.shape)
            keep = x[at]
            x[at] = keep + eps
            up = loss()
            x[at] = keep - eps
            down = loss()
            x[at] = keep
            # central differences: truncation eps² and rounding 1e-16·|loss|/eps are below 1e-8
            assert abs((up - down) / (2 * eps) - got[name][at]) < 1e-7, (name, at)
