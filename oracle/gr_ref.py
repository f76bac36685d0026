"""Gated linear recurrence in float64: token after token, and its adjoint.

Test infrastructure only: nothing in the package imports this, and it shares no code with the
library.  The definitions are include/ss.h's.
"""
import numpy as np


def gates(x, r, i, lam, c, lengths=None, reset=None):
    """a, s = sqrt(1 - a^2), v = sigma(i) x, the gates, log a; live and first as [B, T] truth values."""
    B, T, D = x.shape
    live = np.ones((B, T), bool)
    if lengths is not None:
        for b, n in enumerate(lengths):
            live[b, max(0, int(n)):] = False
    first = np.zeros((B, T), bool) if reset is None else np.asarray(reset) != 0
    x, r, i = (np.where(live[..., None], t, 0.0) for t in (x, r, i))
    sr, si = 1.0 / (1.0 + np.exp(-r)), 1.0 / (1.0 + np.exp(-i))
    la = -c * np.logaddexp(0.0, lam) * sr
    a, s = np.exp(la), np.sqrt(-np.expm1(2.0 * la))
    a[first], s[first] = 0.0, 1.0
    a[~live], s[~live] = 1.0, 0.0
    return a, s, si * x, sr, si, la, x, live, first


def fwd(x, r, i, lam, h0=None, c=8.0, lengths=None, reset=None):
    """y [B, T, D] and the states [B, T + 1, D], the first before any token."""
    a, s, v, *_, live, first = gates(x, r, i, lam, c, lengths, reset)
    B, T, D = x.shape
    h = np.zeros((B, T + 1, D))
    if h0 is not None:
        h[:, 0] = h0
    for t in range(T):
        old = np.where(first[:, t, None] & live[:, t, None], 0.0, h[:, t])
        h[:, t + 1] = a[:, t] * old + s[:, t] * v[:, t]
    return np.where(live[..., None], h[:, 1:], 0.0), h


def bwd(x, r, i, lam, dy, h0=None, dh_final=None, c=8.0, lengths=None, reset=None):
    a, s, v, sr, si, la, x, live, first = gates(x, r, i, lam, c, lengths, reset)
    _, h = fwd(x, r, i, lam, h0, c, lengths, reset)
    B, T, D = x.shape
    g = np.zeros((B, D)) if dh_final is None else dh_final.astype(np.float64).copy()
    dx, dr, di, dlam = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape), np.zeros(D)
    for t in reversed(range(T)):
        on, cut = live[:, t, None], first[:, t, None]
        g = g + np.where(on, dy[:, t], 0.0)
        dv = g * s[:, t]
        dx[:, t] = np.where(on, dv * si[:, t], 0.0)
        di[:, t] = np.where(on, dv * x[:, t] * si[:, t] * (1 - si[:, t]), 0.0)
        with np.errstate(divide="ignore", invalid="ignore"):
            root = np.where(s[:, t] > 1e-15, a[:, t] ** 2 / s[:, t], 0.0)
        dla = np.where(on & ~cut, g * (a[:, t] * h[:, t] - root * v[:, t]), 0.0)
        dr[:, t] = dla * la[:, t] * (1 - sr[:, t])
        dlam += (dla * sr[:, t]).sum(0) * -c / (1.0 + np.exp(-lam))
        g = np.where(on & cut, 0.0, a[:, t] * g)
    return {"dx": dx, "dr": dr, "di": di, "dlam": dlam, "dh0": g if h0 is not None else None}
