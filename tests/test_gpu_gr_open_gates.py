"""Gradients of gates that are almost open or almost shut: dr and di are relative to themselves, not to
what 1 - σ loses beside 1.

One token, in closed form (la = log a, g = dy + dh):
  dr = g·(a h0 - a²/s·v)·la·σ(-r)        di = g·s·x·σ(i)·σ(-i)
Units of u = 2^-24 of the absolute terms, as in test_gpu_gr.py: σ(z) and σ(-z) within (|z| + 8)u, log a
within (|r| + 16)u, a within |la|·that and 2u, s within half of log a's and 16u; twelve for the products.
"""
import numpy as np
import pytest

from tests.gpu_util import note
from tests.test_gpu_gr import U, hold, num

pytestmark = pytest.mark.gpu


def sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 77, 512])
def test_one_token(gpu, D, dt):
    note(f"gr open gates {D} {dt}")
    B, c = 600, 8.0
    r = np.random.default_rng(D)
    p = {n: hold(r.normal(size=(B, 1, D)), dt) for n in ("x", "dy")}
    # gates whose gradients are normal numbers (and 1 - a² above the 1e-30 where the root's slope ends)
    p["r"], p["i"] = (hold(r.uniform(-60, 70, size=(B, 1, D)), dt) for _ in range(2))
    lam = hold(r.uniform(-2, 3, size=D), "f32")
    h0, dh = (hold(r.normal(size=(B, D)), "f32") for _ in range(2))
    got = gpu.ss_gr_bwd(p["x"], p["r"], p["i"], lam, p["dy"], h0, dh)
    x, R, i, dy = (num(p[n])[:, 0] for n in ("x", "r", "i", "dy"))
    g, h = dy + num(dh), num(h0)
    la = -c * np.logaddexp(0.0, num(lam)) * sigmoid(R)
    a, s, v = np.exp(la), np.sqrt(-np.expm1(2 * la)), sigmoid(i) * x
    eg, ela = U, (np.abs(R) + 16) * U
    es = ela / 2 + 16 * U
    ev = (np.abs(i) + 8) * U
    first, second = a * h, a * a / s * v
    err = np.abs(first) * (np.abs(la) * ela + 2 * U) + np.abs(second) * (2 * np.abs(la) * ela + es + ev + 8 * U)
    slope = np.abs(la) * sigmoid(-R)
    dr = g * (first - second) * la * sigmoid(-R)
    terms = np.abs(first) + np.abs(second)
    tol = np.abs(g) * slope * (err + terms * (ela + (np.abs(R) + 8) * U + 12 * U)) + 4 * eg * (np.abs(dy) + np.abs(num(dh))) * slope * terms
    di = g * s * x * sigmoid(i) * sigmoid(-i)
    toli = np.abs(x) * s * sigmoid(i) * sigmoid(-i) * (
        np.abs(g) * (es + 2 * (np.abs(i) + 8) * U + 12 * U) + 4 * eg * (np.abs(dy) + np.abs(num(dh))))
    for name, want, bound in (("dr", dr, tol), ("di", di, toli)):
        y = num(got[name])[:, 0]
        bound = 1.01 * bound + (1.01 * 2.0 ** -8 * np.abs(want) if dt == "bf16" else 0) + 1e-36
        over = (np.abs(y - want) - bound) / np.maximum(np.abs(want), 1e-30)
        w = np.unravel_index(over.argmax(), over.shape)
        assert (over <= 0).all(), (name, float(over[w]), float(R[w]), float(i[w]), float(y[w]), float(want[w]))


@pytest.mark.parametrize("T", [40, 300])
def test_gates_that_are_shut_or_open_for_good(gpu, T):
    """±infinity: the gates are 0 and 1, their gradients 0, nothing is NaN."""
    import torch
    D = 64
    r = np.random.default_rng(T)
    x, dy = (hold(r.normal(size=(1, T, D)), "f32") for _ in range(2))
    gate = torch.full((1, T, D), float("inf"), device="cuda")
    gate[..., ::2] = -float("inf")
    lam = hold(r.normal(size=D), "f32")
    mid = hold(r.normal(size=(1, T, D)), "f32")
    for R, i in ((gate, mid), (mid, gate), (gate, gate)):
        y = gpu.ss_gr_fwd(x, R, i, lam)
        g = gpu.ss_gr_bwd(x, R, i, lam, dy)
        assert torch.isfinite(y).all()
        for n in ("dx", "dr", "di", "dlam"):
            assert torch.isfinite(g[n]).all(), n
        if R is gate:
            assert g["dr"].abs().max() < 1e-36
        if i is gate:
            assert g["di"].abs().max() < 1e-36
