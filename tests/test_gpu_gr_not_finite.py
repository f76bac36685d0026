"""States and adjoints that are not finite stay so until a document begins, however long the text and
however small the decays' product: float32 products of decays reach 0 after a few hundred tokens, which
is not the same as a document's beginning.
"""
import numpy as np
import pytest

from tests.gpu_util import note
from tests.test_gpu_gr import make

pytestmark = pytest.mark.gpu

LAM = [-4.0, -1.0, 0.0, 1.0, 2.0, 3.0]          # decays of a token from 0.93 down to 1e-8 and less


def inputs(T, dt, B=2, D=130):
    import torch
    p = make(T, B, T, D, dt)
    p["lam"] = torch.tensor(LAM, device="cuda").repeat(-(-D // len(LAM)))[:D].contiguous()
    return p


def kept(y, bad, what):
    """Whether every value along axis 1 is what a state of `bad` gives: NaN, or the infinity."""
    import torch
    ok = torch.isnan(y) if np.isnan(bad) else y.float() == bad
    assert ok.all(), (what, bad, int((~ok).sum()), ok.numel())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [1, 30, 128, 129, 700, 5000])
def test_a_state_that_is_not_finite(gpu, T, bad, dt):
    """From h0 on, and from a token on, in whole texts; the same in two calls and token after token."""
    import torch
    note(f"gr not finite {T} {bad} {dt}")
    p = inputs(T, dt)
    clean = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"])
    h0 = p["h0"].clone()
    h0[1, ::2] = bad
    y, hf, ck = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], h0, return_final=True, return_ckpt=True)
    for t in (y[1, :, ::2], hf[1, ::2], ck[1, :, ::2]):
        kept(t, bad, "h0")
    assert torch.equal(y[0], clean[0]) and torch.equal(y[1, :, 1::2], clean[1, :, 1::2])
    # the same text in calls of other lengths, which take other ways through it
    cut = T // 3
    if cut:
        a = [p[n] for n in ("x", "r", "i")]
        _, h = gpu.ss_gr_fwd(*[t[:, :cut] for t in a], p["lam"], h0, return_final=True)
        gpu.ss_gr_step(*[t[:, cut] for t in a], p["lam"], h)
        y2, h = gpu.ss_gr_fwd(*[t[:, cut + 1:] for t in a], p["lam"], h, return_final=True)
        kept(y2[1, :, ::2], bad, "calls")
        kept(h[1, ::2], bad, "calls")
    # a token of the text brings it in
    at = T // 2
    x = p["x"].clone()
    x[0, at, 3::5] = bad
    y, hf = gpu.ss_gr_fwd(x, p["r"], p["i"], p["lam"], p["h0"], return_final=True)
    assert torch.equal(y[0, :at], clean[0, :at]) and torch.equal(y[1], clean[1])
    kept(y[0, at:, 3::5], bad, "x")
    kept(hf[0, 3::5], bad, "x")


@pytest.mark.parametrize("marks", ["none", "length", "document"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [30, 65, 600, 2100])
def test_an_adjoint_that_is_not_finite(gpu, T, bad, marks):
    """From dh_final on, and from a token's dy on, back to the text's beginning or the document's."""
    import torch
    note(f"gr adjoint not finite {T} {bad} {marks}")
    p = inputs(T, "f32")
    first, n = 0, T
    kw = {}
    if marks == "length":
        n = T - 3
        kw["lengths"] = torch.full((2,), n, dtype=torch.int32, device="cuda")
    if marks == "document":
        first = T // 4
        kw["reset"] = torch.zeros(2, T, dtype=torch.bool, device="cuda")
        kw["reset"][:, first] = True
    args = (p["x"], p["r"], p["i"], p["lam"])
    clean = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], p["dh"], **kw)
    dh = p["dh"].clone()
    dh[1, ::2] = bad
    g = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], dh, **kw)
    kept(g["dx"][1, first:n, ::2], bad, "dh_final")
    if marks != "document":
        kept(g["dh0"][1, ::2], bad, "dh_final")
    at = 3 * T // 4
    dy = p["dy"].clone()
    dy[0, at, 3::5] = bad
    q = gpu.ss_gr_bwd(*args, dy, p["h0"], p["dh"], **kw)
    kept(q["dx"][0, first:at + 1, 3::5], bad, "dy")
    assert not torch.isfinite(q["dr"][0, first + 1:at, 3::5]).any()
    for name in ("dx", "dr", "di"):
        for a, row in ((g, 0), (q, 1)):
            assert torch.equal(a[name][row], clean[name][row]), name
        assert torch.equal(q[name][0, at + 1:], clean[name][0, at + 1:]), name
        assert torch.equal(g[name][1, :first], clean[name][1, :first]), name
    if marks == "document":
        assert torch.equal(g["dh0"], clean["dh0"]) and torch.equal(q["dh0"], clean["dh0"])


def test_decays_that_vanish_leave_no_trace(gpu):
    """Finite states: what has decayed below float32 is nothing, as before."""
    import torch
    p = inputs(3000, "f32")
    p["h0"][:] = 3e38
    y = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"])
    z = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], torch.zeros_like(p["h0"]))
    fast = p["lam"] >= 1.0
    assert torch.isfinite(y).all() and torch.equal(y[:, 1500:, fast], z[:, 1500:, fast])
