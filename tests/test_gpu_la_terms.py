"""bfloat16 linear attention keeps 16 bits of the scores and of the states where they feed o, dq, dk
and dv: what is left of the error is the result's own rounding.

Bound of each element, A the sum of absolute values as in test_gpu_la.py: two bfloat16 terms hold a
value to 2^-8 of what the first leaves, 2^-16 of it; the float32 sums add units(c); the result's
rounding is at most 2^-8 of the result, not of A.
"""
import numpy as np
import pytest

from oracle import la_ref
from tests import test_gpu_la as la
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

CASES = [  # B, T, H, Hk, dk, dv, decay, s0, lengths
    (1, 64, 2, 2, 64, 64, "none", True, None),
    (2, 333, 4, 2, 64, 128, "token", True, None),
    (1, 1500, 2, 2, 128, 128, "head", True, None),
    (2, 300, 2, 1, 100, 36, "token", True, [300, 170]),
    (1, 129, 1, 1, 256, 256, "token", True, None),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_outputs_are_rounded_once(gpu, case):
    B, T, H, Hk, dk, dv, decay, s0, n = case
    c = la.make(61 + T, B, T, H, Hk, dk, dv, "bf16", decay, s0, n)
    note(f"la terms {case}")
    a = la.absolute(c)
    args = (c["scale"], c["lengths"])
    o, _ = la.run_fwd(gpu, c)
    got = dict(la.run_bwd(gpu, c), o=o)
    want = la_ref.bwd(c["q"], c["k"], c["v"], c["do"], c["g"], c["s0"], c["ds"], *args)
    want["o"], _ = la_ref.fwd(c["q"], c["k"], c["v"], c["g"], c["s0"], *args)
    A = la_ref.bwd(a["q"], a["k"], a["v"], a["do"], c["g"], a["s0"], a["ds"], *args)
    A["o"], _ = la_ref.fwd(a["q"], a["k"], a["v"], c["g"], a["s0"], *args)
    for m in ("o", "dq", "dk", "dv"):
        la.near(got[m], want[m], np.abs(want[m]) * 2.0 ** -8 + A[m] * (2.0 ** -16 + la.units(c)) + 1e-37, m)


def test_an_infinite_state_stays_infinite(gpu):
    """s0 infinite at one place: o is infinite, not NaN, in that column, and the others are as
    they are without it."""
    c = la.make(67, 1, 40, 1, 1, 64, 64, "bf16", "token", True)
    note("la infinite state")
    c["q"] = np.abs(c["q"]) + 1
    c["s0"][0, 0, 3, 5] = np.inf
    c["g"][:] = -0.01
    c2 = dict(c, s0=np.where(np.isinf(c["s0"]), 0, c["s0"]).astype(np.float32))
    clean, _ = la.run_fwd(gpu, c2)
    o, s = la.run_fwd(gpu, c)
    o, clean = o.float().cpu().numpy(), clean.float().cpu().numpy()
    keep = np.arange(64) != 5
    assert np.array_equal(o[..., keep], clean[..., keep])
    assert (o[..., 5] == np.inf).all() and s[0, 0, 3, 5].item() == np.inf
