"""The norm's gradient for rows far from 1 and without an eps to hold them up: rows of zeros, of
1e-17, 1e-14, 1e13 and 1e17.  Bounds of test_gpu_norm.py."""
import numpy as np
import pytest

from oracle import norm_q4_ref as ref
from tests import test_gpu_norm as norm
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [40, 513, 2560, 9000])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-26])
def test_gradient_of_large_and_small_rows(gpu, eps, D):
    note(f"rms_bwd range {eps} {D}")
    sizes = np.array([0.0, 1e-17, 1e-14, 1.0, 1e13, 1e17, 3e-14, 1e-16])
    if eps == 0.0:
        sizes[0] = 1e-15                       # a row of zeros has no gradient without an eps
    r = np.random.default_rng(D)
    M = len(sizes)
    a = norm.hold(r.normal(size=(M, D)) * sizes[:, None], "f32")
    dy = norm.hold(r.normal(size=(M, D)), "f32")
    w = norm.hold(1 + 0.2 * r.normal(size=D), "f32")
    x, y, z = norm.num(a), norm.num(dy), norm.num(w)
    eps32 = float(np.float32(eps))
    wx, _ = ref.rms_bwd(y, x, z, None, eps32)
    dx, _ = gpu.ss_rms_bwd(dy, a, w, eps=eps)
    c = (np.square(x).mean(-1, keepdims=True) + eps32) ** -0.5
    terms = np.abs(z * y * c) + np.abs(x) * c ** 3 * np.abs(z * y * x).mean(-1, keepdims=True)
    norm.near(dx, wx, terms * 4 * norm.eps_of(D), "dx")
