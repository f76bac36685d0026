"""4-bit products of rows that hold infinities, NaN, or values whose sums with 16 added to each code
would leave float32: the value that the formula gives, in that row alone."""
import numpy as np
import pytest

from oracle import norm_q4_ref as ref
from tests import test_gpu_q4 as q4
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(6, 40, 256, 64), (3, 33, 160, 128), (16, 600, 96, 32), (7, 9000, 64, 32)], ids=str)
def test_infinities(gpu, case, x, zeros):
    M, N, K, group = case
    t = q4.make(3 + sum(case), M, N, K, group, x, zeros)
    note(f"q4 infinite {case} {x} {zeros}")
    args = (t["wq"], t["scales"], t["zeros"])
    clean = gpu.ss_q4_mv(t["x"], *args, group=group)
    t["x"] = t["x"].clone()
    t["x"][1, 7] = float("inf")
    t["x"][2, 9], t["x"][2, K - 1] = float("-inf"), float("inf")
    bad = [1, 2]
    if M > 5:
        t["x"][4, 3] = float("nan")
        bad.append(4)
    y = gpu.ss_q4_mv(t["x"], *args, group=group)
    keep = [m for m in range(M) if m not in bad]
    assert np.array_equal(q4.num(y)[keep], q4.num(clean)[keep])
    with np.errstate(invalid="ignore"):
        W = ref.q4_weights(t["wq"].cpu().numpy(), q4.num(t["scales"]), q4.num(t["zeros"]), group)
        for m in bad:      # inf·0 is NaN, and so is inf - inf
            row = q4.num(t["x"])[m]
            want = (row[None] * W)[:, ~np.isfinite(row)].sum(-1)
            got = q4.num(y)[m]
            assert np.array_equal(np.isnan(got), np.isnan(want)), m
            assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)]), m


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_large_values(gpu, x):
    """128 values of up to 2e36: with 24 for a code their sum passes float32, the products do not."""
    import torch
    M, N, K, group = 4, 50, 384, 128
    t = q4.make(8, M, N, K, group, x, True)
    note(f"q4 large {x}")
    r = np.random.default_rng(9)
    u = r.integers(7, 10, size=(N, K)).astype(np.uint8)
    t["wq"] = torch.from_numpy(u[:, 0::2] | (u[:, 1::2] << 4)).cuda()
    t["zeros"] = torch.full_like(t["zeros"], 8)
    t["scales"] = (t["scales"].float() * 0.1).to(torch.bfloat16)
    big = torch.from_numpy(r.uniform(1e36, 2e36, size=(M, K)).astype(np.float32)).cuda()
    t["x"] = big.to(t["x"].dtype)
    y = gpu.ss_q4_mv(t["x"], t["wq"], t["scales"], t["zeros"], group=group)
    q4.check(t, group, y)
