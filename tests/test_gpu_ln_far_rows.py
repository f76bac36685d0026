"""Rows far from 0 whose few elements end inside a piece of eight: what stands for the missing ones has no
part in the row's scale."""
import numpy as np
import pytest

from tests.gpu_util import note
from tests.test_gpu_ln import num

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [1, 2, 4])
@pytest.mark.parametrize("q8", ["fp8", "int8"])
def test_constant_rows(gpu, D, q8):
    """y = b for a constant row (at these widths its mean is exact); the mean times 1/sqrt(eps) is past
    float32."""
    import torch
    note(f"ln far rows {D} {q8}")
    b = torch.linspace(1, -0.5, D, device="cuda")
    w = torch.ones(D, device="cuda")
    x = torch.ones(3, D, device="cuda")
    x[0], x[1] = 2.0 ** 115, -(2.0 ** 114)
    code, top = {"fp8": (gpu.SS_Q8_FP8, 448.0), "int8": (gpu.SS_Q8_INT8, 127.0)}[q8]
    y, s = gpu.ss_ln_fwd(x, w, b, eps=1e-12, q8=code)
    assert np.abs(num(s) * top - 1).max() < 1e-6
    for i in (0, 1):
        assert torch.equal(y[i].view(torch.uint8), y[2].view(torch.uint8))
