"""Small log decays over a million tokens: k = 0, so that s_final is s0 times the decay alone."""
import numpy as np
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [-1e-13, -3e-11, -1e-7, 1e-13], ids=str)
def test_small_decays_do_not_add_up_an_error(gpu, g):
    """2^20 tokens of 8 heads run as 128 segments of 256 chunks of 32 float32 tokens.  A segment's
    decay and a chunk's decay are powers of exact sums, each a power's unit (2^-23) and one
    product's rounding (2^-24) off: at most (128 + 256)·(2^-23 + 2^-24) of the result.  A log decay
    that is off by 2^-32 in base 2 for each token would show as 1.7e-4, 2.4 times that."""
    import torch
    T, H, d = 1 << 20, 8, 4
    note(f"la long decay {g}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    v, s0 = draw(1, T, H, d), draw(1, H, d, d)
    k = torch.zeros(1, T, H, d, device="cuda")
    decay = torch.full((H,), g, device="cuda")
    _, s = gpu.ss_la_fwd(k, k, v, decay, s0, return_final=True)
    want = s0.double().cpu().numpy() * np.exp(float(np.float32(g)) * T)
    err = np.abs(s.double().cpu().numpy() - want) / np.abs(want)
    assert err.max() <= (128 + 256) * (2.0 ** -23 + 2.0 ** -24), err.max()
