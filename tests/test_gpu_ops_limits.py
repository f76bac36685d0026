"""Sizes whose rows of work pass 2^32 threads of one launch."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def test_shared_heads_of_2_to_32_elements(gpu):
    """dq and dk of 2^32 + 2^13 elements, summed over two value heads: the first and the last tokens
    against a call of their own (a decay of -inf cuts them off)."""
    import torch
    n, Hk, H, dk, dv = 64, 32, 64, 128, 4
    T = (1 << 20) + 2
    note("la shared heads of 2^32 elements")
    gen = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = draw(1, T, Hk, dk), draw(1, T, Hk, dk), draw(1, T, H, dv), draw(1, T, H, dv)
    assert q.numel() > 1 << 32
    g = -torch.rand((1, T, H), generator=gen, device="cuda")
    g[:, n] = float("-inf")
    g[:, T - n] = float("-inf")
    r = gpu.ss_la_bwd(q, k, v, do, g, scale=0.25)
    torch.cuda.synchronize()
    for part in (slice(0, n), slice(T - n, T)):
        cut = [x[:, part].contiguous() for x in (q, k, v, do, g)]
        want = gpu.ss_la_bwd(*cut[:4], cut[4], scale=0.25)
        for m in ("dq", "dk", "dv"):
            # the same sums in chunks that begin elsewhere: one rounding to bfloat16 apart
            x, y = r[m][:, part].float(), want[m].float()
            assert (x - y).abs().max() <= 2.0 ** -7 * y.abs().max(), m
        assert torch.isfinite(r["dg"][:, part]).all()
