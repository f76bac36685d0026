"""Linear attention, norm and 4-bit products where offsets pass 2^31 elements: the first and the
last rows against the float64 oracle (a decay of -inf cuts what the oracle need not read).
Tolerances as in test_gpu_la.py, test_gpu_norm.py and test_gpu_q4.py."""
import numpy as np
import pytest

from oracle import la_ref
from oracle import norm_q4_ref as ref
from tests import test_gpu_la as la
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def test_long_sequence(gpu):
    """v, do, o, dv of 2^31 + 3·2048 elements."""
    import torch
    T, H, dk, dv, n = (1 << 20) + 3, 16, 16, 128, 90
    note("la long sequence")
    gen = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = draw(1, T, 1, dk), draw(1, T, 1, dk), draw(1, T, H, dv), draw(1, T, H, dv)
    assert v.numel() > 1 << 31
    g = -torch.rand((1, T, H), generator=gen, device="cuda")
    g[:, n] = float("-inf")       # the first n tokens and the last n stand alone
    g[:, T - n] = float("-inf")
    o, s = gpu.ss_la_fwd(q, k, v, g, scale=0.25, return_final=True)
    r = gpu.ss_la_bwd(q, k, v, do, g, scale=0.25)
    torch.cuda.synchronize()
    for part in (slice(0, n), slice(T - n, T)):
        num = lambda t: t[:, part].float().cpu().numpy()  # noqa: E731
        c = dict(q=num(q), k=num(k), v=num(v), do=num(do), g=num(g), s0=None, ds=None, scale=0.25,
                 lengths=None, dtype="bf16")
        a = la.absolute(c)
        wo, ws = la_ref.fwd(c["q"], c["k"], c["v"], c["g"], None, 0.25)
        Ao, As = la_ref.fwd(a["q"], a["k"], a["v"], c["g"], None, 0.25)
        la.near(o[:, part], wo, la.out_bound(c, Ao), "o")
        if part.start:
            la.near(s, ws, As * la.units(c) + 1e-37, "s_final")
        la.check_bwd(c, {m: None if r[m] is None else r[m] if m == "ds0" else r[m][:, part] for m in r})


def test_many_rows(gpu):
    import torch
    M, D = (1 << 20) + 5, 2048
    note("rms many rows")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    assert x.numel() > 1 << 31
    y8, sc, r = gpu.ss_rms_fwd(x, w, x, q8=gpu.SS_Q8_FP8)
    y, _ = gpu.ss_rms_fwd(x, w, x)
    dx, dw = gpu.ss_rms_bwd(x, x, w)
    rows = [0, 1, M // 2, M - 1]
    num = lambda t: t[rows].float().cpu().numpy().astype(np.float64)  # noqa: E731
    e = (D / 64 + 32) * 2.0 ** -24
    wy, wr = ref.rms_fwd(num(x), w.cpu().numpy(), num(x))
    assert (np.abs(num(y) - wy) <= np.abs(wy) * (2 * e + 2.0 ** -8)).all()
    assert (np.abs(num(r) - wr) <= np.abs(wr) * 1.001 * 2.0 ** -8).all()
    s = sc[rows].cpu().numpy().astype(np.float64)[:, None]
    assert (np.abs(num(y8) * s - wy) <= np.maximum(np.abs(wy) * 2.0 ** -4, 2.0 ** -10 * s) * 1.001).all()
    wx, _ = ref.rms_bwd(num(x), num(x), w.cpu().numpy())
    a = num(x)
    c = (np.square(a).mean(-1, keepdims=True) + 1e-5) ** -0.5
    terms = np.abs(w.cpu().numpy() * a * c) + np.abs(a) * c ** 3 * np.abs(w.cpu().numpy() * a * a).mean(-1, keepdims=True)
    assert (np.abs(num(dx) - wx) <= terms * 4 * e + 1.001 * 2.0 ** -8 * np.abs(wx)).all()


def test_many_weights(gpu):
    import torch
    N, K = (1 << 20) + 7, 4096
    note("q4 many weights")
    gen = torch.Generator(device="cuda").manual_seed(3)
    wq = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    assert wq.numel() > 1 << 31
    sc = torch.rand((N, K // 128), generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn((2, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    y = gpu.ss_q4_mv(x, wq, sc, y_dtype=torch.float32)
    rows = [0, 1, N // 2, N - 2, N - 1]
    xs, ss_ = x.float().cpu().numpy(), sc[rows].float().cpu().numpy()
    want = ref.q4_mv(xs, wq[rows].cpu().numpy(), ss_, None, 128)
    A = np.abs(xs) @ np.repeat(ss_ * 40.0, 128, 1).T
    assert (np.abs(y[:, rows].cpu().numpy() - want) <= A * (K / 32 + 64) * 2.0 ** -24).all()
