"""Gated recurrence, layer norm and 4-bit values where offsets pass 2^31 elements: first and last rows
against the float64 oracles.  Tolerances as in test_gpu_gr.py, test_gpu_ln.py and test_gpu_mx4.py."""
import numpy as np
import pytest

from oracle import ln_mx4_ref as ref
from tests import test_gpu_gr as gr
from tests import test_gpu_ln as ln
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def test_long_sequence(gpu):
    """x, gates, dy and their gradients of 2^31 + 3·2048 elements, slices of one wider tensor.  Two
    documents' beginnings set the first and the last tokens apart."""
    import torch
    T, D, n = (1 << 20) + 3, 2048, 90
    note("gr long sequence")
    gen = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, r, i = draw(1, T, 3 * D).split(D, -1)
    dy = draw(1, T, D)
    lam = gr.make(1, 1, 1, D, "f32")["lam"]
    reset = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    reset[0, n] = reset[0, T - n] = True
    y, hf, ck = gpu.ss_gr_fwd(x, r, i, lam, reset=reset, return_final=True, return_ckpt=True)
    g = gpu.ss_gr_bwd(x, r, i, lam, dy, reset=reset, h_ckpt=ck)
    torch.cuda.synchronize()
    for part in (slice(0, n), slice(T - n, T)):
        for cols in (slice(0, 40), slice(D - 40, D)):
            p = {m: t[:, part, cols].contiguous() for m, t in (("x", x), ("r", r), ("i", i), ("dy", dy))}
            p.update(lam=lam[cols].contiguous(), h0=None, dh=None, lengths=None, reset=reset[:, part].contiguous())
            w, b = gr.oracle(p)
            gr.near(y[:, part, cols], w["y"], b["y"], "bf16", "y")
            for m in ("dx", "dr", "di"):
                gr.near(g[m][:, part, cols], w[m], b[m], "bf16", m)
            if part.start:
                gr.near(hf[:, cols], w["h_final"], b["h_final"], "f32", "h_final")


def test_many_rows(gpu):
    import torch
    M, D = (1 << 20) + 5, 2048
    note("ln many rows")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    codes, exps = gpu.ss_ln_fwd(x, w, q8=gpu.SS_Q4_MX)
    y = gpu.ss_ln_fwd(x, w)
    dx, dw, db = gpu.ss_ln_bwd(x, y, w)
    for rows in (slice(0, 3), slice(M - 3, M)):
        wy, wr = ref.ln_fwd(ln.num(x[rows]), ln.num(w))
        d, c, q, ec = ln.parts(wr, 1e-5)
        e = np.abs(ln.num(w)) * (c * q + np.abs(d * c) * (ec + 4 * ln.U)) + ln.U * np.abs(wy)
        ln.near(y[rows], wy, e + 1.001 * 2.0 ** -8 * np.abs(wy) + 1e-37, "y")
        wx, _, _ = ref.ln_bwd(ln.num(x[rows]), ln.num(y[rows]), ln.num(w))
        assert np.abs(ln.num(dx[rows]) - wx).max() <= 2.0 ** -8 * np.abs(wx).max() * 1.1 + 1e-5
        v = ref.mx4_values(ref.unpack(codes[rows].cpu().numpy()), exps[rows].cpu().numpy().astype(np.int64))
        step = np.repeat(2.0 ** (exps[rows].cpu().numpy() - 127.0), 32, -1)
        assert (np.abs(v - wy) <= 2 * step + e).all()
    assert abs(float(db.double().sum() / x.double().sum()) - 1) < 1e-3


@pytest.mark.parametrize("x", ["mx4", "fp8"])
def test_products(gpu, x):
    """Rows of x, of weights and of y past 2^31 elements."""
    import torch
    note(f"mx4 large {x}")
    gen = torch.Generator(device="cuda").manual_seed(3)
    byte = lambda *s: torch.randint(0, 256, s, generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    for M, N, K in ((64, (1 << 20) + 40, 2080), ((1 << 20) + 33, 200, 2080), ((1 << 18) + 7, 8320, 64)):
        wq, we = byte(N, K // 2), 120 + byte(N, K // 32) % 8
        if x == "mx4":
            xq, xs = byte(M, K // 2), 120 + byte(M, K // 32) % 8
        else:
            xq = torch.randint(0, 120, (M, K), generator=gen, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
            xs = torch.rand(M, generator=gen, device="cuda")
        y = gpu.ss_mx4_mm(xq, xs, wq, we)
        torch.cuda.synchronize()
        for a in (slice(0, 2), slice(M - 2, M)):
            for b in (slice(0, 5), slice(N - 5, N)):
                W = ref.mx4_values(ref.unpack(wq[b].cpu().numpy()), we[b].cpu().numpy().astype(np.int64))
                X = (ref.mx4_values(ref.unpack(xq[a].cpu().numpy()), xs[a].cpu().numpy().astype(np.int64)) if x == "mx4"
                     else ln.num(xq[a]) * ln.num(xs[a])[:, None])
                want, terms = X @ W.T, np.abs(X) @ np.abs(W).T
                assert (np.abs(ln.num(y[a, b]) - want) <= 1.01 * 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * terms).all()
        del wq, we, xq, xs, y


def test_rounding(gpu):
    import torch
    M, K = (1 << 20) + 3, 2080
    note("mx4_quant large")
    x = torch.randn((M, K), device="cuda", dtype=torch.bfloat16)
    codes, exps = gpu.ss_mx4_quant(x)
    for rows in (slice(0, 3), slice(M - 3, M)):
        wc, we = ref.mx4_quant(x[rows].float().cpu().numpy())
        assert (exps[rows].cpu().numpy() == we).all() and (codes[rows].cpu().numpy() == ref.pack(wc)).all()
