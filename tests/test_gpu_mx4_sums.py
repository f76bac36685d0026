"""ss_mx4_mm's sums are float32 for every pair of types: rows of x with columns far above the others,
and every code of the weights with every exponent.

A product of e4m3 and e2m1 is a multiple of 2^-10 of at most 2688, so a sum of K of them in float32 is
off by at most (K / 128 + 16)·2^-24 of its absolute terms, doubled for instructions that cut instead of
rounding, as for two e2m1 codes (test_gpu_mx4.py).  The row's scale and bfloat16 round once each.
"""
import numpy as np
import pytest

from oracle import ln_mx4_ref as ref
from tests.gpu_util import note
from tests.test_gpu_mx4 import U, cuda, num

pytestmark = pytest.mark.gpu

# (M, N, K): rows of 16, 32 and 64 a workgroup; tiles of 64 rows and, where there are many, of 128; odd sizes
SHAPES = [(1, 40, 2048), (7, 300, 96), (20, 4100, 640), (40, 8200, 160), (64, 2560, 1024), (64, 7680, 160),
          (100, 5250, 672), (1100, 1920, 512), (2113, 1025, 96), (5200, 128, 128), (4500, 1500, 96),
          (6200, 1025, 128), (3300, 2050, 672), (64, 99000, 64), (70, 70000, 64)]


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_columns_that_stand_out(gpu, shape, y_dtype):
    """Two of every eight columns are 2^12 times the others and cancel: what is left is the sum of the small
    ones, which an instruction that kept fewer bits than float32 of its products would lose."""
    import torch
    M, N, K = shape
    note(f"mx4 outliers {shape} {y_dtype}")
    r = np.random.default_rng(sum(shape))
    codes = r.integers(0, 16, (N, K))
    codes[:, 0::8] = 7                                  # 6
    codes[:, 3::8] = 15                                 # -6
    wq, we = ref.pack(codes), np.repeat(r.integers(120, 130, (N, 1)), K // 32, 1).astype(np.uint8)
    x = 0.1 * r.normal(size=(M, K))
    top = np.where(r.random((M, K // 8)) < 0.5, 448.0, -416.0)
    x[:, 0::8], x[:, 3::8] = top, top
    t = cuda(x.astype(np.float32)).to(torch.float8_e4m3fn)
    s = (0.01 + r.random(M)).astype(np.float32)
    X, W, f = t.double(), cuda(ref.mx4_values(codes, we.astype(np.int64))), cuda(s).double()[:, None]
    want, terms = X @ W.T * f, X.abs() @ W.abs().T * f
    dt = torch.bfloat16 if y_dtype == "bf16" else torch.float32
    y = gpu.ss_mx4_mm(t, cuda(s), cuda(wq), cuda(we), y_dtype=dt).double()
    tol = (2 * (K / 128 + 16) + 1) * U * terms + (1.001 * 2.0 ** -8 * want.abs() if y_dtype == "bf16" else 0)
    over = ((y - want).abs() - tol).max()
    assert over <= 0, (float(over), float((y - want).norm() / want.norm()))


@pytest.mark.parametrize("top", [448.0, 1.875])
@pytest.mark.parametrize("M", [1, 33, 300, 8200])
def test_products_of_every_size(gpu, M, top):
    """One e4m3 value against one code, over all of both, beside a large product and its negative (the
    largest of all; the largest of values below 2): the sum is the product, exactly."""
    import torch
    note(f"mx4 sizes {M} {top}")
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    v = v[torch.isfinite(v.float())].float()
    K, N = 64, 256
    for at, big in ((0, (1, 2)), (3, (5, 7)), (9, (8, 15)), (40, (47, 41)), (63, (56, 62))):
        codes = np.zeros((N, K), np.int64)
        codes[:, at] = np.arange(N) % 16
        codes[:, big[0]], codes[:, big[1]] = 7, 15
        x = torch.zeros(M, K)
        x[:, at] = v[torch.arange(M) % len(v)] if M > 1 else 9.0 * 2.0 ** -9
        x[:, big[0]] = x[:, big[1]] = top
        t = x.to(torch.float8_e4m3fn).cuda()
        we = np.full((N, K // 32), 127, np.uint8)
        want = num(x)[:, at:at + 1] * ref.mx4_values(codes, we.astype(np.int64))[:, at]
        for dt in (torch.float32, torch.bfloat16):     # (six significant bits: both hold them)
            y = num(gpu.ss_mx4_mm(t, torch.ones(M, device="cuda"), cuda(ref.pack(codes)), cuda(we), y_dtype=dt))
            assert (y == want).all(), (at, dt, int((y != want).sum()))


@pytest.mark.parametrize("M", [1, 40, 300, 2700, 9000])
def test_all_codes_with_all_exponents(gpu, M):
    """Every code of the weights under every exponent, 0 (2^-127) among them, against rows of 1 and -1 (of x
    in both formats) and scales that keep the products in float32's range: exact, NaN at 255."""
    import torch
    note(f"mx4 codes and exponents {M}")
    K, k = 96, 41
    code, e = np.divmod(np.arange(4096), 256)
    wq, we = np.zeros((4096, K), np.int64), np.full((4096, K // 32), 120, np.uint8)
    wq[:, k], we[:, k // 32] = code, e
    wq = ref.pack(wq)
    sign = np.where(np.arange(M) % 2, -1.0, 1.0)
    xq, xe = np.zeros((M, K), np.int64), np.full((M, K // 32), 127, np.uint8)
    xq[:, k] = np.where(sign < 0, 10, 2)
    value = ref.E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    x = torch.zeros(M, K)
    x[:, k] = torch.from_numpy(sign)
    t = x.to(torch.float8_e4m3fn).cuda()
    for part, power in ((slice(0, 128), 30), (slice(128, 255), -30)):
        pick = (e >= part.start) & (e < part.stop)
        want = sign[:, None] * value * 2.0 ** (e + float(power) - 127)
        xe[:, k // 32] = 127 + power
        s = torch.full((M,), 2.0 ** power, device="cuda")
        for dt in (torch.float32, torch.bfloat16):
            y = num(gpu.ss_mx4_mm(cuda(ref.pack(xq)), cuda(xe), cuda(wq), cuda(we), y_dtype=dt))
            assert (y[:, pick] == want[:, pick]).all() and np.isnan(y[:, e == 255]).all(), (part, dt, "4 bits")
            # (e4m3: the row's scale comes after the sum, which has to be a float32 itself)
            z = num(gpu.ss_mx4_mm(t, s, cuda(wq), cuda(we), y_dtype=dt))
            held = pick & (np.abs(value) * 2.0 ** (e - 127.0) < 2.0 ** 128)
            assert (z[:, held] == want[:, held]).all() and np.isnan(z[:, e == 255]).all(), (part, dt, "8 bits")
