"""GPU parity of the microscaled 4-bit values (ss_mx4_quant) and their products (ss_mx4_mm).

Rounding to the format is exact: codes and exponents equal the oracle's.  A product of two codes is
a multiple of 1/4 of at most 36, exact in float32; the sum of K of them in float32 is off by at most
(K / 128 + 16)·2^-24 of its absolute terms (a matrix instruction adds 128 columns, then eight waves
or fewer are joined), doubled for instructions that cut instead of rounding.  With e4m3 rows and
bfloat16 results the products of an instruction lose what is below 2^-13 of the largest of them
(2^-13·Σ over runs of 32 columns of the largest product, four a run); bfloat16 rounds once more, 2^-8.
"""
import numpy as np
import pytest

from oracle import ln_mx4_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def num(t):
    return t.float().cpu().numpy().astype(np.float64)


def weights(seed, N, K, spread=3):
    r = np.random.default_rng(seed)
    return r.integers(0, 256, (N, K // 2), dtype=np.uint8), r.integers(124 - spread, 124 + spread, (N, K // 32)).astype(np.uint8)


def values(codes, exps):
    return ref.mx4_values(ref.unpack(codes), exps.astype(np.int64))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32), (1, 64), (3, 96), (2, 2560), (65, 544), (700, 1024), (1, 65536)], ids=str)
def test_rounding(gpu, shape, dt):
    import torch
    note(f"mx4_quant {shape} {dt}")
    r = np.random.default_rng(sum(shape))
    x = r.normal(size=shape) * 2.0 ** r.integers(-40, 40, size=(shape[0], 1))
    # ties, both zeros, and whole blocks of small and of huge values
    x.reshape(-1)[: 16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0])
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    t = t.to(torch.bfloat16) if dt == "bf16" else t
    codes, exps = gpu.ss_mx4_quant(t)
    wc, we = ref.mx4_quant(t.float().cpu().numpy())
    assert (exps.cpu().numpy() == we).all()
    assert (codes.cpu().numpy() == ref.pack(wc)).all()


def test_rounding_over_the_range(gpu):
    """Every exponent of float32, NaN and infinities, each in a block of its own."""
    import torch
    r = np.random.default_rng(5)
    x = (1 + r.random((256, 32))).astype(np.float32) * np.where(r.random((256, 32)) < 0.5, -1, 1).astype(np.float32)
    bits = x.view(np.uint32) & 0x807FFFFF | (np.arange(256, dtype=np.uint32)[:, None] << 23)
    x = bits.view(np.float32)
    x[:, 7] = 0
    codes, exps = gpu.ss_mx4_quant(cuda(x))
    with np.errstate(invalid="ignore"):
        wc, we = ref.mx4_quant(x)
    assert we[255, 0] == 255 and (exps.cpu().numpy() == we).all()
    assert (codes.cpu().numpy() == ref.pack(wc)).all()
    y = torch.zeros(3, 64, device="cuda")
    y[0, 5], y[1, 40], y[2, 63] = float("inf"), float("nan"), -float("inf")
    codes, exps = gpu.ss_mx4_quant(y)
    assert exps.tolist() == [[255, 1], [1, 255], [1, 255]] and not codes.any()


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 40, 128), (2, 17, 96), (16, 48, 544), (17, 33, 160), (31, 256, 1024),
          (33, 100, 288), (64, 64, 2560), (65, 130, 96), (100, 1, 2048), (128, 128, 128), (129, 257, 416),
          (200, 300, 1056), (255, 250, 64), (256, 256, 256), (300, 520, 32), (513, 129, 672), (1000, 384, 512),
          (33, 5121, 96), (40, 5250, 640), (65, 2600, 160), (100, 2688, 1024), (129, 1801, 416), (257, 1100, 544),
          (300, 1030, 1056), (511, 640, 32), (512, 1024, 128), (700, 500, 672), (1025, 385, 288),
          (2050, 160, 384), (5200, 64, 64), (5121, 65, 256), (700, 513, 2560)]
# N · ceil(M / 64) of 7680 and more go in tiles of 64 rows of x; more than 256 tiles of 64 in tiles of 128,
# and of x in 4 bits, with more than 256 tiles of 128, of 256
TILES = [(33, 10241, 96), (65, 5130, 640), (100, 5250, 160), (129, 3500, 416), (257, 2100, 1056), (511, 1285, 32),
         (1025, 610, 288), (5200, 128, 64), (5121, 131, 256), (700, 1024, 2560),
         (1090, 2050, 96), (1300, 1700, 288), (1100, 1920, 512), (2113, 1025, 544), (40, 33000, 96),
         (2177, 2100, 96), (4200, 1030, 160), (2304, 2048, 640), (8200, 515, 32), (2500, 1793, 1152),
         (700, 1100, 2592), (130, 5203, 1632), (64, 10241, 608), (2300, 2049, 736)]


@pytest.mark.parametrize("x", ["mx4", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products(gpu, shape, x):
    import torch
    M, N, K = shape
    note(f"mx4_mm {shape} {x}")
    wq, we = weights(sum(shape), N, K)
    W = values(wq, we)
    if x == "mx4":
        xq, xe = weights(K + M, M, K)
        X, xs = values(xq, xe), None
        args = (cuda(xq), cuda(xe))
    else:
        r = np.random.default_rng(M + K)
        t = torch.from_numpy((100 * r.normal(size=(M, K))).astype(np.float32)).cuda().clamp(-448, 448).to(torch.float8_e4m3fn)
        xs = (0.01 + r.random(M)).astype(np.float32)
        X = num(t)
        args = (t, cuda(xs))
    want = X @ W.T
    terms = np.abs(X) @ np.abs(W).T
    tol = 2 * (K / 128 + 16) * U * terms
    # the largest product of each run of 32 columns
    cut = np.zeros_like(want)
    for k in range(0, K, 32):
        cut += (np.abs(X[:, None, k:k + 32]) * np.abs(W[None, :, k:k + 32])).max(-1)
    cut *= 4 * 2.0 ** -13 if x == "fp8" else 0
    if xs is not None:
        want, tol, cut = want * xs[:, None], (tol + U * terms) * xs[:, None], cut * xs[:, None]
    y = gpu.ss_mx4_mm(*args, cuda(wq), cuda(we))
    assert y.dtype == torch.bfloat16 and (np.abs(num(y) - want) <= tol + cut + 1.001 * 2.0 ** -8 * np.abs(want)).all()
    y = gpu.ss_mx4_mm(*args, cuda(wq), cuda(we), y_dtype=torch.float32)
    assert y.dtype == torch.float32 and (np.abs(num(y) - want) <= tol).all()


@pytest.mark.parametrize("x", ["mx4", "fp8"])
@pytest.mark.parametrize("M,N,K", TILES)
def test_tiles(gpu, M, N, K, x):
    """As test_products, the oracle's float64 products on the GPU."""
    import torch
    note(f"mx4 tiles {x} M={M} N={N} K={K}")
    wq, we = weights(M + N, N, K)
    W, xs = cuda(ref.mx4_values(ref.unpack(wq), we)), None
    if x == "mx4":
        xq, xe = weights(M * 7 + K, M, K)
        X, args = cuda(ref.mx4_values(ref.unpack(xq), xe)), (cuda(xq), cuda(xe))
    else:
        r = np.random.default_rng(M + K)
        t = torch.from_numpy((100 * r.normal(size=(M, K))).astype(np.float32)).cuda().clamp(-448, 448).to(torch.float8_e4m3fn)
        X, xs = t.double(), cuda((0.01 + r.random(M)).astype(np.float32))
        args = (t, xs)
    want, terms = X @ W.T, X.abs() @ W.abs().T
    tol = 2 * (K / 128 + 16) * U * terms
    cut = torch.zeros_like(want)
    if x == "fp8":
        for k in range(0, K, 32):
            top = torch.zeros_like(want)
            for j in range(k, k + 32):
                top = torch.maximum(top, X[:, j:j + 1].abs() * W[:, j].abs())
            cut += 4 * 2.0 ** -13 * top
        f = xs.double()[:, None]
        want, tol, cut = want * f, (tol + U * terms) * f, cut * f
    y = gpu.ss_mx4_mm(*args, cuda(wq), cuda(we))
    assert ((y.double() - want).abs() <= tol + cut + 1.001 * 2.0 ** -8 * want.abs()).all()
    y = gpu.ss_mx4_mm(*args, cuda(wq), cuda(we), y_dtype=torch.float32)
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M", [1, 40, 300, 2700, 9000])
def test_every_code_and_exponent(gpu, M):
    """One code of weights against one of x, over all codes and exponents: exact, NaN at 255."""
    import torch
    note(f"mx4 codes {M}")
    K = 160
    for k in (0, 33, 100, 159):
        wq = np.zeros((256, K // 2), np.uint8)
        wq[:, k // 2] = (np.arange(256) % 16) << (4 * (k % 2))
        we = np.full((256, K // 32), 120, np.uint8)
        we[:, k // 32] = np.arange(256)
        xq = np.zeros((M, K // 2), np.uint8)
        xq[:, k // 2] = (2 + 8 * (np.arange(M) % 2)) << (4 * (k % 2))       # 1 and -1
        xe = np.full((M, K // 32), 127, np.uint8)
        y = num(gpu.ss_mx4_mm(cuda(xq), cuda(xe), cuda(wq), cuda(we), y_dtype=torch.float32))
        want = (ref.E2M1[np.arange(256) & 7] * np.where(np.arange(256) & 8, -1, 1) * 2.0 ** (np.arange(256) - 127.0))
        want = (want * np.where(np.arange(M) % 2, -1, 1)[:, None]).astype(np.float32).astype(np.float64)
        assert np.isnan(y[:, 255]).all() and (y[:, :255] == want[:, :255]).all(), k
        t = torch.zeros(M, K, device="cuda")
        t[:, k] = cuda(np.where(np.arange(M) % 2, -1.0, 1.0).astype(np.float32))
        one = torch.ones(M, device="cuda")
        for dt in (torch.float32, torch.bfloat16):
            z = num(gpu.ss_mx4_mm(t.to(torch.float8_e4m3fn), one, cuda(wq), cuda(we), y_dtype=dt))
            assert np.isnan(z[:, 255]).all() and (z[:, 1:255] == want[:, 1:255]).all(), (k, dt)


def test_rows_stay_apart(gpu):
    """NaN in a row of x (a block's exponent, a code, a scale) or of the weights stays in its row or
    column."""
    import torch
    for M, N, K in ((20, 40, 256), (300, 200, 320), (3400, 200, 320), (4000, 192, 256), (10000, 290, 160), (4000, 193, 1056), (5000, 211, 864)):
        wq, we = weights(3, N, K)
        xq, xe = weights(4, M, K)
        y = gpu.ss_mx4_mm(cuda(xq), cuda(xe), cuda(wq), cuda(we))
        xe2, we2 = xe.copy(), we.copy()
        xe2[5, -1] = we2[7, 0] = 255
        z = gpu.ss_mx4_mm(cuda(xq), cuda(xe2), cuda(wq), cuda(we2))
        bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        bad[5], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(z), bad) and torch.equal(z[~bad], y[~bad])
        t = torch.randn(M, K, device="cuda").to(torch.float8_e4m3fn)
        s = torch.ones(M, device="cuda")
        y = gpu.ss_mx4_mm(t, s, cuda(wq), cuda(we))
        t.view(torch.uint8)[3, K - 1] = 0x7F
        s[6] = float("nan")
        for dt in (torch.bfloat16, torch.float32):
            z = gpu.ss_mx4_mm(t, s, cuda(wq), cuda(we), y_dtype=dt)
            assert torch.equal(torch.isnan(z).all(-1).nonzero()[:, 0].cpu(), torch.tensor([3, 6]))
            assert torch.isnan(z).sum() == 2 * N


def test_shapes_streams_and_graph(gpu):
    import torch
    note("mx4 stream, graph")
    x = torch.randn(3, 50, 640, device="cuda", dtype=torch.bfloat16)
    wq, we = (cuda(a) for a in weights(6, 300, 640))
    codes, exps = gpu.ss_mx4_quant(x)
    assert codes.shape == (3, 50, 320) and exps.shape == (3, 50, 20)
    y = gpu.ss_mx4_mm(codes, exps, wq, we)
    assert y.shape == (3, 50, 300)
    flat = gpu.ss_mx4_mm(codes.view(150, 320), exps.view(150, 20), wq, we)
    assert torch.equal(y.view(150, 300), flat)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c2, e2 = gpu.ss_mx4_quant(x, stream=side)
    y2 = gpu.ss_mx4_mm(c2, e2, wq, we, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c2, codes) and torch.equal(y2, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.ss_mx4_mm(*gpu.ss_mx4_quant(x), wq, we)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
        torch.randn(1 << 20, device="cuda").sum().item()


def test_refusals(gpu):
    import torch
    x = torch.randn(4, 64, device="cuda")
    codes, exps = gpu.ss_mx4_quant(x)
    wq, we = (cuda(a) for a in weights(1, 8, 64))
    with pytest.raises(ValueError):
        gpu.ss_mx4_quant(x[:, :48].contiguous())
    with pytest.raises(ValueError):
        gpu.ss_mx4_quant(x.half())
    with pytest.raises(ValueError):
        gpu.ss_mx4_quant(x.t())
    with pytest.raises(ValueError):
        gpu.ss_mx4_mm(x, exps, wq, we)
    with pytest.raises(ValueError):
        gpu.ss_mx4_mm(codes, exps[:, :1], wq, we)
    with pytest.raises(ValueError):
        gpu.ss_mx4_mm(codes, exps, wq[:, :16].contiguous(), we)
    with pytest.raises(ValueError):
        gpu.ss_mx4_mm(codes, exps, wq, we, y_dtype=torch.float16)
    with pytest.raises(TypeError):
        gpu.ss_mx4_mm(codes, None, wq, we)
    with pytest.raises(gpu.SSError) as e:      # 16 bytes that are not a block of 32 columns
        gpu.ss_mx4_mm(codes[:, :8].contiguous(), exps[:, :0], wq[:, :8].contiguous(), we[:, :0])
    assert e.value.code == -2
