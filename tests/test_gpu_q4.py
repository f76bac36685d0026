"""GPU parity of the products with 4-bit weights (ss_q4_mv) against the float64 oracle.

Tolerance of each element, with A = Σ_j |x_j|·s·(16 + |z| + 16), the absolute terms of the sum as
it is formed (codes with 16 added, (16 + z)·Σx taken off again): each of a group's at most four
products of 32 terms and the additions across groups, waves and terms is a float32 rounding of a
partial sum, at most K / 32 + 32 of them one after the other, 2^-24·A each; the products of 32
terms add 32 such inside.  Float32 x is held to 2^-24 by its three bfloat16 terms.  A bfloat16
result is rounded once more, 2^-8 of it.
"""
import numpy as np
import pytest

from oracle import norm_q4_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def make(seed, M, N, K, group, x, zeros):
    import torch
    r = np.random.default_rng(seed)
    ng = -(-K // group)
    t = dict(wq=torch.from_numpy(r.integers(0, 256, size=(N, K // 2)).astype(np.uint8)).cuda(),
             scales=torch.from_numpy(r.uniform(-0.05, 0.05, size=(N, ng)).astype(np.float32)).to(torch.bfloat16).cuda(),
             zeros=torch.from_numpy(r.integers(0, 16, size=(N, ng)).astype(np.uint8)).cuda() if zeros else None,
             x_scale=None)
    v = torch.from_numpy(r.normal(size=(M, K)).astype(np.float32)).cuda()
    if x == "fp8":
        t["x"] = (v * 60).to(torch.float8_e4m3fn)
    elif x == "int8":
        t["x"] = torch.from_numpy(r.integers(-127, 128, size=(M, K)).astype(np.int8)).cuda()
    else:
        t["x"] = v.to(torch.bfloat16 if x == "bf16" else torch.float32)
    if x in ("fp8", "int8"):
        t["x_scale"] = torch.from_numpy(r.uniform(0.001, 0.1, size=M).astype(np.float32)).cuda()
    return t


def num(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def check(t, group, y):
    import torch
    x, s = num(t["x"]), num(t["scales"])
    K = x.shape[1]
    want = ref.q4_mv(x, t["wq"].cpu().numpy(), s, num(t["zeros"]), group, num(t["x_scale"]))
    at = np.arange(K) // group
    z = np.full(s.shape, 8.0) if t["zeros"] is None else num(t["zeros"])
    A = np.abs(x) @ (np.abs(s) * (32 + z))[:, at].T
    if t["x_scale"] is not None:
        A = A * num(t["x_scale"])[:, None]
    bound = A * (K / 32 + 64) * 2.0 ** -24 + (2.0 ** -8 * np.abs(want) if y.dtype == torch.bfloat16 else 0)
    got = num(y)
    assert got.shape == want.shape
    over = np.abs(got - want) - bound
    assert np.isfinite(got).all() and (over <= 0).all(), float(over.max())


CASES = [  # M, N, K, group
    (1, 1, 32, 32), (1, 16, 32, 128), (2, 17, 64, 64), (1, 100, 96, 64), (3, 33, 160, 128),
    (5, 48, 256, 32), (6, 31, 512, 128), (16, 64, 1024, 64), (17, 20, 288, 128), (33, 40, 640, 32),
    (1, 257, 2560, 128), (16, 96, 5120, 64), (9, 130, 2080, 128), (1, 40, 40000, 128),
    (40, 16, 4128, 32),
]


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("x", ["bf16", "f32", "fp8", "int8"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_products(gpu, case, x, zeros):
    import torch
    M, N, K, group = case
    t = make(sum(case), M, N, K, group, x, zeros)
    note(f"q4_mv {case} {x} zeros={zeros}")
    args = (t["x"], t["wq"], t["scales"], t["zeros"])
    y = gpu.ss_q4_mv(*args, group=group, x_scale=t["x_scale"])
    assert y.dtype == (torch.float32 if x == "f32" else torch.bfloat16)
    check(t, group, y)
    other = torch.bfloat16 if x == "f32" else torch.float32
    check(t, group, gpu.ss_q4_mv(*args, group=group, x_scale=t["x_scale"], y_dtype=other))


def test_codes_are_exact(gpu):
    """x a unit vector and scales 1: every code comes back as itself, in its own place."""
    import torch
    N, K = 16, 256
    wq = torch.arange(N * K // 2, device="cuda").remainder(256).to(torch.uint8).view(N, K // 2)
    ones = torch.ones(N, 2, dtype=torch.bfloat16, device="cuda")
    zeros = torch.full((N, 2), 0, dtype=torch.uint8, device="cuda")
    note("q4 codes")
    eye = torch.eye(K, device="cuda")
    for x in (eye, eye.to(torch.bfloat16)):
        y = gpu.ss_q4_mv(x, wq, ones, zeros, y_dtype=torch.float32)
        want = torch.stack([wq & 15, wq >> 4], -1).flatten(1).float().t()
        assert torch.equal(y, want)
        assert torch.equal(gpu.ss_q4_mv(x, wq, ones, y_dtype=torch.float32), want - 8)


def test_a_bad_row_stays_alone(gpu):
    import torch
    t = make(5, 6, 40, 256, 64, "f32", True)
    note("q4 bad row")
    args = (t["wq"], t["scales"], t["zeros"])
    clean = gpu.ss_q4_mv(t["x"], *args, group=64)
    x = t["x"].clone()
    x[2, 7], x[4, 9] = float("nan"), float("inf")
    y = gpu.ss_q4_mv(x, *args, group=64)
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()


def test_norm_feeds_the_products(gpu):
    """A token through the norm's 8-bit rows into 4-bit weights, on a stream and in a graph."""
    import torch
    t = make(6, 2, 200, 512, 128, "f32", True)
    w = torch.ones(512, device="cuda")
    note("norm into q4")

    def chain():
        y8, sc = gpu.ss_rms_fwd(t["x"], w, q8=gpu.SS_Q8_FP8)
        return y8, sc, gpu.ss_q4_mv(y8, t["wq"], t["scales"], t["zeros"], x_scale=sc)
    y8, sc, y = chain()
    check(dict(t, x=y8, x_scale=sc), 128, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = gpu.ss_q4_mv(y8, t["wq"], t["scales"], t["zeros"], x_scale=sc, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(3):
        out[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[2], y)
        torch.randn(1 << 20, device="cuda").sum().item()


def test_refusals(gpu):
    import torch
    t = make(7, 2, 32, 128, 64, "bf16", True)
    x, wq, s, z = t["x"], t["wq"], t["scales"], t["zeros"]
    for bad in ((x.half(), wq, s, z), (x, wq.to(torch.int16), s, z), (x, wq, s.float(), z),
                (x, wq, s[:, :1].contiguous(), z), (x, wq, s, z[:31]), (x[:, :96].contiguous(), wq, s, z),
                (x, wq.t().contiguous().t(), s, z), (x.to(torch.float8_e4m3fn), wq, s, z)):
        with pytest.raises(ValueError):
            gpu.ss_q4_mv(*bad, group=64)
    with pytest.raises(ValueError):
        gpu.ss_q4_mv(x, wq, s, z, group=64, x_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        gpu.ss_q4_mv(x, wq, s, z, group=64, y_dtype=torch.float16)
    one = torch.ones(32, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_q4_mv(x, wq, one, group=16)
    assert e.value.code == -2
    odd = torch.zeros(2, 40, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_q4_mv(odd, wq[:, :20].contiguous(), one[:, :1].contiguous(), group=64)
    assert e.value.code == -2
