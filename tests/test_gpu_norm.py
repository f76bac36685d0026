"""GPU parity of the RMS norm (ss_rms_fwd, ss_rms_bwd) against the float64 oracle.

Tolerances of each element.  A float32 sum of D terms in lanes and trees is off by at most
(D / threads + 20)·2^-24 of its absolute terms, which for the sum of squares is all of it: with
n = D / 64 + 32 the factor c is within n·2^-24 and y within 2n·2^-24 of |y|; stored in bfloat16,
2^-8 more.  dx = c·w·dy - r·c³·S with S the mean of w·dy·r: |c·w·dy| and |r|·c³·mean|w·dy·r| are
its two terms, each within 4n·2^-24.  dw adds M rows: (M + 4n)·2^-24 of Σ|dy·r·c|.
8 bits: e4m3 has 4 significant bits above 2^-6 and steps of 2^-9 below, so a code times its
scale is within 2^-4 of |y| or half a step (2^-10·scale), int8 within half a step, and the
float32 error of y and of the scale besides.
"""
import numpy as np
import pytest

from oracle import norm_q4_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 511), (4, 512), (7, 513), (3, 1000), (1, 2048),
          (2, 2049), (1, 2560), (1100, 520), (1030, 1536), (1025, 2560), (2, 4099), (3, 8192),
          (2, 8200), (1, 16384), (1, 16392), (2, 20001), (1, 32768)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def hold(x, dt):
    import torch
    t = torch.from_numpy(x.astype(np.float32))
    return (t.to(torch.bfloat16) if dt == "bf16" else t).cuda()


def num(t):
    return t.float().cpu().numpy().astype(np.float64)


def eps_of(D):
    return (D / 64 + 32) * 2.0 ** -24


def near(got, want, bound, what):
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    over = np.abs(got - want) - bound
    assert np.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()))


def data(seed, M, D, types, res):
    r = np.random.default_rng(seed)
    x = hold(r.normal(size=(M, D)), types[0])
    rs = hold(2 * r.normal(size=(M, D)), types[1]) if res else None
    w = hold(1 + 0.2 * r.normal(size=D), "f32")
    return x, rs, w


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(gpu, shape, types, res):
    M, D = shape
    x, rs, w = data(M + D, M, D, types, res)
    note(f"rms_fwd {shape} {types} res={res}")
    wy, wr = ref.rms_fwd(num(x), num(w), None if rs is None else num(rs), 1e-5)
    out = gpu.ss_rms_fwd(x, w, rs, eps=1e-5)
    y, r = out if res else (out, None)
    e = eps_of(D)
    near(y, wy, np.abs(wy) * (2 * e + (2.0 ** -8 if types[0] == "bf16" else 0)) + 1e-37, "y")
    if res:
        # one float32 addition (2^-24 of the sum), then the residual's type
        near(r, wr, np.abs(wr) * (2.0 ** -23 + (1.001 * 2.0 ** -8 if types[1] == "bf16" else 0)), "r")
    for q8, top in ((gpu.SS_Q8_FP8, 448.0), (gpu.SS_Q8_INT8, 127.0)):
        out = gpu.ss_rms_fwd(x, w, rs, eps=1e-5, q8=q8)
        y8, sc = out[:2]
        ws = np.abs(wy).max(-1) / top
        near(sc, ws, ws * (2 * e + 2.0 ** -22), "scale")
        s = num(sc)[:, None]
        half = np.maximum(np.abs(wy) * 2.0 ** -4, 2.0 ** -10 * s) if top == 448.0 else 0.5 * s
        near(y8.float() * sc[:, None], wy, half * 1.0001 + np.abs(wy) * (4 * e + 2.0 ** -21) +
             (127 * 4 * e) * s, "codes")
        if res:
            assert num(out[2]).tolist() == num(r).tolist()


@pytest.mark.parametrize("dr", [True, False])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(gpu, shape, types, dr):
    M, D = shape
    dy, r, w = data(M + 3 * D, M, D, types, True)
    g = hold(np.random.default_rng(D).normal(size=(M, D)), types[1]) if dr else None
    note(f"rms_bwd {shape} {types} dr={dr}")
    a = [num(dy), num(r), num(w)]
    wx, ww = ref.rms_bwd(*a, None if g is None else num(g), 1e-5)
    dx, dw = gpu.ss_rms_bwd(dy, r, w, g, eps=1e-5)
    c = (np.square(a[1]).mean(-1, keepdims=True) + 1e-5) ** -0.5
    terms = np.abs(a[2] * a[0] * c) + np.abs(a[1]) * c ** 3 * np.abs(a[2] * a[0] * a[1]).mean(-1, keepdims=True)
    terms = terms + (0 if g is None else np.abs(num(g)))
    near(dx, wx, terms * 4 * eps_of(D) + (1.001 * 2.0 ** -8 * np.abs(wx) if types[1] == "bf16" else 0) + 1e-37, "dx")
    near(dw, ww, np.abs(a[0] * a[1] * c).sum(0) * (M * 2.0 ** -24 + 4 * eps_of(D)) + 1e-37, "dw")


def test_gradient_is_the_difference(gpu):
    """The oracle's gradient against central differences of its forward, in float64."""
    r = np.random.default_rng(3)
    x, res, w, dy, dr = (r.normal(size=s) for s in ((3, 11), (3, 11), 11, (3, 11), (3, 11)))

    def loss():
        y, s = ref.rms_fwd(x, w, res, 1e-3)
        return (y * dy).sum() + (s * dr).sum()
    dx, dw = ref.rms_bwd(dy, x + res, w, dr, 1e-3)
    for a, g in ((x, dx), (res, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + 1e-5
            up = loss()
            a[i] = keep - 1e-5
            down = loss()
            a[i] = keep
            assert abs((up - down) / 2e-5 - g[i]) < 1e-7


@pytest.mark.parametrize("D", [64, 2560, 9000])
def test_special_rows(gpu, D):
    """Rows of zeros, of the smallest magnitudes, and rows that hold NaN or infinities: each row
    for itself, the neighbours as without them."""
    import torch
    x, _, w = data(4, 6, D, ("f32", "f32"), False)
    note(f"rms special rows {D}")
    clean = gpu.ss_rms_fwd(x, w, eps=1e-5, q8=gpu.SS_Q8_FP8)
    z = x.clone()
    z[1] = 0.0
    z[2, 3] = float("nan")
    z[4] = 1e-38
    y8, sc = gpu.ss_rms_fwd(z, w, eps=1e-5, q8=gpu.SS_Q8_FP8)
    for i in (0, 3, 5):
        assert torch.equal(y8[i].float(), clean[0][i].float()) and sc[i] == clean[1][i]
    assert not y8[1].float().any() and sc[1] == 0
    assert torch.isnan(sc[2]) and torch.isnan(y8[2].float()).all()
    assert not torch.isnan(y8[4].float()).any() and torch.isfinite(sc[4])
    y = gpu.ss_rms_fwd(z, w, eps=1e-5)
    assert torch.isnan(y[2]).all() and not y[1].any()
    z[2, 3] = float("inf")
    y = gpu.ss_rms_fwd(z, w, eps=1e-5)
    # 1 / sqrt(inf) = 0: inf·0 is NaN, the rest 0
    assert torch.isnan(y[2, 3]) and not y[2, 4:].any() and torch.equal(y[0], gpu.ss_rms_fwd(x, w, eps=1e-5)[0])


def test_in_place_stream_and_graph(gpu):
    import torch
    x, rs, w = data(9, 1500, 2560, ("bf16", "bf16"), True)
    note("rms in place, stream, graph")
    y, r = gpu.ss_rms_fwd(x, w, rs)
    own = rs.clone()
    y2, r2 = gpu.ss_rms_fwd(x, w, own, r=own)
    assert r2 is own and torch.equal(y, y2) and torch.equal(r, own)
    dx, dw = gpu.ss_rms_bwd(y, r, w, rs)
    own = rs.clone()
    dx2, dw2 = gpu.ss_rms_bwd(y, r, w, own, dx=own)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, r3 = gpu.ss_rms_fwd(x, w, rs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and torch.equal(r, r3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.ss_rms_bwd(y, r, w, rs)
    for _ in range(3):
        out[0].zero_()
        out[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], dx) and torch.equal(out[1], dw)
        torch.randn(1 << 20, device="cuda").sum().item()


@pytest.mark.parametrize("D", [9, 76, 311, 918, 1025, 2563, 4099])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_in_place_where_rows_end_inside_a_piece(gpu, types, D):
    """The stream updated in place: every element read before it is written, also where two
    threads read it."""
    import torch
    x, rs, w = data(D, 1200, D, types, True)
    note(f"rms in place {types} {D}")
    y, r = gpu.ss_rms_fwd(x, w, rs)
    own = rs.clone()
    y2, _ = gpu.ss_rms_fwd(x, w, own, r=own)
    assert torch.equal(y, y2) and torch.equal(r, own)
    dx, dw = gpu.ss_rms_bwd(y, r, w, rs)
    own = rs.clone()
    dx2, dw2 = gpu.ss_rms_bwd(y, r, w, own, dx=own)
    assert torch.equal(dx, own) and dx2 is own and torch.equal(dw, dw2)


def test_refusals(gpu):
    import torch
    x, rs, w = data(10, 4, 64, ("bf16", "bf16"), True)
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x.half(), w)
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x, w.to(torch.bfloat16))
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x, w[:32])
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x, w, rs[:3])
    with pytest.raises(ValueError):
        gpu.ss_rms_fwd(x[:0], w)
    for bad in (dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(gpu.SSError) as e:
            gpu.ss_rms_fwd(x, w, **bad)
        assert e.value.code == -2
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_rms_fwd(x, w, q8=7)
    assert e.value.code == -3
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_rms_fwd(x.float(), w, rs)           # float32 rows on a bfloat16 residual
    assert e.value.code == -3
    wide = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_rms_fwd(wide, wide[0])
    assert e.value.code == -2
    flat = torch.zeros(1 + 4 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_rms_fwd(flat[1:].view(4, 64), w)    # off by one element
    assert e.value.code == -4
