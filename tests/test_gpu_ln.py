"""GPU parity of the layer norm (ss_ln_fwd, ss_ln_bwd) against the float64 oracle.

Tolerances of each element, in u = 2^-24.  A float32 sum of D terms in lanes and trees is off by at
most n·u of its absolute terms, n = D / 64 + 32.  With M = mean|r| and d = r - mean:
  d: q = n·u·M + 2u|r| + 2u·M;  the variance: 2·mean(|d| q) + q², and n·u of itself; its inverse root
  c half of that relative to it, and 4u;  y = d·c·w + b: |w|(c·q + |d c|(that + 4u)) and u(|y| + |b|).
  dx = c(wdy - S1 - n S2): S1, S2 within n·u of their absolute terms; n = d·c within N = c·q + |n|·rel;
  dw: N of every row times |dy| and (rows + 8)u of the absolute terms; db: (rows + 8)u of Σ|dy|.
bfloat16 results round once more: 2^-8.  8 bits: as for the RMS norm, half a step and the float32
error.  4-bit blocks: y is within E of the oracle's, so the block's codes are those of some value in
that range: checked against half a step (of the neighbouring codes' spacing at y) and E.
"""
import numpy as np
import pytest

from oracle import ln_mx4_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 96), (2, 511), (4, 512), (7, 513), (3, 1000), (1, 2048),
          (2, 2049), (1, 2560), (1100, 520), (1030, 1536), (1025, 2560), (2, 4099), (3, 8192),
          (2, 8200), (1, 16384), (1, 16416), (2, 20001), (1, 32768), (1200, 1471), (1030, 2563), (1100, 3001)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def hold(x, dt):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return (t.to(torch.bfloat16) if dt == "bf16" else t).cuda()


def num(t):
    return t.float().cpu().numpy().astype(np.float64)


def near(got, want, bound, what):
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    over = np.abs(got - want) - bound
    assert np.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()))


def data(seed, M, D, types, res, bias=True):
    r = np.random.default_rng(seed)
    x = hold(0.3 + r.normal(size=(M, D)), types[0])
    rs = hold(0.5 + 2 * r.normal(size=(M, D)), types[1]) if res else None
    w = hold(1 + 0.2 * r.normal(size=D), "f32")
    b = hold(0.3 * r.normal(size=D), "f32") if bias else None
    return x, rs, w, b


def parts(r, eps):
    """d, c, and the errors of d (q) and of c (relative)."""
    D = r.shape[-1]
    n = (D / 64 + 32) * U
    m = np.abs(r).mean(-1, keepdims=True)
    d = r - r.mean(-1, keepdims=True)
    q = n * m + 2 * U * np.abs(r) + 2 * U * m
    var = np.square(d).mean(-1, keepdims=True)
    evar = 2 * (np.abs(d) * q).mean(-1, keepdims=True) + np.square(q).mean(-1, keepdims=True) + n * var
    c = (var + eps) ** -0.5
    return d, c, q, evar * c * c / 2 * 1.01 + 4 * U


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(gpu, shape, types, res):
    import torch
    M, D = shape
    x, rs, w, b = data(M + D, M, D, types, res, bias=(M + D) % 3 != 0)
    note(f"ln_fwd {shape} {types} res={res}")
    wb = None if b is None else num(b)
    wy, wr = ref.ln_fwd(num(x), num(w), wb, None if rs is None else num(rs), 1e-5)
    out = gpu.ss_ln_fwd(x, w, b, rs, eps=1e-5)
    y, r = out if res else (out, None)
    d, c, q, ec = parts(wr, 1e-5)
    e = np.abs(num(w)) * (c * q + np.abs(d * c) * (ec + 4 * U)) + U * (np.abs(wy) + (0 if b is None else np.abs(wb)))
    near(y, wy, e + (1.001 * 2.0 ** -8 * np.abs(wy) if types[0] == "bf16" else 0) + 1e-37, "y")
    if res:
        near(r, wr, np.abs(wr) * (2.0 ** -23 + (1.001 * 2.0 ** -8 if types[1] == "bf16" else 0)), "r")
    for q8, top in ((gpu.SS_Q8_FP8, 448.0), (gpu.SS_Q8_INT8, 127.0)):
        out = gpu.ss_ln_fwd(x, w, b, rs, eps=1e-5, q8=q8)
        y8, sc = out[:2]
        ws = np.abs(wy).max(-1) / top
        es = e.max(-1) / top
        near(sc, ws, es + ws * 2.0 ** -22, "scale")
        s = num(sc)[:, None]
        half = np.maximum(np.abs(wy) * 2.0 ** -4, 2.0 ** -10 * s) if top == 448.0 else 0.5 * s
        near(y8.float() * sc[:, None], wy, half * 1.0001 + e * 1.1 + top * (es[:, None] + s * 2.0 ** -21), "codes")
        if res:
            assert torch.equal(out[2], r)
    if D % 32 == 0:
        codes, exps = gpu.ss_ln_fwd(x, w, b, rs, eps=1e-5, q8=gpu.SS_Q4_MX)[:2]
        assert codes.shape == (M, D // 2) and exps.shape == (M, D // 32)
        v = ref.mx4_values(ref.unpack(codes.cpu().numpy()), exps.cpu().numpy().astype(np.int64))
        p = np.repeat(2.0 ** (exps.cpu().numpy() - 127.0), 32, -1)
        # half a step: 1/4 below 2, 1/2 below 4, 1 below 6, and what 8 leaves to 6
        a = (np.abs(wy) + e) / p
        step = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, np.where(a <= 6, 1.0, np.maximum(1.0, a - 6))))
        assert (a < 8.0001 + e / p).all()
        assert (np.abs(v - wy) <= step * p + e + 1e-37).all()
        big = np.abs(wy).reshape(M, -1, 32).max(-1)
        eb = e.reshape(M, -1, 32).max(-1)
        es = 2.0 ** (exps.cpu().numpy() - 125.0)       # the block's largest is in [es, 2 es)
        assert ((big + eb >= es) & (big - eb < 2 * es) | (exps.cpu().numpy() == 1)).all()


@pytest.mark.parametrize("dr", [True, False])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(gpu, shape, types, dr):
    M, D = shape
    dy, r, w, _ = data(M + 3 * D, M, D, types, True)
    g = hold(np.random.default_rng(D).normal(size=(M, D)), types[1]) if dr else None
    note(f"ln_bwd {shape} {types} dr={dr}")
    a = [num(dy), num(r), num(w)]
    wx, ww, wb = ref.ln_bwd(*a, None if g is None else num(g), 1e-5)
    dx, dw, db = gpu.ss_ln_bwd(dy, r, w, g, eps=1e-5)
    d, c, q, ec = parts(a[1], 1e-5)
    nn, u = (D / 64 + 32) * U, np.abs(a[0] * a[2])
    N, h = np.abs(d * c), c * q + np.abs(d * c) * (ec + 2 * U)
    s1 = u.mean(-1, keepdims=True)
    s2 = (u * N).mean(-1, keepdims=True)
    e2 = (u * h).mean(-1, keepdims=True) + (nn + 8 * U) * s2
    ex = c * ((u + s1) * (ec + 8 * U) + nn * s1 + h * s2 + N * e2 + N * s2 * (2 * ec + 8 * U))
    ex = ex + (0 if g is None else 2 * U * (np.abs(num(g)) + np.abs(wx)))
    near(dx, wx, ex + (1.001 * 2.0 ** -8 * np.abs(wx) if types[1] == "bf16" else 0) + 1e-37, "dx")
    near(dw, ww, (np.abs(a[0]) * (h + (M + 8) * U * N)).sum(0) + 1e-37, "dw")
    near(db, wb, (M + 8) * U * np.abs(a[0]).sum(0) + 1e-37, "db")


@pytest.mark.parametrize("D", [64, 2560, 9024])
def test_special_rows(gpu, D):
    """Constant rows, rows far from 0, rows that hold NaN or infinities: each for itself."""
    import torch
    x, _, w, b = data(4, 6, D, ("f32", "f32"), False)
    note(f"ln special rows {D}")
    clean = gpu.ss_ln_fwd(x, w, b, eps=1e-5)
    z = x.clone()
    z[1] = 3.0
    z[2, 3] = float("nan")
    z[4] = 4096.0 + x[4].round()          # mean and differences exact in float32
    for q8 in (gpu.SS_Q8_NONE, gpu.SS_Q8_FP8, gpu.SS_Q4_MX):
        out = gpu.ss_ln_fwd(z, w, b, eps=1e-5, q8=q8)
        ref_out = gpu.ss_ln_fwd(x, w, b, eps=1e-5, q8=q8)
        for got, want in zip(out if q8 else (out,), ref_out if q8 else (ref_out,)):
            for i in (0, 3, 5):
                assert torch.equal(got[i].float(), want[i].float())
        if q8 == gpu.SS_Q4_MX:
            assert (out[1][2] == 255).all() and not out[0][2].any() and (out[1][1] != 255).all()
    y = gpu.ss_ln_fwd(z, w, b, eps=1e-5)
    assert torch.equal(y[0], clean[0])
    wy = ref.ln_fwd(num(z), num(w), num(b))[0]
    # the mean of a constant row is off by at most n·u of it, and c is at most 1/sqrt(eps)
    assert np.abs(num(y)[1] - num(b)).max() <= 3 * (D / 64 + 32) * U / 1e-5 ** 0.5 * 1.5
    assert torch.isnan(y[2]).all()
    d, c, q, ec = parts(num(z)[4:5], 1e-5)
    assert (np.abs(num(y)[4] - wy[4]) <= (np.abs(num(w)) * (c * q + np.abs(d * c) * (ec + 4 * U)) + 4 * U * (np.abs(wy[4:5]) + 1))[0]).all()


def test_in_place_stream_and_graph(gpu):
    import torch
    x, rs, w, b = data(9, 1500, 2560, ("bf16", "bf16"), True)
    note("ln in place, stream, graph")
    y, r = gpu.ss_ln_fwd(x, w, b, rs)
    own = rs.clone()
    y2, r2 = gpu.ss_ln_fwd(x, w, b, own, r=own)
    assert r2 is own and torch.equal(y, y2) and torch.equal(r, own)
    want = gpu.ss_ln_bwd(y, r, w, rs)
    own = rs.clone()
    got = gpu.ss_ln_bwd(y, r, w, own, dx=own)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    no = gpu.ss_ln_bwd(y, r, w, rs, bias=False)
    assert no[2] is None and torch.equal(no[0], want[0]) and torch.equal(no[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, r3 = gpu.ss_ln_fwd(x, w, b, rs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and torch.equal(r, r3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu.ss_ln_bwd(y, r, w, rs)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        torch.randn(1 << 20, device="cuda").sum().item()


@pytest.mark.parametrize("D", [9, 76, 311, 918, 1025, 2563, 4099])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_in_place_where_rows_end_inside_a_piece(gpu, types, D):
    import torch
    x, rs, w, b = data(D, 1200, D, types, True)
    note(f"ln in place {types} {D}")
    y, r = gpu.ss_ln_fwd(x, w, b, rs)
    own = rs.clone()
    y2, _ = gpu.ss_ln_fwd(x, w, b, own, r=own)
    assert torch.equal(y, y2) and torch.equal(r, own)
    want = gpu.ss_ln_bwd(y, r, w, rs)
    own = rs.clone()
    got = gpu.ss_ln_bwd(y, r, w, own, dx=own)
    assert torch.equal(want[0], own) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals(gpu):
    import torch
    x, rs, w, b = data(10, 4, 64, ("bf16", "bf16"), True)
    for bad in ((x.half(), w, b), (x, w.to(torch.bfloat16), b), (x, w[:32], b), (x, w, b[:32]),
                (x.t().contiguous().t(), w, b), (x, w, b, rs[:3]), (x[:0], w, b)):
        with pytest.raises(ValueError):
            gpu.ss_ln_fwd(*bad)
    with pytest.raises(ValueError):
        gpu.ss_ln_fwd(x[:, :40].contiguous(), w[:40].contiguous(), q8=gpu.SS_Q4_MX)
    for kw, code in ((dict(eps=-1.0), -2), (dict(eps=float("nan")), -2), (dict(q8=7), -3)):
        with pytest.raises(gpu.SSError) as e:
            gpu.ss_ln_fwd(x, w, b, **kw)
        assert e.value.code == code
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_ln_fwd(x.float(), w, b, rs)
    assert e.value.code == -3
    with pytest.raises(ValueError):
        gpu.ss_ln_bwd(x, rs, w, bias=False, db=torch.empty_like(w))
