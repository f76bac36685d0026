"""GPU parity of the gated recurrence (ss_gr_fwd, ss_gr_bwd, ss_gr_step) against the float64 oracle.

Tolerances of each element, in units of u = 2^-24 (a float32 rounding; a hardware exponential,
reciprocal or root counts two).
  σ(r): the exponent's argument rounds by |r|·u of itself, then 6 roundings: (|r| + 6)u.
  log a: σ's, 6 for softplus and 3 products: e = (|r| + 16)u of itself.  a: |log a|·e and 2u.
  s = sqrt(1 - a²): half of e and of 14u, and 2u.  s·v: that, |i| + 6 for σ(i), 2 products:
      E(r, i) = (|r|/2 + |i| + 26)u of |s v|.
  h: the recursion of these errors, E_t = a E_{t-1} + a|h_{t-1}|(|log a|e + 2u) + |s v|E, and 64u of
      Σ|terms| for the additions of a stretch and the joins of stretches (fewer than 64 on any
      path from a token's term to a state up to the stretches' own joins, whose errors decay with
      the terms).
  g likewise with dy exact.
  dx = g s σ(i): g's error and (|r|/2 + |i| + 34)u; di: the same and 2u·σ(i) of 1 - σ(i).
  ∂/∂log a = g(a h' - a²/s v): g's error over both terms, h's, and (|r| + |i| + 60)u of both;
  dr: times log a (1 - σ(r)), with 2u of σ's 1 - σ; dlam: the sum of the absolute errors, 16u for its
      factors and (16 + count)u of the absolute terms.
bfloat16 results round once more: 2^-8 of themselves.
"""
import numpy as np
import pytest

from oracle import gr_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def hold(x, dt):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return (t.to(torch.bfloat16) if dt == "bf16" else t).cuda()


def num(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(seed, B, T, D, dt, h0=True, lengths=False, reset=False, spread=1.5):
    r = np.random.default_rng(seed)
    p = {n: hold(spread * r.normal(size=(B, T, D)), dt) for n in ("x", "r", "i", "dy")}
    p["lam"] = hold(np.log(np.expm1(-np.log(0.9 + 0.099 * r.random(D)) / 8)), "f32")
    p["h0"] = hold(r.normal(size=(B, D)), "f32") if h0 else None
    p["dh"] = hold(r.normal(size=(B, D)), "f32") if h0 else None
    import torch
    n = r.integers(0, T + 1, size=B)
    p["lengths"] = torch.from_numpy(n.astype(np.int32)).cuda() if lengths else None
    p["reset"] = torch.from_numpy(r.random((B, T)) < 4.0 / (T + 4)).cuda() if reset else None
    return p


def oracle(p, c=8.0):
    """The oracle's values and the bounds of their errors, by name."""
    a64 = {n: None if p[n] is None else num(p[n]) for n in ("x", "r", "i", "dy", "lam", "h0", "dh")}
    kw = {n: None if p[n] is None else p[n].cpu().numpy() for n in ("lengths", "reset")}
    x, r, i, dy, lam, h0, dh = (a64[n] for n in ("x", "r", "i", "dy", "lam", "h0", "dh"))
    y, h = ref.fwd(x, r, i, lam, h0, c, **kw)
    g = ref.bwd(x, r, i, lam, dy, h0, dh, c, **kw)
    a, s, v, sr, si, la, x, live, first = ref.gates(x, r, i, lam, c, **kw)
    r, i = (np.where(live[..., None], t, 0.0) for t in (r, i))
    B, T, D = x.shape
    e = (np.abs(r) + 16) * U
    ea = np.abs(la) * e + 2 * U
    ev = (np.abs(r) / 2 + np.abs(i) + 26) * U
    sv = np.abs(s * v)
    A, E = np.zeros((B, T + 1, D)), np.zeros((B, T + 1, D))
    if h0 is not None:
        A[:, 0] = np.abs(h0)
    for t in range(T):
        A[:, t + 1] = a[:, t] * A[:, t] + sv[:, t]
        E[:, t + 1] = a[:, t] * (E[:, t] + A[:, t] * ea[:, t]) + sv[:, t] * ev[:, t]
    E += 64 * U * A
    G, F = np.zeros((B, T + 1, D)), np.zeros((B, T + 1, D))
    if dh is not None:
        G[:, T] = np.abs(dh)
    for t in reversed(range(T)):       # G[t + 1]: |g_t|'s terms; F its error
        G[:, t + 1] += np.where(live[:, t, None], np.abs(dy[:, t]), 0.0)
        G[:, t] = a[:, t] * G[:, t + 1]
        F[:, t] = a[:, t] * (F[:, t + 1] + G[:, t + 1] * ea[:, t])
    F += 64 * U * G
    g1, f1 = G[:, 1:], F[:, 1:]
    on = live[..., None]
    b = {"y": E[:, 1:], "h_final": E[:, T], "ckpt": E[:, :T:64]}
    w = s * si
    b["dx"] = on * w * (f1 + g1 * (np.abs(r) / 2 + np.abs(i) + 34) * U)
    b["di"] = np.abs(x) * (1 - si) * b["dx"] + on * w * g1 * np.abs(x) * 2 * U * (si + 1)
    with np.errstate(divide="ignore", invalid="ignore"):
        root = np.where(s > 1e-15, a * a / s, 0.0) * np.abs(v)
    both = a * A[:, :T] + root
    moves = on & ~first[..., None]
    edla = np.where(moves, f1 * both + g1 * (a * E[:, :T] + (np.abs(r) + np.abs(i) + 60) * U * both), 0.0)
    dla = np.where(moves, g1 * both, 0.0)
    b["dr"] = np.abs(la) * ((1 - sr) * edla + 2 * U * (1 + sr) * dla)
    k = c / (1 + np.exp(-lam))
    b["dlam"] = k * ((sr * edla).sum((0, 1)) + (16 + 16 + np.log2(B * T + 1) + B * T / 64) * U * (sr * dla).sum((0, 1)))
    b["dh0"] = F[:, 0]
    want = dict(g, y=y, h_final=h[:, T], ckpt=h[:, :T:64])
    return want, b


def near(got, want, bound, dt, what):
    got = num(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = bound * 1.01 + (1.01 * 2.0 ** -8 * np.abs(want) if dt == "bf16" else 0) + 1e-37
    over = np.abs(got - want) - tol
    assert np.isfinite(got).all() and (over <= 0).all(), (what, float(over.max()), float(np.abs(got - want).max()))


def run_all(gpu, p, dt, c=8.0, want=None):
    w, b = want or oracle(p, c)
    marks = dict(c=c, lengths=p["lengths"], reset=p["reset"])
    y, hf, ck = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"], return_final=True,
                              return_ckpt=True, **marks)
    near(y, w["y"], b["y"], dt, "y")
    near(hf, w["h_final"], b["h_final"], "f32", "h_final")
    near(ck, w["ckpt"], b["ckpt"], "f32", "ckpt")
    for given in (ck, None):
        g = gpu.ss_gr_bwd(p["x"], p["r"], p["i"], p["lam"], p["dy"], p["h0"], p["dh"], h_ckpt=given, **marks)
        for n in ("dx", "dr", "di"):
            near(g[n], w[n], b[n], dt, n)
        near(g["dlam"], w["dlam"], b["dlam"], "f32", "dlam")
        if p["h0"] is not None:
            near(g["dh0"], w["dh0"], b["dh0"], "f32", "dh0")
        else:
            assert g["dh0"] is None
    return y, hf, ck, g


SHAPES = [(1, 1, 1), (2, 1, 130), (1, 2, 2), (3, 15, 7), (2, 16, 64), (1, 17, 63), (2, 63, 75),
          (1, 64, 128), (2, 65, 129), (1, 127, 256), (1, 128, 200), (2, 129, 66), (1, 300, 131),
          (2, 513, 34), (1, 1500, 10)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("marks", ["none", "lengths", "reset", "both"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_whole(gpu, shape, marks, dt):
    note(f"gr {shape} {marks} {dt}")
    p = make(sum(shape), *shape, dt, h0=marks != "none", lengths=marks in ("lengths", "both"),
             reset=marks in ("reset", "both"))
    run_all(gpu, p, dt)


@pytest.mark.parametrize("shape", [(1, 5000, 9), (2, 9000, 3), (1, 4096, 128), (1, 4097, 2), (1, 2048, 6), (3, 8321, 4)], ids=str)
def test_long(gpu, shape):
    note(f"gr long {shape}")
    run_all(gpu, make(7, *shape, "f32", reset=shape[2] == 3), "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 1, 75), (1, 1, 128), (5, 1, 130), (70, 1, 256)], ids=str)
def test_step(gpu, shape, dt):
    import torch
    note(f"gr step {shape} {dt}")
    p = make(3 + sum(shape), *shape, dt)
    w, b = oracle(p)
    x, r, i = (p[n][:, 0] for n in "xri")
    h = p["h0"].clone()
    y = gpu.ss_gr_step(x, r, i, p["lam"], h)
    near(y, w["y"][:, 0], b["y"][:, 0], dt, "y")
    near(h, w["h_final"], b["h_final"], "f32", "h")
    out = torch.empty_like(h)
    keep = p["h0"].clone()
    y2 = gpu.ss_gr_step(x, r, i, p["lam"], keep, h_out=out)
    assert torch.equal(y, y2) and torch.equal(out, h) and torch.equal(keep, p["h0"])


def test_steps_continue_a_prompt(gpu):
    """A text in one call, in two (the state in place), and its last tokens one by one: the same
    values but for float32 roundings (64 of them at most on a path, by what the state's terms are)."""
    p = make(5, 2, 200, 96, "f32")
    w, b = oracle(p)
    x, r, i, lam = (p[n] for n in ("x", "r", "i", "lam"))
    y1, h = gpu.ss_gr_fwd(x[:, :150], r[:, :150], i[:, :150], lam, p["h0"], return_final=True)
    y2, h2 = gpu.ss_gr_fwd(x[:, 150:190], r[:, 150:190], i[:, 150:190], lam, h, h_final=h)
    assert h2 is h
    near(y1, w["y"][:, :150], b["y"][:, :150], "f32", "first")
    near(y2, w["y"][:, 150:190], 2 * b["y"][:, 150:190], "f32", "second")
    for t in range(190, 200):
        y = gpu.ss_gr_step(x[:, t], r[:, t], i[:, t], lam, h)
        near(y, w["y"][:, t], 3 * b["y"][:, t], "f32", f"token {t}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 75, 128])
def test_strides(gpu, D, dt):
    """Slices of one projection (odd offsets among them), transposed batches, expanded rows and
    overlapping windows give the bits of dense copies."""
    import torch
    note(f"gr strides {D} {dt}")
    T, B = 90, 2
    wide = hold(np.random.default_rng(D).normal(size=(B, T, 3 * D + 5)), dt)
    lam = make(1, 1, 1, D, dt)["lam"]
    flat = hold(np.random.default_rng(1).normal(size=(B * T * D + 64,)), dt)
    sets = {
        "fused": [wide[..., o:o + D] for o in (0, D, 2 * D)],
        "odd": [wide[..., o:o + D] for o in (1, D + 3, 2 * D + 5)],
        "turned": [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (wide[..., :D], wide[..., 2:D + 2], wide[..., 4:D + 4])],
        "expanded": [wide[:, :1, :D].expand(B, T, D), wide[:1, :, 1:D + 1].expand(B, T, D), wide[..., :D]],
        "windows": [flat.as_strided((B, T, D), (T, 2, 1)), flat.as_strided((B, T, D), (7, 1, 1), 3), wide[..., :D]],
    }
    dy = hold(np.random.default_rng(2).normal(size=(B, T, D)), dt)
    for name, (x, r, i) in sets.items():
        y = gpu.ss_gr_fwd(x, r, i, lam)
        g = gpu.ss_gr_bwd(x, r, i, lam, dy)
        dense = [t.contiguous().clone() for t in (x, r, i)]
        assert torch.equal(y, gpu.ss_gr_fwd(*dense, lam)), name
        d = gpu.ss_gr_bwd(*dense, lam, dy)
        for n in ("dx", "dr", "di", "dlam"):
            assert torch.equal(g[n], d[n]), (name, n)
    s = [t[:, 3] for t in sets["odd"]]
    h, h2 = torch.ones(B, D, device="cuda"), torch.ones(B, D, device="cuda")
    assert torch.equal(gpu.ss_gr_step(*s, lam, h), gpu.ss_gr_step(*[t.contiguous() for t in s], lam, h2))
    assert torch.equal(h, h2)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_what_stands_behind_a_text_is_not_used(gpu, dt):
    import torch
    note(f"gr behind a text {dt}")
    B, T, D = 4, 150, 96
    p = make(11, B, T, D, dt, reset=True)
    p["lengths"] = torch.tensor([0, 1, 70, 150], dtype=torch.int32, device="cuda")
    clean = run_all(gpu, p, dt)
    q = dict(p)
    for n in ("x", "r", "i", "dy"):
        q[n] = p[n].clone()
        for b, m in enumerate((0, 1, 70, 150)):
            q[n][b, m:] = float("nan") if b % 2 else float("inf")
    marks = dict(lengths=p["lengths"], reset=p["reset"])
    y, hf, ck = gpu.ss_gr_fwd(q["x"], q["r"], q["i"], p["lam"], p["h0"], return_final=True, return_ckpt=True, **marks)
    g = gpu.ss_gr_bwd(q["x"], q["r"], q["i"], p["lam"], q["dy"], p["h0"], p["dh"], h_ckpt=ck, **marks)
    for got, want in zip((y, hf, ck), clean):
        assert torch.equal(got, want)
    for n, t in clean[3].items():
        assert torch.equal(g[n], t), n
    assert torch.equal(hf[0], p["h0"][0]) and torch.equal(g["dh0"][0], p["dh"][0])
    assert not y[0].any() and not y[1, 1:].any() and not g["dx"][0].any() and not g["dr"][2, 70:].any()
    # lengths outside [0, T] count as the ends
    out = torch.tensor([-5, 1, 70, 9999], dtype=torch.int32, device="cuda")
    assert torch.equal(gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"], lengths=out, reset=p["reset"]), y)


def test_documents_do_not_see_each_other(gpu):
    """NaN and infinities of one document stay in it, forward and backward."""
    import torch
    T, D = 400, 70
    p = make(12, 1, T, D, "f32")
    starts = [0, 1, 130, 131, 200, 320]
    reset = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    reset[0, starts] = 7
    p["reset"] = reset
    args = lambda q: (q["x"], q["r"], q["i"], p["lam"])  # noqa: E731
    y = gpu.ss_gr_fwd(*args(p), p["h0"], reset=reset)
    g = gpu.ss_gr_bwd(*args(p), p["dy"], p["h0"], p["dh"], reset=reset)
    q = {n: p[n].clone() for n in ("x", "r", "i", "dy")}
    q["x"][0, 150] = float("nan")
    q["r"][0, 220] = float("nan")
    q["dy"][0, 250] = float("inf")
    y2 = gpu.ss_gr_fwd(*args(q), p["h0"], reset=reset)
    g2 = gpu.ss_gr_bwd(*args(q), q["dy"], p["h0"], p["dh"], reset=reset)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[131:200] = bad[200:320] = True
    assert torch.equal(y[0, ~bad], y2[0, ~bad]) and torch.isnan(y2[0, 150:200]).all()
    assert torch.isnan(y2[0, 220:320]).all()
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][0, ~bad], g2[n][0, ~bad]), n
    assert torch.equal(g["dh0"], g2["dh0"])


@pytest.mark.parametrize("gap", [1, 3, 20, 140])
def test_nan_gates_end_with_their_document(gpu, gap):
    """A NaN of the decay's gate shortly before the next document: in the same wave, the same tile,
    the tile before.  And one shortly behind a document's begin, for the adjoint."""
    import torch
    T, D = 600, 5
    p = make(21, 1, T, D, "f32")
    reset = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    cut = 296
    reset[0, cut] = True
    args = (p["x"], p["r"], p["i"], p["lam"])
    y = gpu.ss_gr_fwd(*args, p["h0"], reset=reset)
    g = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], p["dh"], reset=reset)
    for at, fine in ((cut - gap, slice(cut, T)), (cut + gap, slice(0, cut))):
        r = p["r"].clone()
        r[0, at] = float("nan")
        y2 = gpu.ss_gr_fwd(p["x"], r, p["i"], p["lam"], p["h0"], reset=reset)
        g2 = gpu.ss_gr_bwd(p["x"], r, p["i"], p["lam"], p["dy"], p["h0"], p["dh"], reset=reset)
        assert torch.equal(y[0, fine], y2[0, fine])
        for n in ("dx", "dr", "di"):
            assert torch.equal(g[n][0, fine], g2[n][0, fine]), n
        assert torch.isnan(y2[0, at]).all()


def test_extreme_gates(gpu):
    """Gates far out, rates near 0 and large: the oracle's values, finite gradients."""
    import torch
    T, D = 40, 8
    p = make(13, 1, T, D, "f32")
    p["r"] = hold(np.linspace(-80, 80, T)[None, :, None] + np.zeros((1, T, D)), "f32")
    p["i"] = hold(np.linspace(90, -90, T)[None, :, None] + np.zeros((1, T, D)), "f32")
    p["lam"] = hold(np.array([-60.0, -20.0, -8.0, -2.0, 0.0, 3.0, 20.0, 80.0]), "f32")
    w, b = oracle(p)
    y, hf = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"], return_final=True)
    # where log a leaves float32's normal range it is taken as 0: a change of the state of sqrt(2^-126)
    near(y, w["y"], b["y"] + 2.0 ** -58, "f32", "y")
    g = gpu.ss_gr_bwd(p["x"], p["r"], p["i"], p["lam"], p["dy"], p["h0"], p["dh"])
    for n, t in g.items():
        assert torch.isfinite(t).all(), n
    near(g["dx"], w["dx"], b["dx"] + 2.0 ** -58 * 100, "f32", "dx")
    near(g["dr"], w["dr"], b["dr"] + 1e-13, "f32", "dr")


def test_stream_graph_and_repeat(gpu):
    """Another stream; a captured forward and backward replayed with eager work in between; the same
    bits every time."""
    import torch
    note("gr stream, graph")
    p = make(14, 2, 1300, 200, "bf16", lengths=True, reset=True)
    marks = dict(lengths=p["lengths"], reset=p["reset"])
    args = (p["x"], p["r"], p["i"], p["lam"])

    def both():
        y, hf, ck = gpu.ss_gr_fwd(*args, p["h0"], return_final=True, return_ckpt=True, **marks)
        g = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], p["dh"], h_ckpt=ck, **marks)
        return [y, hf, ck] + [g[n] for n in sorted(g)]
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gpu.ss_gr_fwd(*args, p["h0"], stream=side, **marks)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        torch.randn(1 << 20, device="cuda").sum().item()


def test_in_place(gpu):
    import torch
    p = make(15, 2, 700, 150, "f32")
    args = (p["x"], p["r"], p["i"], p["lam"])
    y, hf = gpu.ss_gr_fwd(*args, p["h0"], return_final=True)
    g = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], p["dh"])
    own = p["h0"].clone()
    y2, h2 = gpu.ss_gr_fwd(*args, own, h_final=own)
    assert h2 is own and torch.equal(own, hf) and torch.equal(y, y2)
    own = p["dh"].clone()
    g2 = gpu.ss_gr_bwd(*args, p["dy"], p["h0"], own, out={"dh0": own})
    assert g2["dh0"] is own
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_two_calls_at_once(gpu):
    """Two streams, each with workspaces of its own."""
    import torch
    a, b = make(16, 4, 3000, 256, "bf16"), make(17, 2, 5000, 130, "bf16")
    args = lambda p: (p["x"], p["r"], p["i"], p["lam"], p["h0"])  # noqa: E731
    ya, yb = gpu.ss_gr_fwd(*args(a)), gpu.ss_gr_fwd(*args(b))
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append((gpu.ss_gr_fwd(*args(a), stream=s), gpu.ss_gr_fwd(*args(b), stream=t)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, ya) and torch.equal(y, yb)


def test_refusals(gpu):
    import torch
    p = make(18, 2, 10, 64, "bf16")
    x, r, i, lam = (p[n] for n in ("x", "r", "i", "lam"))
    for bad in ((x.half(), r, i), (x, r.float(), i), (x, r, i[:1]), (x.transpose(1, 2), r, i),
                (x[:, :0], r[:, :0], i[:, :0]), (x[0], r[0], i[0]), (x[:1, :1].expand(2, 10, 64), r, i)):
        with pytest.raises(ValueError):
            gpu.ss_gr_fwd(*bad, lam)
    with pytest.raises(ValueError):
        gpu.ss_gr_fwd(x, r, i, lam.to(torch.bfloat16))
    with pytest.raises(ValueError):
        gpu.ss_gr_fwd(x, r, i, lam, p["h0"][:1])
    with pytest.raises(ValueError):
        gpu.ss_gr_fwd(x, r, i, lam, lengths=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        gpu.ss_gr_fwd(x, r, i, lam, reset=torch.zeros(2, 10, device="cuda"))
    with pytest.raises(ValueError):
        gpu.ss_gr_bwd(x, r, i, lam, p["dy"][:, :5])
    with pytest.raises(TypeError):
        gpu.ss_gr_fwd(None, r, i, lam)
    for c in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gpu.SSError) as e:
            gpu.ss_gr_fwd(x, r, i, lam, c=c)
        assert e.value.code == -2
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_gr_bwd(x, r, i, lam, p["dy"], workspace=small)
    assert e.value.code == -5


def test_far_strides(gpu):
    """Single tokens out of long texts: with one token its stride says nothing, however far the rows are
    apart (here 2^26 elements)."""
    import torch
    B, D, far = 2, 130, 1 << 26
    flat = torch.randn((B - 1) * far + 3 * D, device="cuda", dtype=torch.bfloat16)
    x, r, i = (flat.as_strided((B, D), (far, 1), o) for o in (0, D, 2 * D))
    lam = make(1, 1, 1, D, "f32")["lam"]
    h, h2 = torch.ones(B, D, device="cuda"), torch.ones(B, D, device="cuda")
    y = gpu.ss_gr_step(x, r, i, lam, h)
    dense = [t.contiguous() for t in (x, r, i)]
    assert torch.equal(y, gpu.ss_gr_step(*dense, lam, h2)) and torch.equal(h, h2)
    one = [t[:, None] for t in (x, r, i)]
    y3 = gpu.ss_gr_fwd(*one, lam, torch.ones(B, D, device="cuda"))
    assert torch.equal(y3, gpu.ss_gr_fwd(*[t[:, None] for t in dense], lam, torch.ones(B, D, device="cuda")))
    with pytest.raises(gpu.SSError) as e:      # two tokens that far apart are refused
        t = flat.as_strided((1, 2, D), (1, far, 1))
        gpu.ss_gr_fwd(t, t, t, lam)
    assert e.value.code == -2


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(700, 40, 130), (600, 65, 200), (2100, 128, 33), (5000, 3, 20), (300, 32, 257)], ids=str)
def test_many_short_texts(gpu, shape, dt):
    note(f"gr many short {shape} {dt}")
    run_all(gpu, make(sum(shape), *shape, dt, lengths=True, reset=True), dt)


@pytest.mark.parametrize("T,st", [(2, 1 << 25), (2, 1 << 24), (9, 1 << 23), (9, 1 << 24), (30, 1 << 22), (32, 1 << 23)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_wide_steps_from_token_to_token(gpu, T, st, dt):
    import torch
    D = 70
    note(f"gr steps {T} {st} {dt}")
    flat = torch.zeros((T - 1) * st + 3 * D, device="cuda", dtype=torch.float32 if dt == "f32" else torch.bfloat16)
    own = [flat.as_strided((1, T, D), (0, st, 1), o) for o in (0, D, 2 * D)]
    p = make(T, 1, T, D, dt, h0=False)
    for a, b in zip(own, (p["x"], p["r"], p["i"])):
        a.copy_(b)
    want = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"])
    got = gpu.ss_gr_fwd(*own, p["lam"])
    w, b = oracle(p)
    gr = gpu.ss_gr_bwd(*own, p["lam"], p["dy"])
    near(got, w["y"], b["y"], dt, "y")
    near(want, w["y"], b["y"], dt, "y")
    near(gr["dx"], w["dx"], b["dx"], dt, "dx")


def test_short_texts_equal_single_tokens(gpu):
    import torch
    p = make(3, 5, 30, 200, "bf16")
    y, h = gpu.ss_gr_fwd(p["x"], p["r"], p["i"], p["lam"], p["h0"], return_final=True)
    own = p["h0"].clone()
    for t in range(30):
        yt = gpu.ss_gr_step(p["x"][:, t], p["r"][:, t], p["i"][:, t], p["lam"], own)
        assert torch.equal(yt, y[:, t])
    assert torch.equal(own, h)


def test_graphs_that_share_a_workspace(gpu):
    """Two captured calls of different sizes and an eager one take turns on one workspace, whatever the one
    before left in it."""
    import torch
    note("gr shared workspace")
    a, b = make(21, 2, 1500, 130, "bf16", reset=True), make(22, 3, 700, 260, "f32")
    args = lambda p: (p["x"], p["r"], p["i"], p["lam"])  # noqa: E731

    def fwd(ws):
        return gpu.ss_gr_fwd(*args(a), a["h0"], reset=a["reset"], workspace=ws)

    def bwd(ws):
        g = gpu.ss_gr_bwd(*args(b), b["dy"], b["h0"], b["dh"], workspace=ws)
        return [g[n] for n in sorted(g)]
    want_y, want_g = fwd(None), bwd(None)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        y = fwd(ws)
    with torch.cuda.graph(two):
        g = bwd(ws)
    for n in range(5):
        ws.fill_((0, 255, 1, 128, 77)[n])
        for graph in ((one, two), (two, one, one), (two, two, one))[n % 3]:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and all(torch.equal(s, t) for s, t in zip(g, want_g))
        y.zero_()
        one.replay()
        assert torch.equal(fwd(ws), want_y)
        torch.cuda.synchronize()
        assert torch.equal(y, want_y)


@pytest.mark.parametrize("shape", [(1, 2100, 40), (1, 4200, 200), (2, 2049, 10), (1, 6500, 129)], ids=str)
def test_long_rows_of_few_channels(gpu, shape):
    """Gradients whose chain has groups of 32 tiles: one or two columns of workgroups."""
    note(f"gr few channels {shape}")
    run_all(gpu, make(31, *shape, "bf16", reset=True), "bf16")
    run_all(gpu, make(32, *shape, "f32"), "f32")


@pytest.mark.parametrize("D", [1, 2, 3, 64, 127, 128, 129, 130, 255, 257])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_that_start_anywhere(gpu, dt, D):
    """Slices of wider rows, an odd number of elements apart and from the memory's beginning on; what stands
    between them stays as it is and is not taken in."""
    import torch
    note(f"gr anywhere {dt} {D}")
    for T in (5, 150):
        p = make(D + T, 2, T, D, dt, lengths=True, reset=True)
        for n, (before, after) in {"x": (1, 2), "r": (3, 1), "i": (2, 2 + D % 2)}.items():
            wide = torch.full((2, T, before + D + after), float("nan"), device="cuda", dtype=p[n].dtype)
            wide[..., before:before + D] = p[n]
            p[n] = wide[..., before:before + D]
        run_all(gpu, p, dt)
        h, g = p["h0"].clone(), p["h0"].clone()
        args = [p[n][:, 0] for n in ("x", "r", "i")]
        assert torch.equal(gpu.ss_gr_step(*args, p["lam"], h), gpu.ss_gr_step(*[t.contiguous() for t in args], p["lam"], g))
        assert torch.equal(h, g) and torch.isfinite(h).all()
