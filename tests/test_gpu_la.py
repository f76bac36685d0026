"""GPU parity of linear attention (ss_la_fwd, ss_la_bwd, ss_la_step) against the float64 oracle.

Tolerances are bounds of each element, from the sums of absolute values that the same formulas
give (|q|, |k|, |v|, |s0| ... in place of q, k, v, s0): with A such a sum,
  float32      a result is at most n roundings of 2^-24 of its terms off, n the number of
               additions and products on the longest path: the width of one product (<= 256),
               the tokens of a chunk, one rescaling a chunk, and 16 for the weights
  bfloat16     scores and states are rounded to 8 significant bits (at most 2^-8 of each)
               where they feed o, dq, dk, dv: 2^-8 of A together, each pair being in one of the
               two parts; and the result once, 2^-8 of it: at most 2^-7 of A, and 1/16 of that
               for the rest
  state, dS_0, dg   float32 for either type
dg is a running sum of row and column sums, so its A is theirs summed from the end.
"""
import numpy as np
import pytest

from oracle import la_ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def make(seed, B, T, H, Hk, dk, dv, dtype, decay, s0, lengths=None, hard=False):
    """float32 numpy inputs whose values the dtype holds exactly."""
    import torch
    r = np.random.default_rng(seed)
    hold = lambda x: torch.from_numpy(x.astype(np.float32)).to(  # noqa: E731
        torch.bfloat16 if dtype == "bf16" else torch.float32).float().numpy()
    c = dict(q=hold(r.normal(size=(B, T, Hk, dk))), k=hold(r.normal(size=(B, T, Hk, dk))),
             v=hold(r.normal(size=(B, T, H, dv))), do=hold(r.normal(size=(B, T, H, dv))),
             s0=r.normal(size=(B, H, dk, dv)).astype(np.float32) if s0 else None,
             ds=r.normal(size=(B, H, dk, dv)).astype(np.float32) if s0 else None,
             scale=float(dk) ** -0.5, lengths=lengths, dtype=dtype)
    rate = np.exp(r.uniform(-6, 1, size=H))
    g = {"token": -rate * r.exponential(size=(B, T, H)), "head": -rate, "none": None}[decay]
    if hard and decay == "token":
        # cuts, no decay at all, the lowest float32, and steps that underflow
        pick = r.integers(0, 8, size=g.shape)
        g = np.where(pick == 0, -np.inf, np.where(pick == 1, 0.0, np.where(
            pick == 2, np.finfo(np.float32).min, np.where(pick == 3, -200.0, g))))
    c["g"] = None if g is None else g.astype(np.float32)
    return c


def dev(c):
    import torch
    t = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    out = {n: None if c[n] is None else torch.from_numpy(c[n]).cuda() for n in ("g", "s0", "ds")}
    out.update({n: torch.from_numpy(c[n]).to(t).cuda() for n in ("q", "k", "v", "do")})
    out["lengths"] = None if c["lengths"] is None else torch.tensor(c["lengths"], dtype=torch.int32).cuda()
    return out


def near(got, want, bound, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}{at}: {got[at]} against {want[at]}, bound {bound[at]:.3e}"


def units(c):
    """n·2^-24 of the float32 sums."""
    T, dk, dv = c["v"].shape[1], c["q"].shape[-1], c["v"].shape[-1]
    return (max(dk, dv) + 64 + T // 32 + 16) * 2.0 ** -24


def absolute(c):
    return {n: None if c[n] is None else np.abs(c[n]) for n in ("q", "k", "v", "do", "s0", "ds")}


def out_bound(c, A):
    return A * (2.0 ** -7 * (17 / 16) if c["dtype"] == "bf16" else units(c)) + 1e-37


def check_fwd(c, o, s):
    a = absolute(c)
    wo, ws = la_ref.fwd(c["q"], c["k"], c["v"], c["g"], c["s0"], c["scale"], c["lengths"])
    Ao, As = la_ref.fwd(a["q"], a["k"], a["v"], c["g"], a["s0"], c["scale"], c["lengths"])
    near(o, wo, out_bound(c, Ao), "o")
    near(s, ws, As * units(c) + 1e-37, "s_final")


def check_bwd(c, got):
    a = absolute(c)
    args = (c["scale"], c["lengths"])
    w = la_ref.bwd(c["q"], c["k"], c["v"], c["do"], c["g"], c["s0"], c["ds"], *args)
    A = la_ref.bwd(a["q"], a["k"], a["v"], a["do"], c["g"], a["s0"], a["ds"], *args)
    for n in ("dq", "dk", "dv"):
        near(got[n], w[n], out_bound(c, A[n]), n)
    if c["s0"] is None:
        assert got["ds0"] is None
    else:
        near(got["ds0"], w["ds0"], A["ds0"] * units(c) + 1e-37, "ds0")
    if c["g"] is None:
        assert got["dg"] is None
        return
    # row and column sums of each value head, from the end
    rep = c["v"].shape[2] // c["q"].shape[2]
    wide = lambda x: np.repeat(x, rep, axis=2)  # noqa: E731
    full = la_ref.bwd(wide(a["q"]), wide(a["k"]), a["v"], a["do"], c["g"], a["s0"], a["ds"], *args)
    live = np.ones(c["v"].shape[:2], bool)
    if c["lengths"] is not None:
        live = np.arange(live.shape[1])[None] < np.array(c["lengths"])[:, None]
    sums = (wide(a["q"]) * full["dq"] + wide(a["k"]) * full["dk"]).sum(-1) * live[..., None]
    run = np.cumsum(sums[:, ::-1], 1)[:, ::-1]
    if c["ds"] is not None:
        _, last = la_ref.fwd(wide(a["q"]), wide(a["k"]), a["v"], c["g"], a["s0"], *args)
        run = run + (np.abs(c["ds"]) * last).sum((-1, -2))[:, None]
    run = run * live[..., None]
    if c["g"].ndim == 1:
        run = run.sum((0, 1))
    near(got["dg"], w["dg"], run * units(c) + 1e-37, "dg")


def run_fwd(ss, c, **kw):
    import torch
    t = dev(c)
    o, s = ss.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], t["s0"], scale=c["scale"],
                        lengths=t["lengths"], return_final=True, **kw)
    torch.cuda.synchronize()
    return o, s


def run_bwd(ss, c, **kw):
    import torch
    t = dev(c)
    r = ss.ss_la_bwd(t["q"], t["k"], t["v"], t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"],
                     lengths=t["lengths"], **kw)
    torch.cuda.synchronize()
    return r


CASES = [
    # B, T, H, Hk, dk, dv, decay, s0, lengths
    (1, 1, 1, 1, 1, 1, "token", True, None),
    (2, 1, 3, 1, 16, 16, "token", False, None),
    (1, 2, 2, 2, 8, 24, "head", True, None),
    (2, 31, 2, 1, 17, 5, "token", True, None),
    (1, 32, 2, 2, 64, 64, "token", False, None),
    (1, 33, 4, 2, 64, 128, "token", True, None),
    (2, 63, 2, 2, 128, 64, "none", True, None),
    (1, 64, 3, 3, 128, 128, "token", True, None),
    (2, 65, 2, 1, 100, 128, "token", True, None),
    (1, 127, 2, 2, 48, 36, "head", False, None),
    (1, 129, 1, 1, 256, 256, "token", True, None),
    (1, 200, 2, 2, 192, 40, "token", True, None),
    (1, 130, 2, 2, 40, 200, "token", True, None),
    (4, 203, 6, 2, 24, 40, "token", True, [0, 1, 203, 96]),
    (3, 300, 5, 1, 64, 64, "head", True, [300, 64, 299]),
    (1, 1000, 2, 2, 32, 80, "token", True, None),
    (2, 777, 3, 3, 128, 128, "token", True, [700, 128]),
]
IDS = ["B{}T{}H{}:{}k{}v{}-{}-s{:d}{}".format(*c[:8], "-ragged" if c[8] else "") for c in CASES]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(gpu, case, dtype):
    B, T, H, Hk, dk, dv, decay, s0, n = case
    c = make(31 + T, B, T, H, Hk, dk, dv, dtype, decay, s0, n)
    note(f"la_fwd {case} {dtype}")
    check_fwd(c, *run_fwd(gpu, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(gpu, case, dtype):
    B, T, H, Hk, dk, dv, decay, s0, n = case
    c = make(57 + T, B, T, H, Hk, dk, dv, dtype, decay, s0, n)
    note(f"la_bwd {case} {dtype}")
    check_bwd(c, run_bwd(gpu, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 700, 4, 2, 64, 128), (1, 500, 2, 2, 200, 72)])
def test_segments_without_decays(gpu, shape, dtype):
    """Several segments and no decays: dq and dk one launch each."""
    c = make(23, *shape, dtype, "none", True)
    note(f"la segments without decays {shape} {dtype}")
    check_fwd(c, *run_fwd(gpu, c))
    check_bwd(c, run_bwd(gpu, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("odd", ["q", "k", "v"])
def test_one_operand_off_its_alignment(gpu, odd, dtype):
    """One of q, k, v in rows that start anywhere, the others on 16 bytes, over segments."""
    import torch
    c = make(24, 2, 330, 2, 1, 64, 128, dtype, "token", True)
    t = dev(c)
    x = t[odd]
    wide = torch.full((*x.shape[:3], x.shape[3] + 3), float("nan"), dtype=x.dtype, device=x.device)
    wide[..., 1:-2] = x
    t[odd] = wide[..., 1:-2]
    note(f"la {odd} off its alignment {dtype}")
    o, last = gpu.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], t["s0"], scale=c["scale"], return_final=True)
    check_fwd(c, o, last)
    check_bwd(c, gpu.ss_la_bwd(t["q"], t["k"], t["v"], t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_hard_decays(gpu, dtype):
    """Cuts (-inf, the lowest float32), no decay and underflowing steps inside every chunk."""
    c = make(5, 2, 261, 4, 2, 32, 48, dtype, "token", True, None, hard=True)
    note(f"la hard decays {dtype}")
    check_fwd(c, *run_fwd(gpu, c))
    check_bwd(c, run_bwd(gpu, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_decay_is_exact(gpu, dtype):
    """After 20000 steps of e^-1 nothing of the running sum's size may show in later weights."""
    c = make(6, 1, 700, 1, 1, 16, 16, dtype, "token", True)
    c["g"][:, :200] = -100.0
    c["g"][:, 200:] = -0.01
    note(f"la far decay {dtype}")
    check_fwd(c, *run_fwd(gpu, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_behind_the_end_is_not_read_as_values(gpu, dtype):
    """NaN and infinities behind a row's length reach no output and no gradient."""
    import torch
    n = [70, 0, 133]
    c = make(7, 3, 133, 4, 2, 40, 24, dtype, "token", True, n)
    note(f"la behind the end {dtype}")
    clean_f, clean_b = run_fwd(gpu, c), run_bwd(gpu, c)
    for b, m in enumerate(n):
        for i, x in enumerate((c["q"], c["k"], c["v"], c["do"], c["g"])):
            x[b, m:] = (np.nan, np.inf, -np.inf, np.nan, np.nan)[i]
    f, g = run_fwd(gpu, c), run_bwd(gpu, c)
    for x, y in zip(f, clean_f):
        assert torch.equal(x, y)
    for name in g:
        assert torch.equal(g[name], clean_b[name]), name
    assert not f[0][1].any() and not f[0][0, 70:].any() and torch.equal(f[1][1].cpu(), torch.from_numpy(c["s0"][1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_reaches_no_earlier_one(gpu, dtype, bad):
    """v not finite at one token and column: o stays as it is before that token and beside that
    column; and dv stays as it is behind a token whose do is not finite."""
    c = make(8, 1, 96, 2, 1, 32, 40, dtype, "token", True)
    note(f"la bad token {dtype} {bad}")
    o, s = run_fwd(gpu, c)
    d = run_bwd(gpu, c)
    t, h, j = 45, 1, 7
    c["v"][0, t, h, j] = bad
    o2, s2 = run_fwd(gpu, c)
    c["v"][0, t, h, j] = 0.0
    keep = np.ones(o.shape, bool)
    keep[0, t:, h, j] = False
    o, o2 = o.float().cpu().numpy(), o2.float().cpu().numpy()
    # what the mask leaves is summed in another order where the chunk is formed again: the
    # bound of the plain case holds for both
    a = absolute(c)
    A, _ = la_ref.fwd(a["q"], a["k"], a["v"], c["g"], a["s0"], c["scale"])
    assert (np.abs(o2 - o)[keep] <= 2 * out_bound(c, A)[keep]).all()
    assert not np.isfinite(o2[0, t, h, j])
    keep = np.ones(s.shape, bool)
    keep[0, h, :, j] = False
    # the state's other columns see a zero in place of v[t, h, j] of another column: unchanged
    assert np.array_equal(s.cpu().numpy()[keep], s2.cpu().numpy()[keep])
    assert not np.isfinite(s2.cpu().numpy()[0, h, :, j]).any()
    c["do"][0, t, h, j] = bad
    d2 = run_bwd(gpu, c)
    keep = np.ones(o.shape, bool)
    keep[0, :t + 1, h, j] = False
    x = d2["dv"].float().cpu().numpy()
    assert np.isfinite(x[keep]).all() and not np.isfinite(x[0, t, h, j])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (24, 40), (17, 5)])
def test_strided_inputs(gpu, dtype, dims):
    """q, k, v as slices of one projection, batch-transposed and token-skipping views, equal the
    dense call bit for bit; the widths give 16-byte rows, 8-byte rows and single elements."""
    import torch
    dk, dv = dims
    B, T, H, Hk = 2, 75, 4, 2
    c = make(9, B, T, H, Hk, dk, dv, dtype, "token", True)
    t = dev(c)
    note(f"la strided {dtype} {dims}")
    want = gpu.ss_la_fwd(t["q"], t["k"], t["v"], t["g"], t["s0"], scale=c["scale"], return_final=True)
    wb = gpu.ss_la_bwd(t["q"], t["k"], t["v"], t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"])
    w = [Hk * dk, Hk * dk, H * dv]
    fused = torch.cat([t[n].flatten(2) for n in "qkv"], -1)
    views = [x.unflatten(-1, s) for x, s in zip(fused.split(w, -1), ((Hk, dk), (Hk, dk), (H, dv)))]
    swapped = [t[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qkv"]
    heads = [t[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"]
    skip = []
    for n in "qkv":
        x = torch.full((B, 2 * T, *t[n].shape[2:]), float("nan"), dtype=t[n].dtype, device="cuda")
        x[:, ::2] = t[n]
        skip.append(x[:, ::2])
    for q, k, v in (views, swapped, heads, skip):
        got = gpu.ss_la_fwd(q, k, v, t["g"], t["s0"], scale=c["scale"], return_final=True)
        gb = gpu.ss_la_bwd(q, k, v, t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"])
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for n in wb:
            assert torch.equal(gb[n], wb[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1, "token"), (3, 4, 2, 128, 128, "token"),
                                  (2, 6, 3, 24, 40, "head"), (2, 3, 1, 100, 33, "none"),
                                  (130, 5, 5, 64, 128, "token"), (1, 2, 1, 256, 256, "token"),
                                  (200, 3, 1, 7, 6, "token")], ids=str)
def test_step(gpu, case, dtype):
    """One token: the oracle at T = 1, in place and into a second buffer."""
    import torch
    B, H, Hk, dk, dv, decay = case
    c = make(11, B, 1, H, Hk, dk, dv, dtype, decay, True)
    t = dev(c)
    note(f"la_step {case} {dtype}")
    one = lambda x: None if x is None else x[:, 0] if x.dim() == 3 else x  # noqa: E731
    g = one(t["g"])
    g = None if g is None else g.contiguous()
    out = torch.full_like(t["s0"], float("nan"))
    s_in = t["s0"].clone()
    o = gpu.ss_la_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], s_in, g, scale=c["scale"], s_out=out)
    o2 = gpu.ss_la_step(t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["s0"], g, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(out, t["s0"])
    assert np.array_equal(s_in.cpu().numpy(), c["s0"])
    a = absolute(c)
    wo, ws = la_ref.fwd(c["q"], c["k"], c["v"], c["g"], c["s0"], c["scale"])
    Ao, As = la_ref.fwd(a["q"], a["k"], a["v"], c["g"], a["s0"], c["scale"])
    near(o[:, None], wo, out_bound(c, Ao), "o")
    near(out, ws, As * units(c) + 1e-37, "state")


def test_steps_continue_a_prompt(gpu):
    """A prompt through ss_la_fwd, then single tokens from its state: the forward over all."""
    import torch
    c = make(12, 2, 90, 4, 2, 64, 64, "f32", "token", True)
    t = dev(c)
    note("la prompt then steps")
    n = 83
    g = t["g"]
    o, s = gpu.ss_la_fwd(t["q"][:, :n], t["k"][:, :n], t["v"][:, :n], g[:, :n].contiguous(), t["s0"],
                         scale=c["scale"], return_final=True)
    outs = [o]
    for i in range(n, 90):
        outs.append(gpu.ss_la_step(t["q"][:, i], t["k"][:, i], t["v"][:, i], s, g[:, i].contiguous(),
                                   scale=c["scale"])[:, None])
    check_fwd(c, torch.cat(outs, 1), s)


def test_other_stream_and_graph(gpu):
    """On a stream of its own, with temporaries that the caller drops at once; and captured in a
    graph, replayed with other work between."""
    import torch
    c = make(13, 2, 150, 2, 2, 64, 64, "bf16", "token", True)
    t = dev(c)
    note("la stream and graph")
    args = (t["q"], t["k"], t["v"], t["g"], t["s0"])
    want = gpu.ss_la_fwd(*args, scale=c["scale"], return_final=True)
    wb = gpu.ss_la_bwd(t["q"], t["k"], t["v"], t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gpu.ss_la_fwd(*(x.clone() for x in args), scale=c["scale"], return_final=True, stream=side)
    torch.cuda.synchronize()
    # the clones above were made on the current stream: wait for them before comparing a second run
    got2 = gpu.ss_la_fwd(*args, scale=c["scale"], return_final=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got2[0], want[0]) and torch.equal(got2[1], want[1])
    assert got[0].shape == want[0].shape
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = gpu.ss_la_fwd(*args, scale=c["scale"], return_final=True)
        b = gpu.ss_la_bwd(t["q"], t["k"], t["v"], t["do"], t["g"], t["s0"], t["ds"], scale=c["scale"])
    for _ in range(3):
        f[0].zero_()
        b["dq"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f[0], want[0]) and torch.equal(f[1], want[1])
        for n in wb:
            assert torch.equal(b[n], wb[n]), n
        torch.randn(1 << 20, device="cuda").sum().item()


def test_same_bits_twice(gpu):
    import torch
    c = make(14, 2, 333, 6, 2, 48, 72, "bf16", "head", True)
    note("la twice")
    for f in (run_fwd, run_bwd):
        x, y = f(gpu, c), f(gpu, c)
        x, y = (tuple(z.values()) if isinstance(z, dict) else z for z in (x, y))
        assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_refusals(gpu):
    import torch
    c = make(15, 2, 8, 4, 2, 16, 16, "f32", "token", True)
    t = dev(c)
    q, k, v, g, s = (t[n] for n in ("q", "k", "v", "g", "s0"))
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q, k.to(torch.bfloat16), v, g, s)
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q.half(), k.half(), v.half(), g, s)
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q, k[:, :7], v, g, s)
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q, k, v, g[..., :3].contiguous(), s)
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q, k, v, g, s.transpose(2, 3))
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, g, s)
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q, k, v, g, s, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gpu.ss_la_fwd(q[:1, :1, :1].expand(2, 8, 2, 16), k, v, g, s)
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_la_fwd(q, k, v[:, :, :3], g[..., :3].contiguous(), s[:, :3].contiguous())
    assert e.value.code == -2                       # 3 value heads on 2 key heads
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_la_fwd(q, k, v, g, s, scale=float("nan"))
    assert e.value.code == -2
    big = torch.zeros(1, 4, 1, 257, device="cuda")
    with pytest.raises(gpu.SSError) as e:
        gpu.ss_la_fwd(big, big, big, None, None)
    assert e.value.code == -2
    with pytest.raises(TypeError):
        gpu.ss_la_fwd(q, k, None)
