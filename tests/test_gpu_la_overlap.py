"""Linear attention whose tokens share rows: q, k and v expanded over the tokens (token stride 0),
rows that overlap, and single tokens whose stride says nothing.  What a chunk holds behind a row's
end must not be taken for tokens.  Against the float64 oracle, with the bounds of test_gpu_la.py."""
import numpy as np
import pytest

from tests import test_gpu_la as la
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def call(ss, c, t, views):
    q, k, v = views
    kw = dict(scale=c["scale"], lengths=t["lengths"])
    la.check_fwd(c, *ss.ss_la_fwd(q, k, v, t["g"], t["s0"], return_final=True, **kw))
    la.check_bwd(c, ss.ss_la_bwd(q, k, v, t["do"], t["g"], t["s0"], t["ds"], **kw))


def numpy_of(c, views):
    for n, x in zip("qkv", views):
        c[n] = x.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["kv", "qkv", "k"])
@pytest.mark.parametrize("T,lengths", [(65, None), (97, [97, 33]), (200, [1, 130]), (700, [700, 450])],
                         ids=str)
def test_rows_expanded_over_tokens(gpu, T, lengths, which, dtype):
    B = 2 if lengths else 1
    c = la.make(41 + T, B, T, 4, 2, 64, 64, dtype, "token", True, lengths)
    t = la.dev(c)
    note(f"la expanded {which} T={T} {lengths} {dtype}")
    views = [t[n][:, :1].expand(-1, T, -1, -1) if n in which else t[n] for n in "qkv"]
    assert all(x.stride(1) == 0 for n, x in zip("qkv", views) if n in which)
    numpy_of(c, views)
    call(gpu, c, t, views)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [64, 128, 704])
def test_expanded_rows_of_full_chunks(gpu, T, dtype):
    """No token behind the end in any chunk: the same rows, with and without lengths."""
    import torch
    c = la.make(53 + T, 1, T, 4, 2, 64, 64, dtype, "token", True)
    t = la.dev(c)
    note(f"la expanded, full chunks T={T} {dtype}")
    views = [t[n][:, :1].expand(-1, T, -1, -1) for n in "qkv"]
    numpy_of(c, views)
    call(gpu, c, t, views)
    c["lengths"] = [T - 3]
    t["lengths"] = torch.tensor([T - 3], dtype=torch.int32, device="cuda")
    call(gpu, c, t, views)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("step", [8, 16, 48])
def test_rows_that_overlap(gpu, step, dtype):
    """Token t starts `step` elements behind token t - 1, in rows of 64."""
    import torch
    T = 75
    c = la.make(43, 1, T, 1, 1, 64, 64, dtype, "token", True)
    t = la.dev(c)
    note(f"la overlap {step} {dtype}")
    flat = {n: torch.randn(T * step + 64, device="cuda").to(t[n].dtype) for n in "qkv"}
    views = [flat[n].as_strided((1, T, 1, 64), (T * step, step, 64, 1)) for n in "qkv"]
    numpy_of(c, views)
    call(gpu, c, t, views)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("stride", [0, 16])
def test_one_token_of_any_stride(gpu, stride, dtype):
    """T = 1: the token stride is not used, whatever it is."""
    c = la.make(47, 2, 1, 2, 2, 64, 64, dtype, "token", True)
    t = la.dev(c)
    note(f"la one token stride {stride} {dtype}")
    views = [t[n].as_strided(t[n].shape, (128, stride, 64, 1)) for n in "qkv"]
    call(gpu, c, t, views)
