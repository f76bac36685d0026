"""States updated in place: s_final in s0's memory (a sequence continued), ds0 in ds_final's (its
gradient).  Bit for bit what separate memory gives."""
import pytest

from tests import test_gpu_la as la
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("shape", [(2, 40, 3, 1, 64, 64), (1, 700, 2, 2, 48, 130), (300, 130, 4, 2, 24, 40)], ids=str)
def test_in_place(gpu, shape, decay, dtype):
    import torch
    c = la.make(71, *shape, dtype, decay, True)
    t = la.dev(c)
    note(f"la in place {shape} {decay} {dtype}")
    q, k, v, g = (t[n] for n in ("q", "k", "v", "g"))
    o, s = gpu.ss_la_fwd(q, k, v, g, t["s0"], scale=c["scale"], return_final=True)
    own = t["s0"].clone()
    o2, s2 = gpu.ss_la_fwd(q, k, v, g, own, scale=c["scale"], s_final=own)
    assert s2 is own and torch.equal(o, o2) and torch.equal(s, own)
    want = gpu.ss_la_bwd(q, k, v, t["do"], g, t["s0"], t["ds"], scale=c["scale"])
    own = t["ds"].clone()
    got = gpu.ss_la_bwd(q, k, v, t["do"], g, t["s0"], own, scale=c["scale"], out=dict(ds0=own))
    assert got["ds0"] is own
    for n in want:
        assert want[n] is None or torch.equal(got[n], want[n]), n
