"""Workspaces that are not memory of the call's own device, or not all there, are refused before anything
else happens (no GPU needed)."""
import pytest
import torch

import selective_state_space_34_amd as ss
from selective_state_space_34_amd import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    if _build.stale():
        _build.build()
    return ss.load()


def calls():
    x, lam = torch.zeros(2, 300, 64), torch.zeros(64)
    y, r, w = torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(64)
    return {"gr_fwd": lambda t: ss.ss_gr_fwd(x, x, x, lam, workspace=t),
            "gr_bwd": lambda t: ss.ss_gr_bwd(x, x, x, lam, x, workspace=t),
            "ln_bwd": lambda t: ss.ss_ln_bwd(y, r, w, workspace=t)}


@pytest.mark.parametrize("name", ["gr_fwd", "gr_bwd", "ln_bwd"])
def test_refused(name):
    call = calls()[name]
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 10, 64)[:, ::2],
                torch.empty(1 << 24, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    with pytest.raises(TypeError, match="workspace"):
        call(bytearray(1 << 24))
