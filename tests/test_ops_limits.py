"""Launches of 2^32 threads or more, which the runtime would cut off without an error, are refused
with SS_ERR_DIMS before anything is launched; sizes just below are taken (no GPU needed)."""
import pytest

import selective_state_space_34_amd as ss
from selective_state_space_34_amd import _build

FAKE = 0x10000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if _build.stale():
        _build.build()
    return ss.load()


def size(backward, **kw):
    try:
        return ss.la_workspace_size(ss.make_la_dims(kw["B"], 1, kw["H"], kw["H"], kw["dk"], kw["dv"]), backward)
    except ss.SSError as e:
        return e.code


def test_sweeps(lib):
    # a workgroup of 512 threads for each of two column tiles of 2^22 heads: 2^32
    assert size(False, B=1 << 12, H=1 << 10, dk=16, dv=256) == -2
    assert size(False, B=(1 << 12) - 1, H=1 << 10, dk=16, dv=256) >= 0
    # the gradient's sweeps have their columns over dk
    assert size(True, B=1 << 12, H=1 << 10, dk=256, dv=16) == -2
    assert size(True, B=(1 << 12) - 1, H=1 << 10, dk=256, dv=16) > 0


def test_step(lib):
    def call(B, dv):
        d = ss.make_la_dims(B, 1, 1 << 10, 1 << 10, 16, dv)
        return lib.ss_la_step(d, *[FAKE] * 4, None, FAKE, FAKE, None)
    assert call(1 << 11, 255) == -2                  # 2^21 heads, eight workgroups of 256 each
    assert call((1 << 11) - 1, 255) == -1            # on to the missing state
    assert call((1 << 12) - 1, 256) == -1


def test_q4(lib):
    def call(n):
        return lib.ss_q4_mv(ss.make_q4_dims(1, n, 32), FAKE, None, FAKE, FAKE, None, None, None)
    assert call(1 << 28) == -2                       # 2^23 workgroups of 512
    assert call((1 << 28) - 64) == -1                # on to the missing output
