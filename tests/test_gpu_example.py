"""examples/decode_layer.py: the norm, the 4-bit products and both forms of linear attention
together.  A text read at once and the same text as a prompt and single tokens differ by roundings.
The first layer's rows are the same in both; its outputs differ by the roundings of the two forms
and of bfloat16, about e = 3e-3 relative.  The second layer rounds them to e4m3, whose steps are
d = 2^-4 to 2^-3 of a value: where the two readings fall to different sides the codes differ by a
whole step, sqrt(e·d) = 1.6e-2 in the mean square, in q, k, v and the decays alike, so 3e-2 in the
outputs and states.  The bound is three times that; a wrong token, head or state is of the order
of 1."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_layer(gpu):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_layer
    off, off_state = decode_layer.main()
    assert off < 0.1 and off_state < 0.1
