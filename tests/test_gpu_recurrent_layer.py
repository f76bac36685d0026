"""examples/recurrent_layer.py: the layer norm, the 4-bit products and both forms of the recurrence
together, and a training step's gradients.

Serving: a text read at once and the same text as a prompt and single tokens.  The first layer's rows
are the same in both; its states differ by float32 roundings, about 1e-6, so that one of 3000 of its
bfloat16 outputs falls to another side, 7e-5 in the mean square.  Where 4-bit codes then fall to
different sides they differ by a whole step, d = 0.3 of a value, so sqrt(7e-5·d) = 5e-3; behind the
second layer's norm sqrt(5e-3·d) = 4e-2 in its states, and sqrt(4e-2·d) = 0.11 in what it adds.  The
bounds are three times that; a wrong token, channel or state is of the order of 1.

Training: float32 products of up to 96 · 3 terms, sums over 300 tokens and the kernels' own errors,
each some 1e-6 of its terms; 1e-4 of every gradient's norm allows for cancellation in them.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_serving(gpu):
    import recurrent_layer
    off, off_state = recurrent_layer.serve()
    assert off < 0.33 and off_state < 0.12


def test_training_gradients(gpu):
    """Against float64 autograd of the formulas on the CPU, token after token."""
    import recurrent_layer
    import torch
    par, x, res, reset, target = recurrent_layer.training_problem()
    loss, g = recurrent_layer.gradients(par, x, res, reset, target)
    ins = {n: t.double().cpu().requires_grad_() for n, t in {**par, "x": x, "res": res}.items()}
    cut, tgt = reset.cpu(), target.double().cpu()
    s = ins["x"] + ins["res"]
    d = s - s.mean(-1, keepdim=True)
    n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5) * ins["w"] + ins["b"]
    v, r, i = (n @ ins["w_in"].t()).split(par["lam"].shape[0], -1)
    la = -8 * torch.nn.functional.softplus(ins["lam"]) * torch.sigmoid(r)
    h, ys = torch.zeros_like(v[:, 0]), []
    for t in range(x.shape[1]):
        c = cut[:, t, None]
        a = torch.where(c, 0.0, la[:, t].exp())
        gain = torch.where(c, 1.0, torch.sqrt(-torch.expm1(2 * la[:, t])))
        h = a * h + gain * torch.sigmoid(i[:, t]) * v[:, t]
        ys.append(h)
    want = (tgt * (s + torch.stack(ys, 1) @ ins["w_out"].t())).sum()
    want.backward()
    assert abs(float(loss) - float(want)) < 1e-4 * float((tgt * tgt).sum()) ** 0.5 * 10
    for name, t in ins.items():
        got = g[name].double().cpu()
        assert float((got - t.grad).norm() / t.grad.norm()) < 1e-4, name
