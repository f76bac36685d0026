"""A gated recurrent layer as a server and as a trainer run it.

Serving, with 4-bit weights: a prompt in one piece, then token after token, and both ways of reading
the same text compared.

    per layer   u, e, s = ss_ln_fwd(x, w, b, s, q8=SS_Q4_MX)     norm of the residual stream, 4 bits
                p = ss_mx4_mm(u, e, *W_in)                        x | gate r | gate i of every channel
                y = ss_gr_fwd(x, r, i, lam)                       the prompt, or
                y = ss_gr_step(x, r, i, lam, state)               one token: the state in place
                x = ss_mx4_mm(*ss_mx4_quant(y), *W_out)           what the layer adds to the stream

Training, with dense float32 weights: one loss and the gradients of every parameter and of the
stream, documents packed one after another.

Run on an MI355X:  python examples/recurrent_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import selective_state_space_34_amd as ss  # noqa: E402


def rates(channels, draw):
    """lam with exp(-8 softplus(lam)) between 0.9 and 0.999."""
    return torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.sigmoid(draw(channels))) / 8))


class Layer:
    def __init__(self, width, channels, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.channels = channels
        self.w, self.b, self.lam = 1 + 0.1 * draw(width), 0.1 * draw(width), rates(channels, draw)
        self.w_in = ss.ss_mx4_quant(draw(3 * channels, width) / width ** 0.5)
        self.w_out = ss.ss_mx4_quant(draw(width, channels) / channels ** 0.5)

    def _project(self, x, res):
        u, e, res = ss.ss_ln_fwd(x, self.w, self.b, res, q8=ss.SS_Q4_MX)
        return *ss.ss_mx4_mm(u, e, *self.w_in).split(self.channels, -1), res

    def prompt(self, x, res):
        """x, res [B, T, width] -> what the layer adds, the stream, the state behind the text."""
        v, r, i, res = self._project(x, res)
        y, state = ss.ss_gr_fwd(v, r, i, self.lam, return_final=True)
        return ss.ss_mx4_mm(*ss.ss_mx4_quant(y), *self.w_out), res, state

    def token(self, x, res, state):
        """The same for one token, x, res [B, width]; the state is updated in place."""
        v, r, i, res = self._project(x, res)
        y = ss.ss_gr_step(v, r, i, self.lam, state)
        return ss.ss_mx4_mm(*ss.ss_mx4_quant(y), *self.w_out), res


def serve(width=512, channels=640, layers=2, batch=3, tokens=200, prompt=180, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    net = [Layer(width, channels, seed + 1 + i) for i in range(layers)]
    text = torch.randn((batch, tokens, width), generator=gen, device="cuda").to(torch.bfloat16)

    def whole(x):
        res, states = torch.zeros_like(x), []
        for layer in net:
            x, res, state = layer.prompt(x, res)
            states.append(state)
        return x + res, states

    want, final = whole(text)
    got, states = whole(text[:, :prompt].contiguous())
    outs = [got]
    for t in range(prompt, tokens):
        x = text[:, t].contiguous()
        res = torch.zeros_like(x)
        for layer, state in zip(net, states):
            x, res = layer.token(x, res, state)
        outs.append((x + res)[:, None])
    got = torch.cat(outs, 1)
    off = float((got.float() - want.float()).norm() / want.float().norm())
    off_state = max(float((a - b).norm() / b.norm()) for a, b in zip(states, final))
    print(f"{layers} layers, {batch} texts: {prompt} tokens at once, {tokens - prompt} one by one; "
          f"against all {tokens} at once: outputs {off:.2e}, states {off_state:.2e} (relative)")
    return off, off_state


def training_problem(width=96, channels=160, batch=2, tokens=150, seed=0):
    """Parameters, inputs and the gradient of the loss by y, float32 on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    par = {"w": 1 + 0.1 * draw(width), "b": 0.1 * draw(width), "lam": rates(channels, draw),
           "w_in": draw(3 * channels, width) / width ** 0.5,
           "w_out": draw(width, channels) / channels ** 0.5}
    reset = torch.rand((batch, tokens), generator=gen, device="cuda") < 0.03
    return par, draw(batch, tokens, width), draw(batch, tokens, width), reset, draw(batch, tokens, width)


def gradients(par, x, res, reset, target):
    """Loss sum(target · (stream + layer)) and its gradients by the parameters, x and res."""
    B, T, width = x.shape
    n, s = ss.ss_ln_fwd(x, par["w"], par["b"], res)
    p = n @ par["w_in"].t()
    v, r, i = p.split(par["lam"].shape[0], -1)              # strided slices
    y, ckpt = ss.ss_gr_fwd(v, r, i, par["lam"], reset=reset, return_ckpt=True)
    out = s + y @ par["w_out"].t()
    loss = (target * out).sum()
    flat = lambda t: t.reshape(B * T, -1)  # noqa: E731
    g = {"w_out": flat(target).t() @ flat(y)}
    dg = ss.ss_gr_bwd(v, r, i, par["lam"], (target @ par["w_out"]).contiguous(), reset=reset,
                      h_ckpt=ckpt)
    g["lam"] = dg["dlam"]
    dp = torch.cat([dg["dx"], dg["dr"], dg["di"]], -1)
    g["w_in"] = flat(dp).t() @ flat(n)
    g["x"], g["w"], g["b"] = ss.ss_ln_bwd((dp @ par["w_in"]).contiguous(), s, par["w"], target)
    g["res"] = g["x"]
    return loss, g


if __name__ == "__main__":
    serve()
    loss, g = gradients(*training_problem())
    print(f"loss {float(loss):.4f}; gradients' norms: " + ", ".join(f"{n} {float(t.norm()):.3g}" for n, t in g.items()))
