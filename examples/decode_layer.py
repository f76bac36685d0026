"""One linear-attention layer with 4-bit weights, as a server would run it: a prompt in one piece,
then token after token, and both ways of reading the same text compared.

    per layer   u8, s, r = ss_rms_fwd(x, w, r, q8=SS_Q8_FP8)     norm of the residual stream, 8 bits
                p = ss_q4_mv(u8, W_in, ..., x_scale=s)            q | k | v | decay of every head
                o = ss_la_fwd(q, k, v, g, state)                  the prompt: chunked form, or
                o = ss_la_step(q, k, v, state, g)                 one token: the state in place
                x = ss_q4_mv(o, W_out, ...)                       what the layer adds to the stream

The prompt goes through the same 4-bit products here, so that one set of weights serves both; they
are made for a few rows, and a server with long prompts would widen the weights once and take dense
products for those (2560 by 10240, 1024 rows: 292 us in 4 bits, 51 us dense).

Run on an MI355X:  python examples/decode_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import selective_state_space_34_amd as ss  # noqa: E402

GROUP = 64


def quantize(w):
    """4-bit codes, scales and zeros of W [N, K], GROUP columns to a scale."""
    n, k = w.shape
    g = w.view(n, k // GROUP, GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / 15).clamp(min=1e-6).to(torch.bfloat16)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    u = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8)
    u = u.view(n, k // 2, 2)
    return (u[..., 0] | (u[..., 1] << 4)).contiguous(), scale, zero.to(torch.uint8)


class Layer:
    def __init__(self, width, heads, dk, dv, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.heads, self.dk, self.dv = heads, dk, dv
        self.sizes = [heads * dk, heads * dk, heads * dv, heads]
        self.norm = 1 + 0.1 * draw(width)
        self.w_in = quantize(draw(sum(self.sizes), width) / width ** 0.5)
        self.w_out = quantize(draw(width, heads * dv) / (heads * dv) ** 0.5)
        self.rate = torch.exp(torch.linspace(-4.0, 0.0, heads, device="cuda"))

    def _project(self, x, res):
        """Norm and input projection: q, k, v (strided slices), log decay, and the stream."""
        u, s, res = ss.ss_rms_fwd(x, self.norm, res, q8=ss.SS_Q8_FP8)
        p = ss.ss_q4_mv(u, *self.w_in, group=GROUP, x_scale=s)
        q, k, v, a = p.split(self.sizes, -1)
        q, k = (t.unflatten(-1, (self.heads, self.dk)) for t in (q, k))
        g = -self.rate * torch.nn.functional.softplus(a.float())
        return q, k, v.unflatten(-1, (self.heads, self.dv)), g.contiguous(), res

    def prompt(self, x, res):
        """x, res [B, T, width] -> what the layer adds, the stream, the state behind the text."""
        q, k, v, g, res = self._project(x, res)
        o, state = ss.ss_la_fwd(q, k, v, g, scale=self.dk ** -0.5, return_final=True)
        return ss.ss_q4_mv(o.flatten(2), *self.w_out, group=GROUP), res, state

    def token(self, x, res, state):
        """The same for one token, x, res [B, width]; the state is updated in place."""
        q, k, v, g, res = self._project(x, res)
        o = ss.ss_la_step(q, k, v, state, g, scale=self.dk ** -0.5)
        return ss.ss_q4_mv(o.flatten(1), *self.w_out, group=GROUP), res


def main(width=512, heads=4, dk=64, dv=128, layers=2, batch=2, tokens=96, prompt=80, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    net = [Layer(width, heads, dk, dv, seed + 1 + i) for i in range(layers)]
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


if __name__ == "__main__":
    main()
