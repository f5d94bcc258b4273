"""Gated delta rule blocks out of this package's operators: a prompt, single tokens that go on from it, and
training steps. A block, for rows y of the block before and the sum s of all that came before y:

    s += y;  h = prenorm(s)
    c, z, dt, b = the parts of h W_in^T
    q, k, v = the parts of silu(causal conv(c) + bias)
    o = delta(q, k, v) with decays exp(A softplus(dt + dt_bias)) and strengths sigmoid(b)
    y = postnorm(o, a head at a time) gated by z, times W_out^T

and a last prenorm after the last block.

Run on a HIP device:  python examples/delta_block.py
"""
from __future__ import annotations

import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import masked_depthwise_causal_amd as mdc  # noqa: E402


@dataclass
class State:
    """What a block's sequences carry from one call to the next."""
    conv: torch.Tensor   # [W-1,B,2 G K + H V]
    delta: torch.Tensor  # [B,H,K,V] fp32


class Block:
    """Parameters by name in `p`: 16-bit, but for the decays' A and dt_bias, which are fp32."""

    def __init__(self, width, heads, key_heads, keys, values, taps=4, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.H, self.G, self.K, self.V, self.taps, self.dtype = heads, key_heads, keys, values, taps, dtype
        self.channels = 2 * key_heads * keys + heads * values

        def weight(rows, columns):
            return torch.randn((rows, columns), generator=g) * columns ** -0.5

        d = torch.exp(torch.rand(heads, generator=g) * math.log(100) + math.log(1e-3))
        p = {"pre": torch.ones(width), "in": weight(self.channels + heads * values + 2 * heads, width),
             "conv": torch.randn((taps, self.channels), generator=g) * 0.5,
             "conv_bias": torch.zeros(self.channels), "post": torch.ones(values),
             "out": weight(width, heads * values)}
        self.p = {k: v.to(device, dtype) for k, v in p.items()}
        self.p |= {"A": -(torch.rand(heads, generator=g) * 15 + 1).to(device),
                   "dt_bias": torch.log(torch.expm1(d)).to(device)}  # step sizes from 1e-3 to 0.1

    def state(self, batch):
        device = self.p["A"].device
        return State(torch.zeros((self.taps - 1, batch, self.channels), dtype=self.dtype, device=device),
                     torch.zeros((batch, self.H, self.K, self.V), device=device))

    def _in(self, m):
        c, z, dt, b = m.split([self.channels, self.H * self.V, self.H, self.H], dim=-1)
        return c, z, dt, b

    def _heads(self, c):
        q, k, v = c.split([self.G * self.K, self.G * self.K, self.H * self.V], dim=-1)
        return (q.unflatten(-1, (self.G, self.K)), k.unflatten(-1, (self.G, self.K)),
                v.unflatten(-1, (self.H, self.V)))

    def prompt(self, y, s=None, state=None, lengths=None):
        """(y, s) for the next block, and the state after each sequence's last row, for rows y [S,B,width]."""
        p, state = self.p, state or self.state(y.shape[1])
        h, s = mdc.prenorm_forward(y, p["pre"], residual=s, return_sum=True)
        c, z, dt, b = self._in(mdc.linear_forward(h, p["in"]))
        c, conv = mdc.conv_act_forward(c, p["conv"], p["conv_bias"], lengths=lengths, state=state.conv,
                                       return_state=True)
        o, end = mdc.delta_forward(*self._heads(c), dt, b, p["A"], p["dt_bias"], lengths=lengths,
                                   state=state.delta, return_state=True)
        n = mdc.postnorm_forward(o.flatten(2), p["post"], z=z, groups=self.H)
        return mdc.linear_forward(n, p["out"]), s, State(conv, end)

    def token(self, y, s, state):
        """(y, s) for the next block, for one row y [B,width]; `state` moves on in place."""
        p = self.p
        h, s = mdc.prenorm_forward(y, p["pre"], residual=s, return_sum=True)
        c, z, dt, b = self._in(mdc.linear_forward(h, p["in"]))
        c = mdc.conv_act_step(c, p["conv"], state.conv, p["conv_bias"])
        o = mdc.delta_step(state.delta, *self._heads(c), dt, b, p["A"], p["dt_bias"])
        n = mdc.postnorm_forward(o.flatten(1), p["post"], z=z, groups=self.H)
        return mdc.linear_forward(n, p["out"]), s

    def forward(self, y, s=None, lengths=None):
        """(y, s) for the next block, and what backward needs."""
        p = self.p
        h, total = mdc.prenorm_forward(y, p["pre"], residual=s, return_sum=True)
        m = mdc.linear_forward(h, p["in"])
        c, z, dt, b = self._in(m)
        a = mdc.conv_act_forward(c, p["conv"], p["conv_bias"], lengths=lengths)
        o, saved = mdc.delta_forward(*self._heads(a), dt, b, p["A"], p["dt_bias"], lengths=lengths,
                                     return_saved=True)
        n = mdc.postnorm_forward(o.flatten(2), p["post"], z=z, groups=self.H)
        return mdc.linear_forward(n, p["out"]), total, (y, s, h, m, a, o, n, saved, lengths)

    def backward(self, gy, gs, kept):
        """The gradients of y and s (None if there was no s), for those of the two results, and those of the
        parameters by name."""
        p = self.p
        y, s, h, m, a, o, n, saved, lengths = kept
        c, z, dt, b = self._in(m)
        g_out = mdc.linear_backward(gy, n, p["out"], grad_bias=False)
        post = mdc.postnorm_backward(g_out.x, o.flatten(2), p["post"], z=z, groups=self.H)
        d = mdc.delta_backward(post.x.unflatten(-1, (self.H, self.V)), *self._heads(a), dt, b, p["A"], saved,
                               p["dt_bias"], lengths=lengths)
        conv = mdc.conv_act_backward(torch.cat([t.flatten(2) for t in (d.q, d.k, d.v)], dim=-1), c, p["conv"],
                                     p["conv_bias"], lengths=lengths)
        g_in = mdc.linear_backward(torch.cat([conv.x, post.z, d.dt, d.b], dim=-1), h, p["in"], grad_bias=False)
        pre = mdc.prenorm_backward(g_in.x, y, p["pre"], residual=s, gradSum=gs)
        return pre.x, pre.residual, {"pre": pre.weight, "in": g_in.weight, "conv": conv.weight,
                                     "conv_bias": conv.bias, "A": d.A, "dt_bias": d.dt_bias,
                                     "post": post.weight, "out": g_out.weight}


class Stack:
    def __init__(self, layers, width, *sizes, dtype=torch.bfloat16, seed=0, **kw):
        self.blocks = [Block(width, *sizes, dtype=dtype, seed=seed + i, **kw) for i in range(layers)]
        self.last = torch.ones(width, dtype=dtype, device=self.blocks[0].p["A"].device)

    def state(self, batch):
        return [b.state(batch) for b in self.blocks]

    def prompt(self, x, state=None, lengths=None):
        s, ends = None, []
        for i, block in enumerate(self.blocks):
            x, s, end = block.prompt(x, s, state[i] if state else None, lengths)
            ends.append(end)
        return mdc.prenorm_forward(x, self.last, residual=s), ends

    def token(self, x, state):
        s = None
        for block, st in zip(self.blocks, state):
            x, s = block.token(x, s, st)
        return mdc.prenorm_forward(x, self.last, residual=s)

    def forward(self, x, lengths=None):
        s, kept = None, []
        for block in self.blocks:
            x, s, k = block.forward(x, s, lengths)
            kept.append(k)
        return mdc.prenorm_forward(x, self.last, residual=s), (kept, x, s)

    def backward(self, gout, kept):
        """The gradient of x, that of the last norm's weight, and each block's."""
        kept, x, s = kept
        pre = mdc.prenorm_backward(gout, x, self.last, residual=s)
        gy, gs, grads = pre.x, pre.residual, []
        for block, k in zip(reversed(self.blocks), reversed(kept)):
            gy, gs, g = block.backward(gy, gs, k)
            grads.insert(0, g)
        return gy, pre.weight, grads


def main():
    S, B, width = 257, 4, 256
    stack = Stack(2, width, 8, 4, 32, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((S, B, width), generator=g, device="cuda").to(stack.last.dtype)

    whole, end = stack.prompt(x)
    lengths = torch.tensor([S - 8] * B, device="cuda")
    _, state = stack.prompt(x, lengths=lengths)  # the prompt, padded by eight rows
    tokens = torch.stack([stack.token(x[t], state) for t in range(S - 8, S)])
    off = (tokens.float() - whole[S - 8:].float()).norm() / whole[S - 8:].float().norm()
    far = (state[-1].delta - end[-1].delta).norm() / end[-1].delta.norm()
    print(f"eight tokens after a prompt of {S - 8}: outputs {off:.1e}, state {far:.1e} from the whole")

    # regression onto a fixed target by plain gradient descent on fp32 copies of the parameters
    target = torch.randn((S, B, width), generator=g, device="cuda")
    master = [{k: v.float() for k, v in b.p.items()} for b in stack.blocks]
    for step in range(5):
        out, kept = stack.forward(x)
        diff = out.float() - target
        print(f"step {step}: loss {float(diff.square().mean()):.4f}")
        _, _, grads = stack.backward((diff * (2 / diff.numel())).to(out.dtype), kept)
        for block, copy, grad in zip(stack.blocks, master, grads):
            for k, v in grad.items():
                copy[k] -= 2.0 * v.float()
                block.p[k] = copy[k].to(block.p[k].dtype)


if __name__ == "__main__":
    main()
