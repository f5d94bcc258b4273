"""A selective state space block out of this package's operators: a prompt, single tokens that go on
from it, and training steps.

    xz = x W_in^T                         u, z = its halves
    c  = silu(causal conv(u) + bias)
    p  = c W_x^T                          r, B, C = its parts
    y  = scan(c, r W_dt^T, A, B, C) gated by z, with step sizes softplus(. + dt_bias)
    out = y W_out^T + x

Run on a HIP device:  python examples/ssm_block.py
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
    """What a sequence carries from one call to the next."""
    conv: torch.Tensor  # [W-1,B,H]
    scan: torch.Tensor  # [B,N,H] fp32


class Block:
    """Parameters by name in `p`: 16-bit, but for the scan's A, D and dt_bias, which are fp32."""

    def __init__(self, width, inner, states=16, rank=None, taps=4, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.rank = rank or max(1, math.ceil(width / 16))
        self.inner, self.states, self.taps, self.dtype = inner, states, taps, dtype

        def weight(rows, columns):
            return torch.randn((rows, columns), generator=g) * columns ** -0.5

        d = torch.exp(torch.rand(inner, generator=g) * math.log(100) + math.log(1e-3))
        p = {"in": weight(2 * inner, width), "conv": torch.randn((taps, inner), generator=g) * 0.5,
             "conv_bias": torch.zeros(inner), "x": weight(self.rank + 2 * states, inner),
             "dt": weight(inner, self.rank), "out": weight(width, inner)}
        self.p = {k: v.to(device, dtype) for k, v in p.items()}
        rates = torch.arange(1, states + 1, dtype=torch.float32)[:, None]
        self.p |= {"A": -rates.repeat(1, inner).to(device), "D": torch.ones(inner, device=device),
                   "dt_bias": torch.log(torch.expm1(d)).to(device)}  # step sizes from 1e-3 to 0.1

    def state(self, batch):
        device = self.p["A"].device
        return State(torch.zeros((self.taps - 1, batch, self.inner), dtype=self.dtype, device=device),
                     torch.zeros((batch, self.states, self.inner), device=device))

    def _parts(self, proj):
        return proj.split([self.rank, self.states, self.states], dim=-1)

    def prompt(self, x, state=None, lengths=None):
        """out [S,B,width] and the state after each sequence's last row, for rows x [S,B,width]."""
        p = self.p
        state = state or self.state(x.shape[1])
        u, z = mdc.linear_forward(x, p["in"]).chunk(2, dim=-1)
        c, conv = mdc.conv_act_forward(u, p["conv"], p["conv_bias"], lengths=lengths,
                                       state=state.conv, return_state=True)
        r, B, C = self._parts(mdc.linear_forward(c, p["x"]))
        y, scan = mdc.scan_forward(c, mdc.linear_forward(r, p["dt"]), p["A"], B, C, D=p["D"], z=z,
                                   dt_bias=p["dt_bias"], lengths=lengths, state=state.scan,
                                   return_state=True)
        return mdc.linear_forward(y, p["out"], residual=x), State(conv, scan)

    def token(self, x, state):
        """out [B,width] for one row x [B,width]; `state` moves on in place."""
        p = self.p
        u, z = mdc.linear_forward(x, p["in"]).chunk(2, dim=-1)
        c = mdc.conv_act_step(u, p["conv"], state.conv, p["conv_bias"])
        r, B, C = self._parts(mdc.linear_forward(c, p["x"]))
        y = mdc.scan_step(state.scan, c, mdc.linear_forward(r, p["dt"]), p["A"], B, C, D=p["D"], z=z,
                          dt_bias=p["dt_bias"])
        return mdc.linear_forward(y, p["out"], residual=x)

    def forward(self, x, lengths=None):
        """out [S,B,width], and what backward needs."""
        p = self.p
        xz = mdc.linear_forward(x, p["in"])
        u, z = xz.chunk(2, dim=-1)
        c = mdc.conv_act_forward(u, p["conv"], p["conv_bias"], lengths=lengths)
        proj = mdc.linear_forward(c, p["x"])
        r, B, C = self._parts(proj)
        dt = mdc.linear_forward(r, p["dt"])
        y, saved = mdc.scan_forward(c, dt, p["A"], B, C, D=p["D"], z=z, dt_bias=p["dt_bias"],
                                    lengths=lengths, return_saved=True)
        return mdc.linear_forward(y, p["out"], residual=x), (x, xz, c, proj, dt, y, saved, lengths)

    def backward(self, gout, kept):
        """The gradient of x and those of the parameters by name."""
        p = self.p
        x, xz, c, proj, dt, y, saved, lengths = kept
        u, z = xz.chunk(2, dim=-1)
        r, B, C = self._parts(proj)
        g_out = mdc.linear_backward(gout, y, p["out"], grad_bias=False)
        s = mdc.scan_backward(g_out.x, c, dt, p["A"], B, C, saved, D=p["D"], z=z,
                              dt_bias=p["dt_bias"], lengths=lengths)
        g_dt = mdc.linear_backward(s.dt, r, p["dt"], grad_bias=False)
        g_x = mdc.linear_backward(torch.cat([g_dt.x, s.B, s.C], dim=-1), c, p["x"], grad_bias=False)
        conv = mdc.conv_act_backward(s.x + g_x.x, u, p["conv"], p["conv_bias"], lengths=lengths)
        g_in = mdc.linear_backward(torch.cat([conv.x, s.z], dim=-1), x, p["in"], grad_bias=False)
        return g_in.x + gout, {"in": g_in.weight, "conv": conv.weight, "conv_bias": conv.bias,
                               "x": g_x.weight, "dt": g_dt.weight, "out": g_out.weight, "A": s.A,
                               "D": s.D, "dt_bias": s.dt_bias}


def main():
    S, B, width, inner = 257, 4, 256, 512
    block = Block(width, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((S, B, width), generator=g, device="cuda").to(block.dtype)

    whole, end = block.prompt(x)
    lengths = torch.tensor([S - 8] * B, device="cuda")
    _, state = block.prompt(x, lengths=lengths)  # the prompt, padded by eight rows
    tokens = torch.stack([block.token(x[t], state) for t in range(S - 8, S)])
    off = (tokens.float() - whole[S - 8:].float()).norm() / whole[S - 8:].float().norm()
    far = (state.scan - end.scan).norm() / end.scan.norm()
    print(f"eight tokens after a prompt of {S - 8}: outputs {off:.1e}, state {far:.1e} from the whole")

    # regression onto a fixed target by plain gradient descent on fp32 copies of the parameters
    target = torch.randn((S, B, width), generator=g, device="cuda")
    master = {k: v.float() for k, v in block.p.items()}
    for step in range(5):
        out, kept = block.forward(x)
        diff = out.float() - target
        print(f"step {step}: loss {float(diff.square().mean()):.4f}")
        _, grads = block.backward((diff * (2 / diff.numel())).to(block.dtype), kept)
        for k, v in grads.items():
            master[k] -= 2.0 * v.float()
            block.p[k] = master[k].to(block.p[k].dtype)


if __name__ == "__main__":
    main()
