"""The tests' 64-bit forms of the state space block's operators, pinned on the CPU: gradients against
central differences of the forward form, and hand-worked values."""
from __future__ import annotations

import pytest
import torch

from . import ssm_ref as ref

F = torch.float64


def randn(g, *shape):
    return torch.randn(shape, generator=g, dtype=F)


def differences(f, inputs, weights, eps=1e-6):
    """d sum(f * weights) / d input by central differences, for every element of every input."""
    def total():
        return sum((v * w).sum() for v, w in zip(f(), weights))

    out = []
    for t in inputs:
        g = torch.zeros_like(t)
        flat, gf = t.view(-1), g.view(-1)
        for i in range(flat.numel()):
            old = flat[i].item()
            flat[i] = old + eps
            up = total()
            flat[i] = old - eps
            down = total()
            flat[i] = old
            gf[i] = (up - down) / (2 * eps)
        out.append(g)
    return out


def agree(got, want):
    # central differences in 64 bits: truncation ~eps^2, rounding ~1e-16/eps
    assert torch.allclose(got, want, rtol=1e-7, atol=1e-8), (got - want).abs().max()


@pytest.mark.parametrize("W,kind", [(1, "silu"), (3, None), (4, "silu")])
@pytest.mark.parametrize("lengths", [None, [0, 5, 1]])
def test_conv_gradients_against_differences(W, kind, lengths):
    g = torch.Generator().manual_seed(W)
    S, B, H = 5, 3, 2
    x, w, b, s = randn(g, S, B, H), randn(g, W, H), randn(g, H), randn(g, W - 1, B, H)
    gy, gf = randn(g, S, B, H), randn(g, W - 1, B, H)

    def forward():
        r = ref.conv(x, w, b, kind, lengths, s)
        return r["y"][0], r["state"][0]

    want = differences(forward, (x, w, b, s), (gy, gf))
    r = ref.conv(x, w, b, kind, lengths, s, gy, gf)
    for k, v in zip(("gx", "gw", "gb", "gs"), want):
        agree(r[k][0], v)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("lengths", [None, [0, 4, 1]])
def test_scan_gradients_against_differences(gate, lengths):
    g = torch.Generator().manual_seed(9)
    S, B, H, N, G = 4, 3, 4, 3, 2
    x, dt, z = (randn(g, S, B, H) for _ in range(3))
    A, Bm, Cm = -torch.rand((N, H), generator=g, dtype=F) - 0.1, randn(g, S, B, G, N), randn(g, S, B, G, N)
    D, bias, s = randn(g, H), randn(g, H), randn(g, B, N, H)
    gout, gf = randn(g, S, B, H), randn(g, B, N, H)
    z = z if gate else None

    def forward():
        r = ref.scan(x, dt, A, Bm, Cm, D, z, bias, True, lengths, s)
        return r["out"][0], r["state"][0]

    ins = {"gx": x, "gdt": dt, "gA": A, "gB": Bm, "gC": Cm, "gD": D, "gbias": bias, "gs": s}
    if gate:
        ins["gz"] = z
    want = differences(forward, ins.values(), (gout, gf))
    r = ref.scan(x, dt, A, Bm, Cm, D, z, bias, True, lengths, s, gout, gf)
    for k, v in zip(ins, want):
        agree(r[k][0], v)


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu", "softplus", None])
def test_activation_slopes_against_differences(kind):
    v = torch.linspace(-6, 6, 241, dtype=F) + 0.013  # keeps off relu's corner
    e = 1e-6
    agree(ref.act_slope(v, kind), (ref.act(v + e, kind) - ref.act(v - e, kind)) / (2 * e))


def test_scan_by_hand():
    # one channel, one state, no softplus: s1 = 1*2*3 = 6; s2 = exp(-1) 6 + 1*1*5; y = C s + D x
    one = lambda *v: torch.tensor(v, dtype=F).view(-1, 1, 1)  # noqa: E731
    r = ref.scan(one(2, 1), one(1, 1), torch.tensor([[-1.0]]), one(3, 5)[..., None],
                 one(1, 10)[..., None], torch.tensor([0.5]), None, None, False)
    s2 = 6 * torch.exp(torch.tensor(-1.0, dtype=F)) + 5
    assert r["out"][0].flatten().tolist() == [7.0, float(10 * s2 + 0.5)]
    assert float(r["state"][0]) == float(s2)


def test_conv_by_hand():
    # two taps, carried row 7: y0 = 2*7 + 3*1 + 1, y1 = 2*1 + 3*4 + 1; the next call carries 4
    x = torch.tensor([1.0, 4.0]).view(2, 1, 1)
    r = ref.conv(x, torch.tensor([[2.0], [3.0]]), torch.tensor([1.0]), None,
                 state=torch.tensor([[[7.0]]]))
    assert r["y"][0].flatten().tolist() == [18.0, 15.0]
    assert r["state"][0].flatten().tolist() == [4.0]
