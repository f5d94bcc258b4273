"""The delta rule's and the norms' 64-bit reference forms against differences of their own forward."""
from __future__ import annotations

import pytest
import torch

from . import delta_ref as ref
from .ssm_ref import F


def rand(g, *shape):
    return torch.randn(shape, generator=g, dtype=F)


def differences(f, ins, grads, g, h=1e-6):
    """d f along a random direction of every input against the gradients' product with it."""
    for name, x in ins.items():
        u = rand(g, *x.shape)
        up, down = f({**ins, name: x + h * u}), f({**ins, name: x - h * u})
        want, got = float((up - down) / (2 * h)), float((grads[name] * u).sum())
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), (name, got, want)


@pytest.mark.parametrize("normalize,softplus", [(True, True), (False, False)])
def test_delta(normalize, softplus):
    g = torch.Generator().manual_seed(3)
    S, B, H, G, K, V = 5, 2, 4, 2, 3, 4
    ins = {"q": rand(g, S, B, G, K), "k": rand(g, S, B, G, K) * 0.5, "v": rand(g, S, B, H, V), "dt": rand(g, S, B, H),
           "b": rand(g, S, B, H), "A": -torch.rand(H, generator=g, dtype=F) - 0.1, "dt_bias": rand(g, H),
           "state": rand(g, B, H, K, V)}
    go, gf, lengths = rand(g, S, B, H, V), rand(g, B, H, K, V), [5, 3]
    go[3:, 1] = 0

    def run(p, **kw):
        return ref.delta(p["q"], p["k"], p["v"], p["dt"], p["b"], p["A"], p["dt_bias"], softplus, normalize, None,
                         lengths, p["state"], **kw)

    r = run(ins, gout=go, gfinal=gf)
    grads = {n: r["g" + n] for n in ins}
    differences(lambda p: ((lambda o: (o["out"] * go).sum() + (o["state"] * gf).sum())(run(p))), ins, grads, g)
    assert not r["out"][3:, 1].any()


def test_norms():
    g = torch.Generator().manual_seed(4)
    ins = {"x": rand(g, 3, 12), "weight": rand(g, 12), "residual": rand(g, 3, 12), "scale": rand(g, 12)}
    go, gs = rand(g, 3, 12), rand(g, 3, 12)
    r = ref.prenorm(**ins, gout=go, gsum=gs)
    grads = {"x": r["gx"][0], "weight": r["gw"][0], "residual": r["gresidual"][0], "scale": r["gscale"][0]}
    differences(lambda p: (lambda o: (o["out"][0] * go).sum() + (o["sum"][0] * gs).sum())(ref.prenorm(**p)), ins, grads, g)
    for shared in (False, True):
        ins = {"x": rand(g, 3, 12), "weight": rand(g, 4 if shared else 12), "z": rand(g, 3, 12), "scale": rand(g, 12)}
        r = ref.postnorm(**ins, groups=3, gout=go)
        grads = {"x": r["gx"][0], "weight": r["gw"][0], "z": r["gz"][0], "scale": r["gscale"][0]}
        differences(lambda p: (ref.postnorm(**p, groups=3)["out"][0] * go).sum(), ins, grads, g)
