"""The delta rule, the norms, the convolution and the products together: the example stack's prompt, tokens and
gradients, and the same calls recorded into a HIP graph."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from .gpu_util import announce
from .ssm_ref import F

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("delta_block",
                                                  os.path.join(ROOT, "examples", "delta_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def unit(v):
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) + 1e-6)


def rms(v):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)


def plain_block(block, y, s, p):
    """(y, s) in 64 bits on the CPU, differentiable, row by row."""
    S, B, _ = y.shape
    W, H, G, K, V, N = block.taps, block.H, block.G, block.K, block.V, block.channels
    s = y if s is None else s + y
    c, z, dt, b = (rms(s) * p["pre"] @ p["in"].t()).split([N, H * V, H, H], -1)
    rows = torch.cat([torch.zeros((W - 1, B, N), dtype=F), c])
    pre = sum(p["conv"][k] * rows[k:k + S] for k in range(W)) + p["conv_bias"]
    q, k, v = (pre * torch.sigmoid(pre)).split([G * K, G * K, H * V], -1)
    spread = lambda t: unit(t.unflatten(-1, (G, K))).repeat_interleave(H // G, dim=2)  # noqa: E731
    q, k, v = spread(q) * K ** -0.5, spread(k), v.unflatten(-1, (H, V))
    a, beta = torch.exp(p["A"] * torch.nn.functional.softplus(dt + p["dt_bias"])), torch.sigmoid(b)
    state, out = torch.zeros((B, H, K, V), dtype=F), []
    for t in range(S):
        state = a[t][..., None, None] * state
        u = beta[t][..., None] * (v[t] - (k[t][..., None] * state).sum(2))
        state = state + k[t][..., None] * u[..., None, :]
        out.append((q[t][..., None] * state).sum(2))
    o = (rms(torch.stack(out)) * p["post"]).flatten(2) * z * torch.sigmoid(z)
    return o @ p["out"].t(), s


def plain(stack, x, params, last):
    s = None
    for block, p in zip(stack.blocks, params):
        x, s = plain_block(block, x, s, p)
    return rms(x + s) * last


def wide(stack):
    return [{k: v.detach().cpu().to(F).requires_grad_() for k, v in b.p.items()} for b in stack.blocks], \
        stack.last.detach().cpu().to(F).requires_grad_()


def near(got, want, bound, name):
    off = (got.detach().cpu().to(F) - want).norm() / want.norm()
    assert off < bound, f"{name}: {off}"


def test_stack_forward_backward_and_tokens():
    """Two blocks. A block rounds six tensors to 16 bits on the way (the sum, h, its product, the convolution, o, the
    gated norm, and y), each by at most 2^-11 of a value: with the last norm 15 in all, and as many again for a
    gradient. Roundings are independent and the norms keep relative errors as they are, so their plain sum is
    well above what comes out."""
    m = example()
    stack = m.Stack(2, 48, 4, 2, 16, 24, dtype=torch.float16, seed=3)
    g = torch.Generator().manual_seed(4)
    x, go = torch.randn((75, 2, 48), generator=g).half(), torch.randn((75, 2, 48), generator=g).half()
    params, last = wide(stack)
    x64 = x.to(F).requires_grad_()
    want = plain(stack, x64, params, last)
    want.backward(go.to(F))
    announce("stack forward and backward")
    out, kept = stack.forward(x.cuda())
    gx, glast, grads = stack.backward(go.cuda(), kept)
    torch.cuda.synchronize()
    near(out, want.detach(), 15 * 2.0 ** -11, "out")
    near(gx, x64.grad, 30 * 2.0 ** -11, "gx")
    near(glast, last.grad, 30 * 2.0 ** -11, "glast")
    for i, (got, p) in enumerate(zip(grads, params)):
        for k, v in got.items():
            near(v, p[k].grad, 30 * 2.0 ** -11, f"{k} of block {i}")
    announce("stack prompt and tokens")
    whole, end = stack.prompt(x.cuda())
    assert torch.equal(whole, out)
    part, state = stack.prompt(x[:68].cuda())
    tokens = torch.stack([stack.token(x[t].cuda(), state) for t in range(68, 75)])
    near(torch.cat([part, tokens]), want.detach(), 15 * 2.0 ** -11, "prompt and tokens")
    for a, b in zip(state, end):
        near(a.delta, b.delta.cpu().to(F), 15 * 2.0 ** -11, "state")


def test_ragged_prompt_continues():
    m = example()
    stack = m.Stack(2, 32, 4, 4, 8, 16, seed=5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((70, 3, 32), generator=g).bfloat16().cuda()
    lengths = torch.tensor([70, 0, 7], device="cuda")
    out, state = stack.prompt(x, lengths=lengths)
    for b, n in enumerate(lengths.tolist()):
        if not n:
            assert all(not s.delta[b].any() and not s.conv[:, b].any() for s in state)
            continue
        alone, one = stack.prompt(x[:n, b:b + 1].contiguous())
        near(out[:n, b], alone[:, 0].cpu().to(F), 15 * 2.0 ** -8, "rows")
        near(state[0].delta[b], one[0].delta[0].cpu().to(F), 1e-5, "state of one")
        assert torch.equal(state[0].conv[:, b], one[0].conv[:, 0])


def test_graph_replays():
    m = example()
    stack = m.Stack(2, 64, 4, 2, 32, 32, seed=7)
    g = torch.Generator().manual_seed(8)
    x = torch.randn((330, 2, 64), generator=g).bfloat16().cuda()
    go = torch.randn((330, 2, 64), generator=g).bfloat16().cuda()

    def step():
        out, kept = stack.forward(x)
        gx, glast, grads = stack.backward(go, kept)
        return [out, gx, glast, *(v for d in grads for v in d.values())]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    announce("capture of the stack's forward and backward")
    with torch.cuda.graph(graph, stream=side):
        got = step()
    torch.cuda.synchronize()
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        junk = torch.randn(1 << 20, device="cuda") * 2  # unrelated eager work
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk).all()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {rep}"


def test_token_in_a_graph_advances_its_state():
    m = example()
    stack = m.Stack(2, 64, 4, 2, 32, 32, seed=9)
    x = torch.randn((6, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    eager, st = [], stack.state(4)
    for t in range(6):
        eager.append(stack.token(x[t], st))
    st2, row = stack.state(4), x[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = stack.token(row, st2)
    for t in range(6):
        row.copy_(x[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[t]), t
    for a, b in zip(st, st2):
        assert torch.equal(a.delta, b.delta) and torch.equal(a.conv, b.conv)
