"""The operators together: the example block's prompt, tokens and gradients, the same calls recorded
into a HIP graph, and on a stream that is not torch's current one."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from . import ssm_ref as ref
from .gpu_util import announce

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("ssm_block",
                                                  os.path.join(ROOT, "examples", "ssm_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(block, x, p):
    """The block in 64 bits on the CPU, differentiable, row by row."""
    S, B, _ = x.shape
    W, R, N, H = block.taps, block.rank, block.states, block.inner
    u, z = (x @ p["in"].t()).chunk(2, -1)
    rows = torch.cat([torch.zeros((W - 1, B, H), dtype=ref.F), u])
    pre = sum(p["conv"][k] * rows[k:k + S] for k in range(W)) + p["conv_bias"]
    c = pre * torch.sigmoid(pre)
    r, Bm, Cm = (c @ p["x"].t()).split([R, N, N], -1)
    d = torch.nn.functional.softplus(r @ p["dt"].t() + p["dt_bias"])
    s, ys = torch.zeros((B, N, H), dtype=ref.F), []
    for t in range(S):
        s = torch.exp(d[t][:, None] * p["A"]) * s + (d[t] * c[t])[:, None] * Bm[t][:, :, None]
        ys.append((Cm[t][:, :, None] * s).sum(1) + p["D"] * c[t])
    y = torch.stack(ys) * z * torch.sigmoid(z)
    return y @ p["out"].t() + x


def near(got, want, bound, name):
    off = (got.detach().cpu().double() - want).norm() / want.norm()
    assert off < bound, f"{name}: {off}"


def test_block_forward_backward_and_tokens():
    m = example()
    block = m.Block(48, 96, states=8, taps=4, dtype=torch.float16, seed=3)
    g = torch.Generator().manual_seed(4)
    x, go = torch.randn((37, 2, 48), generator=g).half(), torch.randn((37, 2, 48), generator=g).half()
    p = {k: v.detach().cpu().double().requires_grad_() for k, v in block.p.items()}
    x64 = x.double().requires_grad_()
    want = plain(block, x64, p)
    want.backward(go.double())
    announce("block forward and backward")
    out, kept = block.forward(x.cuda())
    gx, grads = block.backward(go.cuda(), kept)
    torch.cuda.synchronize()
    # five 16-bit roundings (2^-11 each) on the way to an output, about ten to a gradient, in sums
    # whose roundings are independent
    near(out, want.detach(), 5 * 2.0 ** -11, "out")
    near(gx, x64.grad, 10 * 2.0 ** -11, "gx")
    for k, v in grads.items():
        near(v, p[k].grad, 10 * 2.0 ** -11, k)
    announce("block prompt and tokens")
    whole, end = block.prompt(x.cuda())
    part, state = block.prompt(x[:30].cuda())
    tokens = torch.stack([block.token(x[t].cuda(), state) for t in range(30, 37)])
    near(torch.cat([part, tokens]), want.detach(), 5 * 2.0 ** -11, "prompt and tokens")
    near(state.scan, end.scan.cpu().double(), 5 * 2.0 ** -11, "state")


def test_ragged_prompt_continues():
    m = example()
    block = m.Block(32, 64, states=4, seed=5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((20, 3, 32), generator=g).bfloat16().cuda()
    lengths = torch.tensor([20, 0, 7], device="cuda")
    _, state = block.prompt(x, lengths=lengths)
    for b, n in enumerate(lengths.tolist()):
        if n:
            _, one = block.prompt(x[:n, b:b + 1].contiguous())
            assert torch.equal(state.conv[:, b], one.conv[:, 0])
            near(state.scan[b], one.scan[0].cpu().double(), 1e-5, "state of one")
        else:
            assert not state.scan[b].any() and not state.conv[:, b].any()


def test_graph_replays():
    m = example()
    block = m.Block(64, 128, states=16, seed=7)
    g = torch.Generator().manual_seed(8)
    x = torch.randn((530, 2, 64), generator=g).bfloat16().cuda()  # long enough to be cut into chunks
    go = torch.randn((530, 2, 64), generator=g).bfloat16().cuda()

    def step():
        out, kept = block.forward(x)
        gx, grads = block.backward(go, kept)
        return [out, gx, *grads.values()]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    announce("capture of the block's forward and backward")
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
    block = m.Block(64, 128, states=16, seed=9)
    x = torch.randn((6, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    eager, st = [], block.state(4)
    for t in range(6):
        eager.append(block.token(x[t], st))
    st2, row = block.state(4), x[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = block.token(row, st2)
    for t in range(6):
        row.copy_(x[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[t]), t
    assert torch.equal(st2.scan, st.scan) and torch.equal(st2.conv, st.conv)


def test_other_stream():
    """What a call allocates belongs to the stream given."""
    g = torch.Generator().manual_seed(2)
    S, B, H, N = 1200, 1, 128, 16
    x, dt, z, go = (torch.randn((S, B, H), generator=g).bfloat16().cuda() for _ in range(4))
    Bm, Cm = (torch.randn((S, B, N), generator=g).bfloat16().cuda() for _ in range(2))
    A, w = -torch.rand((N, H), generator=g).cuda() - 0.1, torch.randn((4, H), generator=g).bfloat16().cuda()
    q = torch.randn((96, H), generator=g).bfloat16().cuda()

    def calls(stream=None):
        c = mdc.conv_act_forward(x, w, stream=stream)
        out, saved = mdc.scan_forward(c, dt, A, Bm, Cm, z=z, return_saved=True, stream=stream)
        gr = mdc.scan_backward(go, c, dt, A, Bm, Cm, saved, z=z, stream=stream)
        lo = mdc.linear_forward(out, q, stream=stream)
        lg = mdc.linear_backward(lo, out, q, stream=stream)
        cg = mdc.conv_act_backward(gr.x, x, w, stream=stream)
        return [c, out, lo, *(t for t in (*gr, *lg, *cg) if t is not None)]

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(3):
        side.wait_stream(torch.cuda.current_stream())
        announce(f"side stream, rep {rep}")
        got = calls(side)
        for _ in range(30):  # work on the current stream with blocks of every size
            for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
