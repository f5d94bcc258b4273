"""How the delta rule and the norms are called: what the front end refuses, streams, graphs, versions, and that nothing is
left behind."""
from __future__ import annotations

import gc
import sys

import pytest
import torch

import masked_depthwise_causal_amd as mdc

from .gpu_util import announce

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def t(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt, device="cuda")


def rule(**kw):
    a = dict(q=t(5, 2, 2, 16), k=t(5, 2, 2, 16), v=t(5, 2, 4, 24), dt=t(5, 2, 4), b=t(5, 2, 4), A=t(4, dt=F32))
    a.update(kw)
    return mdc.delta_forward(**a)


def token(**kw):
    a = dict(state=t(2, 4, 16, 24, dt=F32), q=t(2, 2, 16), k=t(2, 2, 16), v=t(2, 4, 24), dt=t(2, 4), b=t(2, 4),
             A=t(4, dt=F32))
    a.update(kw)
    return mdc.delta_step(**a)


def pre(**kw):
    a = dict(x=t(6, 32), weight=t(32))
    a.update(kw)
    return mdc.prenorm_forward(**a)


def post(**kw):
    a = dict(x=t(6, 32), weight=t(32))
    a.update(kw)
    return mdc.postnorm_forward(**a)


@pytest.mark.parametrize("call,kw,error,text", [
    (rule, lambda: dict(k=t(5, 2, 2, 15)), ValueError, r"k has shape \(5, 2, 2, 15\)"),
    (rule, lambda: dict(v=t(5, 2, 4)), ValueError, r"v must be \[S,B,H,V\]"),
    (rule, lambda: dict(q=t(5, 2, 32)), ValueError, r"q must be \[S,B,G,K\]"),
    (rule, lambda: dict(q=t(5, 2, 2, 32)[..., ::2]), ValueError, "q's last dimension must be contiguous"),
    (rule, lambda: dict(dt=t(5, 2, 3)), ValueError, "dt has shape"),
    (rule, lambda: dict(b=t(5, 2, 4, dt=F32)), ValueError, "b has dtype"),
    (rule, lambda: dict(A=t(4)), ValueError, "A has dtype"),
    (rule, lambda: dict(dt_bias=t(3, dt=F32)), ValueError, "dt_bias has shape"),
    (rule, lambda: dict(state=t(2, 4, 24, 16, dt=F32)), ValueError, "state has shape"),
    (rule, lambda: dict(lengths=t(2, dt=torch.int32)), ValueError, "lengths has dtype"),
    (rule, lambda: dict(out=t(5, 2, 4, 23)), ValueError, "out has shape"),
    (rule, lambda: dict(q=t(5, 2, 3, 16), k=t(5, 2, 3, 16)), mdc.MccbError, None),  # 4 heads of 3 key heads
    (rule, lambda: dict(q=t(5, 2, 2, 130), k=t(5, 2, 2, 130)), mdc.MccbError, None),
    (rule, lambda: dict(v=t(5, 2, 4, 257)), mdc.MccbError, None),
    (rule, lambda: dict(scale=float("inf")), mdc.MccbError, None),
    (token, lambda: dict(state=t(2, 4, 16, 24)), ValueError, "state has dtype"),
    (token, lambda: dict(state=t(4, 2, 16, 24, dt=F32).transpose(0, 1)), ValueError, "state must be contiguous"),
    (token, lambda: dict(q=t(1, 2, 2, 16)), ValueError, r"q must be \[B,G,K\]"),
    (pre, lambda: dict(weight=t(16)), ValueError, "weight has shape"),
    (pre, lambda: dict(weight=t(32, dt=torch.float16)), ValueError, "weight has dtype"),
    (pre, lambda: dict(residual=t(6, 31)), ValueError, "residual has shape"),
    (pre, lambda: dict(x=t(6, 64)[:, ::2]), ValueError, "contiguous"),
    (pre, lambda: dict(x=t(32)), ValueError, "two dimensions"),
    (pre, lambda: dict(eps=0.0), mdc.MccbError, None),
    (pre, lambda: dict(x=t(2, 16385), weight=t(16385)), mdc.MccbError, None),
    (post, lambda: dict(groups=5), ValueError, "groups must divide"),
    (post, lambda: dict(groups=0), ValueError, "groups must divide"),
    (post, lambda: dict(weight=t(16)), ValueError, "weight has shape"),
    (post, lambda: dict(z=t(5, 32)), ValueError, "z has shape"),
    (post, lambda: dict(scale=t(16)), ValueError, "scale has shape"),
])
def test_refuses(call, kw, error, text):
    kw = kw()
    with pytest.raises(error, match=text):
        call(**kw)


def test_refuses_outputs_over_inputs_and_what_was_not_saved():
    x, w = t(6, 32), t(32)
    with pytest.raises(mdc.MccbError):
        mdc.prenorm_forward(x, w, out=x)
    v = t(5, 2, 4, 24)
    with pytest.raises(mdc.MccbError):
        rule(v=v, out=v)
    q, d, A = t(5, 2, 2, 16), t(5, 2, 4), t(4, dt=F32)
    with pytest.raises(ValueError, match="saved has shape"):
        mdc.delta_backward(v, q, q, v, d, d, A, t(16, dt=torch.uint8))
    _, saved = rule(return_saved=True)
    with pytest.raises(ValueError, match="saved must be contiguous|saved has shape"):
        mdc.delta_backward(v, q, q, v, d, d, A, saved[::2])


def values(seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, dt=BF):
        return torch.randn(shape, generator=g).to(dt).cuda()

    S, B, G, H, K, V = 150, 2, 2, 4, 32, 40
    return {"q": r(S, B, G, K), "k": r(S, B, G, K), "v": r(S, B, H, V), "dt": r(S, B, H), "b": r(S, B, H),
            "A": -r(H, dt=F32).abs() - 0.1, "go": r(S, B, H, V), "state": r(B, H, K, V, dt=F32), "w": r(V), "z": r(S, B, H * V),
            "w2": r(H * V), "x": r(S, B, H * V), "sc": r(H * V)}


def calls(v, stream=None):
    s = {"stream": stream}
    ins = (v["q"], v["k"], v["v"], v["dt"], v["b"], v["A"])
    out, fs, saved = mdc.delta_forward(*ins, state=v["state"], return_state=True, return_saved=True, **s)
    g = mdc.delta_backward(v["go"], *ins, saved, state=v["state"], gradFinalState=v["state"], **s)
    one = mdc.delta_step(fs, *(x[0] for x in ins[:5]), v["A"], **s)
    p, total = mdc.prenorm_forward(v["x"], v["w2"], residual=v["z"], scale=v["sc"], return_sum=True, **s)
    pg = mdc.prenorm_backward(p, v["x"], v["w2"], residual=v["z"], scale=v["sc"], gradSum=total, **s)
    n = mdc.postnorm_forward(v["x"], v["w"], z=v["z"], residual=v["x"], scale=v["sc"], groups=4, **s)
    ng = mdc.postnorm_backward(n, v["x"], v["w"], z=v["z"], scale=v["sc"], groups=4, **s)
    return [out, fs, one, p, total, n, *(x for x in (*g, *pg, *ng) if x is not None)]


def test_calls_run_on_the_stream_that_is_given():
    """On the side stream the inputs are rewritten after a delay, so a call that ran anywhere else would read what they
    held before."""
    old, new = values(1), values(2)
    want = [x.clone() for x in calls({k: x.clone() for k, x in new.items()})]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    announce("calls behind a delay on a side stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        for k in old:
            old[k].copy_(new[k])
    got = calls(old, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_a_call_allocates_belongs_to_its_stream():
    v = values(3)
    want = calls(v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(3):
        side.wait_stream(torch.cuda.current_stream())
        announce(f"side stream, rep {rep}")
        got = calls(v, side)
        for _ in range(30):
            for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs_replay():
    """Two graphs of one pool, replayed in turns with eager work between, against the eager results."""
    vs = [values(4), values(5)]
    want = [calls({k: x.clone() for k, x in v.items()}) for v in vs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, got, pool = [], [], None
    for v in vs:
        graph = torch.cuda.CUDAGraph()
        announce("capture")
        with torch.cuda.graph(graph, stream=side, pool=pool):
            got.append(calls(v))
        pool = graph.pool()
        graphs.append(graph)
    torch.cuda.synchronize()
    for rep in range(4):
        for i in (0, 1):
            for x in got[i]:
                x.fill_(float("nan"))
            junk = torch.randn(1 << 20, device="cuda") * 2
            torch.cuda.synchronize()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.isfinite(junk).all()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])), (rep, i)


def test_token_in_a_graph_advances_its_state():
    v = values(6)
    rows = [tuple(v[n][r].clone() for n in ("q", "k", "v", "dt", "b")) for r in range(5)]
    s1, s2 = v["state"].clone(), v["state"].clone()
    eager = [mdc.delta_step(s1, *r, v["A"]) for r in rows]
    held = tuple(x.clone() for x in rows[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = mdc.delta_step(s2, *held, v["A"])
    for r, want in zip(rows, eager):
        for x, y in zip(held, r):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(s1, s2)


def test_writes_are_counted():
    out, fs, st, o1, y, s = t(5, 2, 4, 24), t(2, 4, 16, 24, dt=F32), t(2, 4, 16, 24, dt=F32), t(2, 4, 24), t(6, 32), t(6, 32)
    x = t(6, 32)
    before = [v._version for v in (out, fs, st, o1, y, s, x)]
    rule(out=out, final_state=fs)
    token(state=st, out=o1)
    pre(x=x, out=y, sum_out=s)
    assert [v._version for v in (out, fs, st, o1, y, s, x)] == [n + 1 for n in before[:6]] + [before[6]]
    post(x=x, out=y)
    assert y._version == before[4] + 2


def test_autograd_sees_that_a_state_moved_on():
    s = t(2, 4, 16, 24, dt=F32)
    leaf = torch.ones_like(s, requires_grad=True)
    loss = (leaf * s).sum()
    token(state=s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_leaves_nothing_behind():
    v = values(7)
    bad = t(16)

    def once():
        calls({k: x.clone() for k, x in v.items()})
        with pytest.raises(ValueError):
            pre(weight=bad)

    once()
    gc.collect()
    torch.cuda.synchronize()
    before, counts = torch.cuda.memory_allocated(), [sys.getrefcount(o) for o in (v["q"], v["w"], bad)]
    for _ in range(10):
        once()
    gc.collect()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    assert [sys.getrefcount(o) for o in (v["q"], v["w"], bad)] == counts


@pytest.mark.parametrize("S,B,H,G,K,V", [(700, 2, 8, 4, 128, 128), (1300, 1, 4, 4, 40, 70), (200, 20, 8, 8, 128, 128)])
def test_calls_at_once_give_the_same_bits(S, B, H, G, K, V):
    """On three streams, each with outputs and workspaces of its own."""
    g = torch.Generator(device="cuda").manual_seed(S)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, v, dt, b, go = (r(*s).to(BF) for s in ((S, B, G, K), (S, B, G, K), (S, B, H, V), (S, B, H), (S, B, H), (S, B, H, V)))
    A, state = -torch.rand(H, generator=g, device="cuda") * 4, r(B, H, K, V)

    def calls():
        out, end, saved = mdc.delta_forward(q, k, v, dt, b, A, state=state, return_state=True, return_saved=True)
        gr = mdc.delta_backward(go, q, k, v, dt, b, A, saved, state=state, gradFinalState=state)
        return [out, end, *(x for x in gr if x is not None)]

    want = calls()
    torch.cuda.synchronize()
    announce(f"three streams at once, S={S}")
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            got.append(calls())
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(x, y) for x, y in zip(one, want))
