"""The mixer's operators among the library's other calls: a call that follows reads what
they wrote, whatever it may do before its own wait for them.

The forward's mat-vec path converts its tokens ahead of its wait for the routing.  After a
projection or a delta rule that writes these tokens it must not: here the tokens' buffer is
poisoned before the call that writes them, so that one element read too early makes the
output NaN, and the output is compared bit for bit with that of synchronised calls.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
D, HEADS = 128, 8
WIDTH = D * HEADS                       # of the experts' tokens
LONG = 32768                            # the projection's input width: it runs for tens of microseconds


@pytest.fixture(scope="module")
def k3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    return k3


def make_layer(k3, T, n_shared):
    """Random experts of moderate weights."""
    E, f = 64, 256
    g = torch.Generator("cuda").manual_seed(T)
    m = k3.MoELayer(k3.k3moe_config(d=WIDTH, f=f, n_experts=E, top_k=4, n_shared=n_shared), T)
    codes = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    scale = lambda *s: torch.full(s, 121, dtype=torch.uint8, device="cuda")  # noqa: E731
    w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).bfloat16()  # noqa: E731
    m.pack_experts(0, E, codes(E, f, WIDTH // 2), scale(E, f, WIDTH // 32), codes(E, f, WIDTH // 2),
                   scale(E, f, WIDTH // 32), codes(E, WIDTH, f // 2), scale(E, WIDTH, f // 32))
    m.w_router = w(E, WIDTH)
    if n_shared:
        m.sh_w1, m.sh_w3, m.sh_w2 = w(n_shared, f, WIDTH), w(n_shared, f, WIDTH), w(n_shared, WIDTH, f)
    return m


def writers(k3, T):
    """Calls that write the tokens x [T][WIDTH]: a projection of a long row, and the delta
    rule of one sequence of T tokens, or of single tokens."""
    h = torch.randn(T, LONG, device="cuda").bfloat16()
    proj = k3.Linear(k3.k3moe_linear_config(WIDTH, LONG), T)
    proj.w = (torch.randn(WIDTH, LONG, device="cuda") / LONG ** 0.5).bfloat16()
    mix = k3.DeltaRule(k3.k3moe_delta_config(HEADS, HEADS, gate_dim=D), T, T)
    q, k, v = (torch.randn(T, HEADS, D, device="cuda").bfloat16() for _ in range(3))
    gate, beta = torch.full((T, HEADS, D), -0.1, device="cuda"), torch.rand(T, HEADS, device="cuda")
    pool, after = torch.randn(T, HEADS, D, D, device="cuda"), torch.empty(T, HEADS, D, D, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lambda x: x.view(T, HEADS, D)  # noqa: E731
    return {"linear": lambda x: proj(h, x),
            "delta": lambda x: mix(q, k, v, gate, beta, out(x), pool, after),
            "sequence": lambda x: mix(q, k, v, gate, beta, out(x), pool, after, slots=one)}


@pytest.mark.parametrize("n_shared", [0, 2])
@pytest.mark.parametrize("T", [1, 3, 8, 24])
def test_forward_reads_what_the_mixer_wrote(k3, T, n_shared):
    layer = make_layer(k3, T, n_shared)
    x = torch.randn(T, WIDTH, device="cuda").bfloat16()
    layer.route(x)                                        # the routing is there before, as after a wider router
    out = torch.empty(T, WIDTH, device="cuda")
    for name, write in writers(k3, T).items():
        write(x)
        torch.cuda.synchronize()
        want_x = x.clone()
        torch.cuda.synchronize()
        want = layer.forward(x, out) or out.clone()
        torch.cuda.synchronize()
        assert torch.isfinite(want).all()
        for _ in range(20):
            x.fill_(float("nan"))
            write(x)
            layer.forward(x, out)
            assert torch.equal(x, want_x) and torch.equal(out, want), name
        # in a captured graph, where the calls are launched back to back
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            x.fill_(float("nan"))
            write(x)
            layer.forward(x, out)
            layer.forward(x, out)                         # and once more on the same tokens
        for _ in range(20):
            out.fill_(float("nan"))
            graph.replay()
            assert torch.equal(x, want_x) and torch.equal(out, want), name
    assert k3.k3moe_device_status(layer.ws) == (0, 0)


def test_forward_after_a_capture_that_routed(k3):
    """What a capture recorded says nothing of the calls around it: a projection before the
    capture, on its stream, is still waited for after it."""
    T = 8
    layer, write = make_layer(k3, T, 1), writers(k3, T)["linear"]
    x = torch.randn(T, WIDTH, device="cuda").bfloat16()
    layer.route(x)
    write(x)
    out, other, dst = torch.empty(T, WIDTH, device="cuda"), x.clone(), torch.empty(T, WIDTH, device="cuda")
    spare = make_layer(k3, T, 1)
    want = layer.forward(x, out) or out.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(10):
            x.fill_(float("nan"))
            write(x)
            graph = torch.cuda.CUDAGraph()
            graph.capture_begin()
            spare.route(other)
            spare.forward(other, dst)
            graph.capture_end()
            layer.forward(x, out)
            s.synchronize()
            assert torch.equal(out, want)


@pytest.mark.parametrize("T,n_seq", [(1, 1), (2, 2), (40, 1), (300, 2), (2000, 1)])
def test_a_chain_of_calls_reads_this_turns_results(k3, T, n_seq):
    """Projections, the delta rule, a projection and the router back to back on buffers that are
    used again: every turn's inputs differ, and nothing of the turn before is read."""
    heads = 4
    d = heads * D
    lin = lambda n, k, act, f32=False: k3.Linear(k3.k3moe_linear_config(n, k, act, f32), T)  # noqa: E731
    qkv, gate, step, proj = lin(3 * d, 512, "silu"), lin(d, 512, "logsigmoid", True), lin(heads, 512, "sigmoid", True), lin(d, d, "none")
    for op in (qkv, gate, step, proj):
        op.w = (torch.randn(op.lc.n, op.lc.k, device="cuda") / op.lc.k ** 0.5).bfloat16()
    gate.bias = torch.empty(d, device="cuda")
    mix = k3.DeltaRule(k3.k3moe_delta_config(heads, heads, gate_dim=D), n_seq, T)
    moe = k3.MoELayer(k3.k3moe_config(d=d, f=128, n_experts=32, top_k=4, n_shared=0), T)
    moe.w_router = (torch.randn(32, d, device="cuda") / d ** 0.5).bfloat16()
    start = torch.tensor([T * i // n_seq for i in range(n_seq + 1)], dtype=torch.int32, device="cuda")
    new = lambda n, kind=torch.bfloat16: torch.empty(T, n, dtype=kind, device="cuda")  # noqa: E731
    x, a, o, y = new(512), new(3 * d), new(d), new(d)
    g, b, bias = new(d, torch.float32), new(heads, torch.float32), torch.empty(d, device="cuda")
    state = mix.new_state(n_seq)

    def calls(meet):
        steps = [lambda: gate.bias.copy_(bias), lambda: qkv(x, a), lambda: gate(x, g), lambda: step(x, b),
                 lambda: mix(*(t.view(T, heads, D) for t in (a[:, :d], a[:, d:2 * d], a[:, 2 * d:])), g.view(T, heads, D), b,
                             o.view(T, heads, D), state, state, seq_start=start),
                 lambda: proj(o, y), lambda: moe.route(y)]
        for s in steps:
            s()
            if meet:
                torch.cuda.synchronize()

    outs = (a, g, b, o, y, state, moe.idx, moe.weight)
    turns = [(torch.randn(T, 512, device="cuda").bfloat16(), 3 + torch.randn(d, device="cuda")) for _ in range(6)]
    state.zero_()
    want = []
    for xt, bt in turns:
        x.copy_(xt)
        bias.copy_(bt)
        calls(True)
        want.append([t.clone() for t in outs])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(False)
    for run in (graph.replay, lambda: calls(False)):
        state.zero_()
        for (xt, bt), ref in zip(turns, want):
            x.copy_(xt)
            bias.copy_(bt)
            for t in (a, g, b, o, y):
                t.fill_(float("nan"))
            run()
            got = [t.clone() for t in outs]
            for i, (u, v) in enumerate(zip(got, ref)):
                assert torch.equal(u, v), i
    for op in (qkv, gate, step, proj, mix, moe):
        assert k3.k3moe_device_status(op.ws) == (0, 0)


_THREADS = r"""
import threading, torch
import sparse_moe_expert_k3moe_gb300 as k3
D, H, T = 128, 4, 100
g = torch.Generator("cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
x, w = {n: r(n, 16384).bfloat16() for n in (1, 2, 40, 700)}, r(512, 16384).bfloat16()
q, k, v, beta, state = r(T, H, D).bfloat16(), r(T, H, D).bfloat16(), r(T, H, D).bfloat16(), r(T, H).sigmoid(), r(1, H, D, D)
gates, one = {n: -r(T, H, n).abs() for n in (1, D)}, torch.zeros(1, dtype=torch.int32, device="cuda")
n = 8
results, meet = [None] * n, threading.Barrier(n)

def go(i):
    out = []
    with torch.cuda.stream(torch.cuda.Stream()):
        ops = [k3.Linear(k3.k3moe_linear_config(512, 16384), m) for m in x]
        mixes = [k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=G), 1, T) for G in gates]
        ys = [torch.zeros(m, 512, dtype=torch.bfloat16, device="cuda") for m in x]
        outs = [(torch.zeros_like(v), torch.zeros_like(state)) for _ in gates]
        torch.cuda.synchronize()
        if n > 1:
            meet.wait()
        for op, y, a in zip(ops, ys, x.values()):
            op.w = w
            op(a, y)
        for m, gate, (o, s) in zip(mixes, gates.values(), outs):
            m(q, k, v, gate, beta, o, state, s, slots=one)
        torch.cuda.synchronize()
    results[i] = ys + [t for pair in outs for t in pair]

threads = [threading.Thread(target=go, args=(i,)) for i in range(n)]
for t in threads:
    t.start()
for t in threads:
    t.join()
for other in results[1:]:
    assert all(torch.equal(a, b) for a, b in zip(results[0], other))
assert all(torch.isfinite(a).all() and a.any() for a in results[0])
print("threads agree")
"""


def test_first_calls_from_several_threads(k3):
    """The first calls of a process, eight threads at once, each on a stream of its own: what the
    library sets up on first use is there for all."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _THREADS], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "threads agree" in r.stdout, r.stdout + r.stderr
