"""The delta rule's chunk form on the GPU where chunks meet: decays that differ from chunk to
chunk, sequences of one chunk to many, and what lies behind a sequence's last token.

Tolerances as in test_gpu_mixer: the output's rounding to bf16, 2^-8 of a head's 2-norm, and
2e-5 of the state's (a step shrinks earlier errors, a chunk's float sums are of 64 to 128
products).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
D, C = 128, 64
OUT_TOL, STATE_TOL = 2.0 ** -8, 2e-5


@pytest.fixture(scope="module")
def k3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    return k3


def reference(q, k, v, g, beta, S):
    """(out [T][H][D], state [H][D][D]) of one sequence in float64, token by token."""
    q, k, v, g, beta, S = (t.double() for t in (q, k, v, g, beta, S))
    q, k = (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    out = torch.zeros_like(v)
    for t in range(q.shape[0]):
        S = S * g[t].exp().unsqueeze(-1)
        u = beta[t].unsqueeze(-1) * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t].unsqueeze(-1) * u.unsqueeze(-2)
        out[t] = torch.einsum("hk,hkv->hv", q[t] * D ** -0.5, S)
    return out, S


def inputs(T, H, channel, seed):
    r = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, device="cuda")  # noqa: E731
    q, k, v = (n(T, H, D).bfloat16() for _ in range(3))
    g = -torch.exp(2 * n(T, H, D if channel else 1) - 4)
    return q, k, v, g, torch.sigmoid(n(T, H))


def near(got, ref, tol, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got.double() - ref).norm() / ref.norm()
    assert err <= tol, f"{what}: {err:.3e} > {tol:.1e}"


def check(out, state, q, k, v, g, beta, S0, what):
    ref_out, ref_S = reference(q, k, v, g, beta, S0)
    for h in range(ref_S.shape[0]):
        near(out[:, h], ref_out[:, h], OUT_TOL, f"{what}, head {h}, out")
        near(state[h], ref_S[h], STATE_TOL, f"{what}, head {h}, state")


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("T", [64, 65, 130, 192, 3 * 64 + 1, 5 * 64, 6 * 64 + 33, 9 * 64 + 5, 16 * 64])
def test_every_chunk_decays_by_its_own(k3, T, channel):
    """Chunks that keep the state beside chunks that nearly forget it, in no simple turn: a
    chunk that took another one's decay would be off by far more than the tolerance."""
    H = 3
    q, k, v, g, beta = inputs(T, H, channel, T)
    for c in range((T + C - 1) // C):                     # one token of the chunk carries its decay
        g[c * C:(c + 1) * C] = 0
        for h in range(H):
            g[c * C + (7 * c + h) % min(C, T - c * C), h] = -[0.0, 4.0, 0.1, 1.0, 2.0][(2 * c + h) % 5]
    op = k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=D if channel else 1), 1, T)
    S0 = torch.randn(1, H, D, D, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out, state = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(S0)
        op(q, k, v, g, beta, out, S0, state, slots=one)
        check(out, state[0], q, k, v, g, beta, S0[0], f"{T} tokens")
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# In a call's tokens: sequences in chunks whose last one holds 1, 15, 16, 17, 63 or all of its 64
# tokens; None: tokens of no sequence.
AROUND = [[65, None], [70, 65, 90, None], [64, 33, None], [127, 128, 129, 15, None], [80, 81, 79, 48, 47, 49, None],
          [64 * 40 + 1, None]]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("lens", AROUND, ids=str)
def test_nothing_behind_a_sequence_takes_part(k3, lens, channel, value):
    """Every other sequence, the tokens after the last one and the tokens before the first are
    of values that no arithmetic survives; the sequences between them do not know."""
    H, Hq, before = 4, 2, 5
    n = len(lens) - 1
    sizes = [x if x else 70 for x in lens]
    T = before + sum(sizes)
    t0 = [before + sum(sizes[:i]) for i in range(n + 1)]
    q, k, v, g, beta = inputs(T, H, channel, n)
    q, k = q[:, :Hq].clone(), k[:, :Hq].clone()
    spoiled = torch.ones(T, dtype=torch.bool, device="cuda")
    for i in range(0, n, 2):
        spoiled[t0[i]:t0[i] + sizes[i]] = False
    for t in (q, k, v, g, beta):
        t[spoiled] = value
    if value == value:
        g[spoiled] = -value if value > 0 else value       # a decay's logarithm is not above zero
    op = k3.DeltaRule(k3.k3moe_delta_config(H, Hq, gate_dim=D if channel else 1), n, T)
    S0 = 0.5 * torch.randn(n, H, D, D, device="cuda")
    out, state = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.empty_like(S0)
    op(q, k, v, g, beta, out, S0, state, seq_start=torch.tensor(t0, dtype=torch.int32, device="cuda"))
    assert k3.k3moe_device_status(op.ws) == (0, 0)
    heads = lambda t: t.repeat_interleave(H // Hq, 1)  # noqa: E731
    for i in range(0, n, 2):
        s = slice(t0[i], t0[i] + sizes[i])
        check(out[s], state[i], heads(q[s]), heads(k[s]), v[s], g[s], beta[s], S0[i], f"sequence {i}")
    assert (out[:before] == 7).all() and (out[t0[n]:] == 7).all()


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "beta"])
def test_a_spoiled_token_reaches_no_other_chunk_or_sequence(k3, which, channel):
    """NaN in one token: with q that token's output alone, else nothing before the token's
    chunk and nothing of another sequence; bit for bit the same as without it."""
    H, lens, at = 2, [200, 130, 90], 200 + 64 + 20        # in the second sequence's second chunk
    T = sum(lens)
    given = dict(zip(("q", "k", "v", "g", "beta"), inputs(T, H, channel, 5)))
    op = k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=D if channel else 1), 3, T)
    start = torch.tensor([0, 200, 330, 420], dtype=torch.int32, device="cuda")
    S0 = torch.randn(3, H, D, D, device="cuda")

    def go():
        out, state = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(S0)
        op(**given, out=out, state_in=S0, state_out=state, seq_start=start)
        assert k3.k3moe_device_status(op.ws) == (0, 0)
        return out, state

    ref, ref_state = go()
    given[which] = given[which].clone()
    given[which][at] = float("nan")
    out, state = go()
    same = torch.ones(T, dtype=torch.bool, device="cuda")
    same[at if which == "q" else slice(264, 330)] = False
    same[at + 1:330] = which == "q"
    assert torch.equal(out[same], ref[same]) and torch.isnan(out[at]).all()
    keeps = [0, 1, 2] if which == "q" else [0, 2]
    assert torch.equal(state[keeps], ref_state[keeps])
    if which != "q":
        assert torch.isnan(out[at:330]).flatten(1).any(1).all() and torch.isnan(state[1]).any()
