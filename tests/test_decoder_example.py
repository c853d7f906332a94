"""The example's decoder layer: against the formulas in 64 bits, a prompt against the same in
pieces, and its captured step against a plain one."""
import importlib.util
import os

import pytest
import torch

from sparse_moe_expert_k3moe_gb300 import build as kbuild

D, d, H, HQ = 128, 256, 4, 2


def example():
    kbuild.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def layer(mod, n_seq, T_max, device="cuda"):
    cfg = mod.k3.k3moe_config(d=d, f=128, n_experts=4, top_k=4, n_shared=1)   # all of them: no ties to fall either way
    return mod.DecoderLayer(d, H, HQ, cfg, n_seq, T_max, device)


def test_layer_is_laid_out_without_a_gpu():
    made = layer(example(), 2, 6, "cpu")
    assert made.qkv.lc.n == (2 * HQ + H) * D and made.gate.lc.y_f32 and made.proj.lc.n == made.qkv.lc.k == d
    assert tuple(made.state.shape) == (2, H, D, D)


def mixer64(made, x, lens, state):
    """x + o Wo^T in 64 bits; the operators' bf16 results (q, k, v and o) rounded as they are stored."""
    T, x = x.shape[0], x.double()
    z = x @ made.qkv.w.double().t()
    qkv = (z * torch.sigmoid(z)).bfloat16().double()
    q, k, v = qkv[:, :HQ * D].view(T, HQ, D), qkv[:, HQ * D:2 * HQ * D].view(T, HQ, D), qkv[:, 2 * HQ * D:].view(T, H, D)
    g = torch.nn.functional.logsigmoid(x @ made.gate.w.double().t() + made.gate.bias.double()).view(T, H, D)
    b = torch.sigmoid(x @ made.beta.w.double().t())
    q, k = (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(H // HQ, 1) for t in (q * D ** -0.5, k))
    o, state, t0 = torch.zeros(T, H, D, dtype=torch.float64, device=x.device), state.double(), 0
    for i, n in enumerate(lens):
        S = state[i]
        for t in range(t0, t0 + n):
            S = S * g[t].exp().unsqueeze(-1)
            u = b[t].unsqueeze(-1) * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
            S = S + k[t].unsqueeze(-1) * u.unsqueeze(-2)
            o[t] = torch.einsum("hk,hkv->hv", q[t], S)
        state[i], t0 = S, t0 + n
    return x + o.bfloat16().double().view(T, -1) @ made.proj.w.double().t(), state


# Each of q, k, v, o and y is rounded once to bf16 (up to 2^-8 of an element, 2^-9.8 rms): what a
# rounding that falls the other way changes stays below the sum of five of them, 5 * 2^-8; so do
# the routed experts' 5e-3 of their output.
TOL = 5 * 2.0 ** -8


def near(got, ref, tol=TOL):
    err = (got.double() - ref.double()).norm() / ref.double().norm()
    assert torch.isfinite(got).all() and err <= tol, f"{err:.3e} > {tol:.1e}"


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1, 1, 1], [150, 0, 33]])
def test_mixer_against_the_formulas(lens):
    torch.manual_seed(len(lens) + sum(lens))
    made = layer(example(), 3, sum(lens)).randomise(1)
    start = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), d, device="cuda").bfloat16()
    made.state.normal_().mul_(0.3)
    ref, ref_state = mixer64(made, x, lens, made.state)
    made.moe = lambda x, y: y.zero_()                                 # the first half alone
    near(made(x.clone(), None if max(lens) == 1 else start), ref)
    near(made.state, ref_state)


@pytest.mark.gpu
def test_prompt_then_captured_steps():
    """A prompt and four tokens, the tokens by replaying a captured step, as one prompt of all."""
    torch.manual_seed(5)
    n, T, steps = 2, 96, 4
    made = layer(example(), n, n * (T + steps)).randomise(2)
    x = torch.randn(n, T + steps, d, device="cuda").bfloat16()
    starts = lambda m: torch.arange(0, n * m + 1, m, device="cuda").int()  # noqa: E731
    whole = made(x.reshape(-1, d).clone(), starts(T + steps)).view(n, T + steps, d).clone()
    state = made.state.clone()
    made.state.zero_()
    made(x[:, :T].reshape(-1, d).clone(), starts(T))
    token = x[:, T].clone()
    graph = made.capture(token)
    for i in range(steps):
        token.copy_(x[:, T + i])
        graph.replay()
        near(token, whole[:, T + i])
    near(made.state, state)
