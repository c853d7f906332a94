"""The example's latent-attention layer: a prompt and single tokens, expanded and absorbed, against one prompt of all."""
import importlib.util
import os

import pytest
import torch

from sparse_moe_expert_k3moe_gb300 import build as kbuild

d, H = 256, 4


def example():
    kbuild.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def layer(mod, n_seq, max_len, T_max, device="cuda"):
    cfg = mod.k3.k3moe_config(d=d, f=128, n_experts=4, top_k=4, n_shared=1)   # all of them: no ties to fall either way
    return mod.LatentLayer(d, H, cfg, n_seq, max_len, T_max, 16, device)


def test_layer_is_laid_out_without_a_gpu():
    made = layer(example(), 2, 40, 6, "cpu")
    assert tuple(made.cache.shape) == (6, 16, 576) and tuple(made.pages.shape) == (2, 3)
    assert sorted(made.pages.flatten().tolist()) == list(range(6))


# What a token meets on its way (h, q, c, the row, absorbed q or keys and values, o and the attended latent, y, z, h
# again, the experts' input) is rounded to bf16 some ten times in either form, 2^-8 each at most of an element and 2^-9.8 rms; what
# goes into the residual stream beside x, of about its size, is off by less than the sum of ten roundings.
TOL = 10 * 2.0 ** -8


@pytest.mark.gpu
def test_prompt_then_captured_steps():
    torch.manual_seed(5)
    mod = example()
    lens, steps = [61, 30], 5
    whole = [n + steps for n in lens]
    made = layer(mod, 2, max(whole), sum(whole)).randomise(2)
    x = [torch.randn(n, d, device="cuda").bfloat16() for n in whole]
    want = made.prompt(torch.cat(x), *mod.places(whole)).clone().split(whole)
    made.cache.fill_(float("nan"))                        # what is read has been written
    made.prompt(torch.cat([t[:n] for t, n in zip(x, lens)]), *mod.places(lens))
    token = torch.stack([t[n] for t, n in zip(x, lens)])
    graph = made.capture(token)
    for i in range(steps):
        token.copy_(torch.stack([t[n + i] for t, n in zip(x, lens)]))
        graph.replay()
        for s, n in enumerate(lens):
            ref = want[s][n + i].double()
            err = (token[s].double() - ref).norm() / ref.norm()
            assert torch.isfinite(token).all() and err <= TOL, f"step {i}, sequence {s}: {err:.3e}"
    assert made.lens.tolist() == whole


def test_slots_past_the_pages():
    """Tokens that no page holds are written nowhere, and indexed nowhere."""
    made = layer(example(), 2, 40, 6, "cpu")                 # three pages of 16 each
    sequences, positions = torch.tensor([0, 1, 1, 0, 1, 0, 2, -1]), torch.tensor([0, 47, 17, 48, 1 << 30, -1, 5, 5], dtype=torch.int32)
    want = [made.pages[0, 0] * 16, made.pages[1, 2] * 16 + 15, made.pages[1, 1] * 16 + 1, -1, -1, -1, -1, -1]
    assert made._slots(sequences, positions).tolist() == [int(x) for x in want]


def test_step_with_full_pages_is_laid_out():
    made = layer(example(), 2, 40, 6, "cpu")
    made._half = lambda x, attend: x
    made.lens.copy_(torch.tensor([48, 7]))
    made.step(torch.zeros(2, d, dtype=torch.bfloat16))
    assert made.lens.tolist() == [49, 8]


@pytest.mark.gpu
def test_step_with_full_pages():
    """The full sequence is left out and reported, the other one goes on; nothing but its row is written."""
    mod = example()
    made = layer(mod, 2, 40, 60).randomise(3)
    made.prompt(torch.randn(55, d, device="cuda").bfloat16(), *mod.places([48, 7]))
    assert mod.k3.k3moe_device_status(made.attn.ws) == (0, 0)
    cache, token = made.cache.clone(), torch.randn(2, d, device="cuda").bfloat16()
    made.step(token)
    assert mod.k3.k3moe_device_status(made.attn.ws) == (6, 0x2)
    written = (made.cache != cache).any(-1).flatten().nonzero().flatten()
    assert written.tolist() == [int(made.pages[1, 0]) * 16 + 7]
    assert torch.isfinite(token[1]).all()
