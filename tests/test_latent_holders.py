"""The latent attention's holders against a config that changes after they were made (no GPU needed: nothing is launched)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def k3():
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    k3.lib()
    return k3


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def changed(op, config, call, changes):
    """call goes through as the config is, and is refused by the holder, before the library, while one of its numbers is
    another: the library would take the tensors for that size or type."""
    made = []
    op._run = lambda entry, args, stream: made.append(entry)
    call()
    assert len(made) == 1
    for name, value in changes:
        kept = getattr(config, name)
        setattr(config, name, value)
        with pytest.raises(ValueError):
            call()
        setattr(config, name, kept)
    assert len(made) == 1
    call()
    assert len(made) == 2


def test_norm_config_changes(k3):
    nc = k3.k3moe_norm_config(256, group=128)
    op = k3.Norm(nc, "cpu")
    op.post_gain, op.pre_gain = torch.ones(128), torch.ones(256)
    x, y, out = bf(3, 256), bf(3, 256), bf(3, 256)
    changed(op, nc, lambda: op(x, out=out, residual=y, total=y), [("n", 512), ("n", 128), ("group", 256), ("x_f32", 1), ("sum_f32", 1)])


def test_head_linear_config_changes(k3):
    hc = k3.k3moe_head_linear_config(8, 64, 128)
    op = k3.HeadLinear(hc, 4, "cpu")
    op.w = bf(8, 64, 128)
    x, y = bf(4, 8, 128), bf(4, 8, 64)
    changed(op, hc, lambda: op(x, y), [("n_heads", 16), ("n", 128), ("k", 256)])


def test_latent_config_changes(k3):
    lc = k3.k3moe_latent_config(8, page_size=32)
    op = k3.LatentAttention(lc, 3, 10, "cpu")
    op.gain, op.inv_freq = torch.ones(512), torch.ones(32, dtype=torch.float64)
    cache, slots = op.new_cache(4), torch.zeros(10, dtype=torch.int64)
    changes = [("n_heads", 16), ("page_size", 64)]
    changed(op, lc, lambda: op.write(bf(10, 576), i32(10), cache=cache, slots=slots, q=bf(10, 8, 64), q_rope=bf(10, 8, 64)), changes)
    changed(op, lc, lambda: op.attend(bf(10, 8, 576), cache, i32(3, 2), i32(3), bf(10, 8, 512), seq_start=i32(4)), changes)
    changed(op, lc, lambda: op.prompt(bf(10, 8, 192), bf(12, 8, 256), bf(12, 64), bf(10, 8, 128), seq_start=i32(4), kv_start=i32(4)), changes[:1])
    lc.page_size = 64
    assert tuple(op.new_cache(2).shape) == (2, 64, 576)
