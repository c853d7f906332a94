"""Refusals and sizes of the token mixer's entry points (no GPU needed): every check is on
the host and comes before any CUDA call."""
import ctypes

import pytest

from sparse_moe_expert_k3moe_gb300 import build as kbuild

A = 0x10000000      # a fake, 256-aligned address: never dereferenced on the host
BIG = 1 << 40
EINVAL, ESHAPE, EALIGN, EWORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def k3():
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    k3.lib()
    return k3


def vp(a):
    return ctypes.c_void_p(a) if a else None


def linear(k3, lc=None, T=4, x=A, xs=256, w=A, bias=A, res=A, rs=100, y=A + 4096, ys=100, ws=A, wb=BIG):
    lc = lc or k3.k3moe_linear_config(100, 256, "silu")
    return k3.lib().k3moe_linear(ctypes.byref(lc), T, vp(x), xs, vp(w), vp(bias), vp(res), rs, vp(y), ys, vp(ws), wb, None)


def test_linear_refusals(k3):
    cfg = k3.k3moe_linear_config
    for lc in (cfg(0, 256), cfg(100, 0), cfg(-1, 256), cfg(100, 256, 6), cfg(100, 256, -1), cfg(100, 256, 0, 2)):
        assert linear(k3, lc) == EINVAL
        with pytest.raises(k3.K3MoEError):
            k3.k3moe_linear_workspace_bytes(lc, 4)
    for lc in (cfg(100, 252), cfg((1 << 20) + 1, 256), cfg(100, 65544)):
        assert linear(k3, lc) == ESHAPE
    assert linear(k3, T=-1) == ESHAPE and linear(k3, T=(1 << 20) + 1) == ESHAPE
    assert linear(k3, x=0) == linear(k3, w=0) == linear(k3, y=0) == EINVAL
    assert linear(k3, xs=248) == linear(k3, xs=260) == linear(k3, ys=99) == linear(k3, rs=99) == ESHAPE
    assert linear(k3, xs=1 << 40) == linear(k3, ys=1 << 40) == linear(k3, rs=1 << 40) == ESHAPE
    assert linear(k3, res=A + 4096, rs=101) == EINVAL                 # y itself, with another stride
    assert linear(k3, x=A + 8) == linear(k3, w=A + 8) == linear(k3, y=A + 1) == linear(k3, bias=A + 2) == EALIGN
    assert linear(k3, cfg(100, 256, 0, 1), y=A + 2) == EALIGN
    assert linear(k3, ws=0) == linear(k3, ws=A + 8) == linear(k3, wb=256) == EWORKSPACE
    assert k3.lib().k3moe_linear(None, 4, vp(A), 8, vp(A), None, None, 0, vp(A), 8, vp(A), BIG, None) == EINVAL
    assert linear(k3, T=0, x=0, w=0, y=0, ws=0) == 0                  # nothing to do


def delta(k3, dc=None, n=3, T=10, start=A, q=A, qs=512, k=A, ks=512, v=A, vs=1024, g=A, beta=A, si=A, so=A, slots_n=8,
          slots=A, out=A, ws=A, wb=BIG):
    dc = dc or k3.k3moe_delta_config(8, 4)
    return k3.lib().k3moe_delta_rule(ctypes.byref(dc), n, T, vp(start), vp(q), qs, vp(k), ks, vp(v), vs, vp(g), vp(beta),
                                     vp(si), vp(so), slots_n, vp(slots), vp(out), vp(ws), wb, None)


def test_delta_refusals(k3):
    cfg = k3.k3moe_delta_config
    for dc in (cfg(0, 1), cfg(8, 0), cfg(8, 3), cfg(8, 4, head_dim=0), cfg(8, 4, gate_dim=2), cfg(8, 4, gate_dim=0),
               cfg(8, 4, qk_norm=2), cfg(8, 4, norm_eps=0.0), cfg(8, 4, norm_eps=float("inf")), cfg(8, 4, scale=float("nan"))):
        assert k3.k3moe_delta_validate_config(dc) == EINVAL
        assert delta(k3, dc) == EINVAL
        with pytest.raises(k3.K3MoEError):
            k3.k3moe_delta_workspace_bytes(dc, 1, 1)
    for dc in (cfg(8, 4, head_dim=64), cfg(2048, 1024)):
        assert k3.k3moe_delta_validate_config(dc) == ESHAPE
    assert k3.k3moe_delta_validate_config(cfg(8, 4, qk_norm=0, norm_eps=0.0)) == 0
    assert delta(k3, n=-1) == delta(k3, T=-1) == delta(k3, n=(1 << 16) + 1) == delta(k3, T=(1 << 20) + 1) == ESHAPE
    assert delta(k3, n=0) == ESHAPE and delta(k3, n=0, T=0, so=0, ws=0) == 0
    assert delta(k3, start=0) == EINVAL                               # 3 sequences, 10 tokens, no offsets
    assert delta(k3, so=0) == EINVAL
    for name in ("q", "k", "v", "g", "beta", "out"):
        assert delta(k3, **{name: 0}) == EINVAL
    assert delta(k3, qs=504) == delta(k3, ks=516) == delta(k3, vs=1016) == delta(k3, vs=1 << 40) == ESHAPE
    assert delta(k3, slots_n=0) == delta(k3, slots=0, slots_n=2) == ESHAPE
    for name in ("q", "k", "v", "g", "si", "so", "out"):
        assert delta(k3, **{name: A + 8}) == EALIGN
    assert delta(k3, beta=A + 2) == delta(k3, start=A + 2) == delta(k3, slots=A + 2) == EALIGN
    need = k3.k3moe_delta_workspace_bytes(cfg(8, 4), 3, 10)
    assert delta(k3, ws=0) == delta(k3, ws=A + 8) == delta(k3, wb=need - 1) == EWORKSPACE
    assert k3.lib().k3moe_delta_validate_config(None) == EINVAL


@pytest.mark.parametrize("gate", [1, 128])
def test_delta_workspace_covers_every_smaller_call(k3, gate):
    """The size for (n, T) serves every call of fewer sequences and tokens."""
    dc = k3.k3moe_delta_config(8, 4, gate_dim=gate)
    size = lambda n, T: k3.k3moe_delta_workspace_bytes(dc, n, T)  # noqa: E731
    grid = [(n, T) for n in (0, 1, 2, 7, 40, 300) for T in (0, 1, 31, 64, 65, 500, 1281, 10000)]
    for n, T in grid:
        for m, U in grid:
            if m <= n and U <= T:
                assert size(m, U) <= size(n, T), (m, U, n, T)
    for bad in ((-1, 4), (4, -1), ((1 << 16) + 1, 4), (1, (1 << 20) + 1)):
        with pytest.raises(k3.K3MoEError):
            size(*bad)
    with pytest.raises(k3.K3MoEError):
        k3.k3moe_linear_workspace_bytes(k3.k3moe_linear_config(8, 8), -1)


def test_holders_refuse_what_does_not_fit(k3):
    """The holders check what a pointer cannot say: types, shapes, strides, devices."""
    torch = pytest.importorskip("torch")
    op = k3.Linear(k3.k3moe_linear_config(32, 64), 8, device="cpu")
    x, y = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.bfloat16)
    op.w = torch.zeros(32, 64, dtype=torch.bfloat16)
    for kw in (dict(x=x.float()), dict(x=x[:, :56]), dict(x=torch.zeros(9, 64, dtype=torch.bfloat16)),
               dict(x=torch.zeros(64, 8, dtype=torch.bfloat16).t()), dict(y=y.float()), dict(y=y[:4]),
               dict(residual=y.float()), dict(residual=y[:, :8])):
        with pytest.raises(ValueError):
            op(kw.get("x", x), kw.get("y", y), residual=kw.get("residual"))
    op.w = torch.zeros(64, 32, dtype=torch.bfloat16).t()
    with pytest.raises(ValueError):
        op(x, y)
    dr = k3.DeltaRule(k3.k3moe_delta_config(4, 2), 3, 10, device="cpu")
    S = dr.new_state(3)
    good = dict(q=torch.zeros(10, 2, 128, dtype=torch.bfloat16), k=torch.zeros(10, 2, 128, dtype=torch.bfloat16),
                v=torch.zeros(10, 4, 128, dtype=torch.bfloat16), g=torch.zeros(10, 4, 1), beta=torch.zeros(10, 4),
                out=torch.zeros(10, 4, 128, dtype=torch.bfloat16), state_in=S, state_out=S.clone(),
                seq_start=torch.zeros(4, dtype=torch.int32), slots=torch.zeros(3, dtype=torch.int32))
    for name, bad in (("q", good["v"]), ("k", good["k"].float()), ("v", good["v"][:, :2]), ("g", torch.zeros(10, 4, 128)),
                      ("beta", torch.zeros(10, 4).double()), ("out", torch.zeros(10, 4, 256, dtype=torch.bfloat16)[..., :128]),
                      ("state_in", S[:2]), ("state_out", S.transpose(2, 3)), ("seq_start", torch.zeros(4)),
                      ("seq_start", torch.zeros(6, dtype=torch.int32)), ("slots", torch.zeros(2, dtype=torch.int32)),
                      ("q", torch.zeros(2, 10, 128, dtype=torch.bfloat16).transpose(0, 1))):
        with pytest.raises(ValueError):
            dr(**{**good, name: bad})
