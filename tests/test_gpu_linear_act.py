"""The activations of k3moe_linear in float, on a grid of z that the product gives exactly: each
within its own relative error, into the tails.

z has 16 significant bits and enters as two bf16 weights against ones, so that the sum is exact
in float whatever its order.  The tolerances, in units of 2^-23 of |act(z)|, are those of the
operations: the fast exponential errs by 2 + 1.173 |x| of them (its documented bound), the fast
division by 2, a rounding by a half.
  sigmoid, silu   an exponential of -z, an addition, a division, a product: 6 + 1.2 |z|
  logsigmoid      the same, then a series and an addition: 10 + 1.2 |z|
  gelu            exp(-z^2/2) by two products (an error of 1.25 z^2 / 2 units in the exponent)
                  and the exponential of 2 (1.5), a fraction (2), its polynomial (fitted to 1.3, rounded to
                  within 4 by the sum of its terms), two products: 10 + 0.7 z^2
Below 2^-119 a result may be zero (1 + exp(-z) is then past the division's range, or the
exponential below the smallest normal number).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def k3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    return k3


def grid():
    """z of 16 significant bits, float64: both signs, from 1e-6 to past where the tails vanish."""
    z = torch.cat([torch.logspace(-6, 0, 2000, dtype=torch.float64), torch.linspace(1, 16, 6000, dtype=torch.float64),
                   torch.linspace(16, 120, 2000, dtype=torch.float64)])
    m, e = torch.frexp(torch.cat([z, -z]))
    return torch.ldexp(torch.round(torch.ldexp(m, torch.tensor(16))), e - 16).cuda()


UNITS = {"none": lambda z: 0 * z, "relu": lambda z: 0 * z, "sigmoid": lambda z: 6 + 1.2 * z.abs(),
         "silu": lambda z: 6 + 1.2 * z.abs(), "logsigmoid": lambda z: 10 + 1.2 * z.abs(), "gelu": lambda z: 10 + 0.7 * z * z}


def act64(z, act):
    """In 64 bits, exact in relative terms on both sides."""
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.special.expit(z),
            "gelu": lambda: 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5), "sigmoid": lambda: torch.special.expit(z),
            "logsigmoid": lambda: z.clamp(max=0) - torch.log1p(torch.exp(-z.abs()))}[act]()


@pytest.mark.parametrize("T", [1, 2, 4, 40, 700])
@pytest.mark.parametrize("act", sorted(UNITS))
def test_activation_is_relatively_exact(k3, act, T):
    z = grid()
    w = torch.zeros(z.numel(), 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = z.bfloat16()
    w[:, 5] = (z - w[:, 0].double()).bfloat16()
    assert torch.equal(w.double().sum(1), z)
    op = k3.Linear(k3.k3moe_linear_config(z.numel(), 8, act, True), T)
    op.w = w
    y = op(torch.ones(T, 8, dtype=torch.bfloat16, device="cuda"), torch.empty(T, z.numel(), device="cuda"))
    ref = act64(z, act)
    tol = UNITS[act](z) * 2.0 ** -23 * ref.abs() + (2.0 ** -119 if act not in ("none", "relu") else 0)
    over = (y.double() - ref).abs() - tol
    worst = int(over.max(0).values.argmax())
    assert (over <= 0).all(), f"z = {float(z[worst]):.6g}: {float(y[0, worst]):.9g}, not {float(ref[worst]):.9g}"
