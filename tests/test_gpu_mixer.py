"""The token mixer's operators on the GPU (k3moe_linear, k3moe_delta_rule) against their
definitions in 64 bits.

Tolerances, from the arithmetic:
  linear: z is a float sum of K products.  A float addition errs by at most 2^-23 of the
    running sum (a tensor core may truncate), with signs that vary: 4 sqrt(K) 2^-23 of
    sum |x w| bounds the sum's error (four standard deviations of a random walk whose
    every step is the worst one).  The activations' slopes are at most 1.13, their own
    error and the epilogue's additions at most 2^-20 of the values they add, and a bf16
    result (8 significant bits) is off by 2^-8 of itself at most.
  delta rule: rounding out to bf16 costs at most 2^-8 of each element and less in the
    2-norm, float products next to nothing: 2-norm of the error over a head at most
    2^-8 of the result's.  The state takes float sums of up to 128 products (128 2^-24
    = 8e-6 at worst), and a step shrinks earlier errors (|k| <= 1, beta <= 1): 2e-5.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
D = 128
OUT_TOL, STATE_TOL = 2.0 ** -8, 2e-5


@pytest.fixture(scope="module")
def k3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    return k3


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ----------------------------------------------------------------------------- linear

def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.special.expit(z),
            "gelu": lambda: z * torch.special.ndtr(z), "sigmoid": lambda: torch.special.expit(z),
            "logsigmoid": lambda: -torch.logaddexp(torch.zeros_like(z), -z)}[act]()


def check_linear(y, x, w, bias, residual, act):
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ref = act64(z, act)
    tol = 1.13 * 4 * x.shape[1] ** 0.5 * 2.0 ** -23 * mag
    if residual is not None:
        tol = tol + 2.0 ** -20 * residual.double().abs()
        ref = ref + residual.double()
    tol = tol + 2.0 ** -20 * (z.abs() + ref.abs()) + 1e-30
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    bad = (y.double() - ref).abs() > tol
    assert torch.isfinite(y).all()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {((y.double() - ref).abs() / tol).max():.2f}"


LINEAR = [  # T, N, K, act, bias, residual, f32, x pad, y pad
    (1, 1, 8, "none", False, False, True, 0, 0),
    (1, 3584, 3584, "silu", True, False, False, 0, 0),
    (1, 257, 7168, "none", True, True, True, 8, 3),
    (2, 1000, 1024, "gelu", False, True, False, 0, 0),
    (3, 129, 4096, "sigmoid", True, False, True, 24, 1),
    (4, 77, 520, "none", False, True, False, 0, 7),
    (5, 4999, 256, "relu", True, True, False, 0, 0),
    (7, 128, 65536, "none", True, False, True, 0, 0),
    (8, 640, 3592, "silu", False, False, False, 0, 0),
    (16, 1344, 3584, "logsigmoid", True, False, True, 0, 0),
    (17, 333, 1992, "none", True, True, False, 16, 5),
    (31, 2048, 136, "silu", True, False, False, 0, 0),
    (48, 7168, 3584, "none", False, True, False, 0, 0),
    (64, 64, 64, "relu", True, True, True, 0, 0),
    (65, 1001, 72, "gelu", True, True, True, 0, 1),
    (100, 3333, 2048, "none", False, False, False, 0, 0),
    (127, 129, 8, "sigmoid", True, True, False, 8, 0),
    (128, 256, 8192, "silu", True, False, False, 0, 0),
    (129, 513, 1000, "gelu", True, True, False, 40, 3),
    (255, 1024, 1024, "none", True, True, True, 0, 0),
    (257, 4999, 712, "logsigmoid", True, False, True, 0, 0),
    (333, 300, 24, "none", True, True, False, 0, 0),
    (512, 7168, 1536, "none", False, True, False, 0, 0),
    (1003, 2500, 3584, "silu", True, True, False, 64, 12),
    (2048, 2048, 2048, "gelu", True, True, False, 0, 0),
    (4097, 1, 64, "sigmoid", True, False, True, 0, 0),
    (5000, 260, 136, "none", True, True, True, 8, 4),
    (4100, 1300, 520, "silu", True, True, False, 0, 0),      # several waves of tiles, ragged both ways
    (3001, 1537, 1096, "none", False, True, True, 8, 1),
    (19969, 200, 136, "gelu", True, False, False, 0, 0),
    (640, 6500, 264, "relu", True, True, False, 0, 0),
    (500, 9001, 2000, "none", True, True, True, 8, 3),       # pairs of blocks, ragged both ways
    (501, 9000, 2000, "gelu", True, True, False, 0, 0),
    (2047, 7169, 2048, "silu", True, False, False, 0, 1),    # and tile after tile
    (3, 2100, 4096, "silu", True, True, False, 0, 0),        # a few tokens, weights on either side of the rule
    (4, 2000, 4096, "silu", True, True, False, 0, 0),
    (9, 2000, 2048, "none", True, False, True, 0, 0),        # a cluster of six, eight
    (10, 1800, 8192, "none", True, True, False, 0, 0),
]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(v) for v in c))
def test_linear(k3, case):
    T, N, K, act, has_bias, has_res, f32, xpad, ypad = case
    g = gen(T * 7 + N)
    x = torch.randn(T, K + xpad, generator=g, device="cuda").bfloat16()[:, :K]
    w = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    kind = torch.float32 if f32 else torch.bfloat16
    bias = torch.randn(N, generator=g, device="cuda") if has_bias else None
    residual = torch.randn(T, N + 2 * ypad, generator=g, device="cuda").to(kind)[:, :N] if has_res else None
    op = k3.Linear(k3.k3moe_linear_config(N, K, act, f32), T)
    op.w, op.bias = w, bias
    wide = torch.full((T, N + ypad), 7.5, dtype=kind, device="cuda")
    y = op(x, wide[:, :N], residual=residual)
    check_linear(y, x, w, bias, residual, act)
    assert (wide[:, N:] == 7.5).all()                    # nothing is written beside the rows
    again = op(x, torch.empty((T, N), dtype=kind, device="cuda"), residual=residual)
    assert torch.equal(again, y)                         # and the sums' order is fixed
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_linear_unaligned_y_and_residual(k3):
    """y and residual need only their element's alignment."""
    T, N, K = 70, 250, 256
    g = gen(3)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(N, K, generator=g, device="cuda") / 16).bfloat16()
    for kind in (torch.bfloat16, torch.float32):
        buf = torch.zeros(T * N + 8, dtype=kind, device="cuda")
        res = torch.randn(T * N + 8, generator=g, device="cuda").to(kind)
        op = k3.Linear(k3.k3moe_linear_config(N, K, "none", kind == torch.float32), T)
        op.w = w
        for off in (1, 3):
            y, r = buf[off:off + T * N].view(T, N), res[off:off + T * N].view(T, N)
            op(x, y, residual=r)
            check_linear(y, x, w, None, r, "none")


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_linear_residual_in_place(k3, T):
    g = gen(T)
    x = torch.randn(T, 512, generator=g, device="cuda").bfloat16()
    w = (torch.randn(640, 512, generator=g, device="cuda") / 22).bfloat16()
    h = torch.randn(T, 640, generator=g, device="cuda").bfloat16()
    before = h.clone()
    op = k3.Linear(k3.k3moe_linear_config(640, 512), T)
    op.w = w
    op(x, h, residual=h)
    check_linear(h, x, w, None, before, "none")


@pytest.mark.parametrize("T", [1, 40, 200])
def test_linear_propagates_only_its_rows_and_columns(k3, T):
    """An infinity or NaN in one token's row or one weight row reaches that row or column
    of y alone (padding inside a tile takes no part)."""
    g = gen(T + 1)
    x = torch.randn(T, 192, generator=g, device="cuda").bfloat16()
    w = (torch.randn(200, 192, generator=g, device="cuda") / 14).bfloat16()
    x[T // 2, 5] = float("nan")
    w[131, 190] = float("inf")
    op = k3.Linear(k3.k3moe_linear_config(200, 192, "none", True), T)
    op.w = w
    y = op(x, torch.empty(T, 200, device="cuda"))
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[T // 2] = True
    want[:, 131] = True
    assert torch.equal(bad, want)


def test_linear_on_another_stream(k3):
    T, N, K = 90, 384, 2048
    x = torch.randn(T, K, device="cuda").bfloat16()
    w = (torch.randn(N, K, device="cuda") / 45).bfloat16()
    op = k3.Linear(k3.k3moe_linear_config(N, K, "silu"), T)
    op.w = w
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(s):
        op(x, y)
    z = torch.empty_like(y)
    op(x, z, stream=s)
    s.synchronize()
    check_linear(y, x, w, None, None, "silu")
    assert torch.equal(y, z)


# ----------------------------------------------------------------------------- delta rule

def delta64(q, k, v, g, beta, S, lens, slots, norm, scale, eps=1e-6):
    """(out, states [n][H][D][D]) in float64, token by token."""
    H, rep = v.shape[1], v.shape[1] // q.shape[1]
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    if norm:
        q = q / (q.pow(2).sum(-1, keepdim=True) + eps).sqrt()
        k = k / (k.pow(2).sum(-1, keepdim=True) + eps).sqrt()
    q, k = (q * scale).repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    S = S.clone()
    t0 = np.concatenate([[0], np.cumsum(lens)])
    for t in range(max(lens) if lens else 0):
        live = torch.tensor([i for i, n in enumerate(lens) if n > t], device=v.device)
        at = torch.tensor([int(t0[i]) + t for i, n in enumerate(lens) if n > t], device=v.device)
        W = S[live] * g[at].exp().unsqueeze(-1)
        u = beta[at].unsqueeze(-1) * (v[at] - torch.einsum("nhk,nhkv->nhv", k[at], W))
        W = W + k[at].unsqueeze(-1) * u.unsqueeze(-2)
        S[live] = W
        out[at] = torch.einsum("nhk,nhkv->nhv", q[at], W)
    return out, S


def delta_inputs(lens, H, Hq, channel, seed, bias=0.0, decay="mixed"):
    gn = gen(seed)
    T, G = sum(lens), D if channel else 1
    r = lambda *s: torch.randn(*s, generator=gn, device="cuda")  # noqa: E731
    qkv = r(T, (2 * Hq + H) * D)
    qkv[:, :2 * Hq * D] += bias                                       # keys that resemble one another
    qkv = qkv.bfloat16()
    q, k, v = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:2 * Hq * D].view(T, Hq, D), qkv[:, 2 * Hq * D:].view(T, H, D)
    if decay == "mixed":
        g = -torch.exp(r(T, H, G) * 2 - 3)                            # from none to a few per token
    elif decay == "none":
        g = torch.zeros(T, H, G, device="cuda")
    else:                                                             # strong: resets, and infinities
        g = -torch.exp(r(T, H, G) * 3 + 1)
        g[torch.rand(T, H, G, generator=gn, device="cuda") < 0.02] = -float("inf")
    return q, k, v, g, torch.sigmoid(r(T, H))


def check_delta(out, state, ref_out, ref_state, what=""):
    assert torch.isfinite(out).all() and torch.isfinite(state).all()
    for got, ref, tol, name in ((out, ref_out, OUT_TOL, "out"), (state, ref_state, STATE_TOL, "state")):
        dims = tuple(i for i in range(ref.dim()) if i != 1)           # every head on its own
        err = (got.double() - ref).pow(2).sum(dims).sqrt()
        norm = ref.pow(2).sum(dims).sqrt()
        assert (err <= tol * norm + 1e-30).all(), f"{what} {name}: {(err / norm).max():.3e} > {tol:.1e}"


def run_delta(k3, lens, H, Hq, channel, norm=1, seed=1, zero_state=False, in_place=False, start_given=True, **kw):
    q, k, v, g, beta = delta_inputs(lens, H, Hq, channel, seed, **kw)
    if not norm:
        k = (k.float() / k.float().norm(dim=-1, keepdim=True)).bfloat16()
    n, T = len(lens), sum(lens)
    dc = k3.k3moe_delta_config(H, Hq, gate_dim=D if channel else 1, qk_norm=norm)
    op = k3.DeltaRule(dc, n, T)
    gn = gen(seed + 100)
    slots = torch.randperm(n + 2, generator=gn, device="cuda")[:n].int()
    pool = 0.5 * torch.randn(n + 2, H, D, D, generator=gn, device="cuda")
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda").int()
    S0 = torch.zeros(n, H, D, D, dtype=torch.float64, device="cuda") if zero_state else pool[slots.long()].double()
    ref_out, ref_S = delta64(q, k, v, g, beta, S0, lens, slots, norm, D ** -0.5)
    dst = pool.clone() if in_place else torch.full_like(pool, 3.25)
    out = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    op(q, k, v, g, beta, out, None if zero_state else (dst if in_place else pool), dst,
       seq_start=start if start_given else None, slots=slots)
    assert k3.k3moe_device_status(op.ws) == (0, 0)
    check_delta(out, dst[slots.long()], ref_out, ref_S, f"{lens}")
    rest = torch.ones(n + 2, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert torch.equal(dst[rest], (pool if in_place else torch.full_like(pool, 3.25))[rest])
    return out, dst


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("lens,H,Hq", [
    ([1], 1, 1), ([1], 56, 56), ([1] * 33, 8, 4), ([2, 1, 5, 0, 3], 6, 2), ([8] * 40, 16, 16),
    ([63], 2, 2), ([64], 2, 1), ([65], 2, 2), ([127, 1, 128, 0, 129], 3, 3), ([200, 17, 64, 300], 4, 2),
    ([1, 1, 1, 700, 1], 2, 2), ([1031], 3, 1)])
def test_delta_rule(k3, lens, H, Hq, channel):
    run_delta(k3, lens, H, Hq, channel, seed=len(lens) + H)


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("lens", [[3, 2], [130, 70]])
@pytest.mark.parametrize("kw", [dict(norm=0), dict(zero_state=True), dict(in_place=True), dict(bias=1.5),
                                dict(decay="none"), dict(decay="strong"), dict(decay="none", bias=3.0)],
                         ids=lambda kw: "-".join(kw))
def test_delta_rule_forms(k3, lens, channel, kw):
    run_delta(k3, lens, 4, 2, channel, seed=7, **kw)


@pytest.mark.parametrize("n", [1, 5])
def test_delta_rule_without_seq_start(k3, n):
    """NULL offsets: one token each, or one sequence."""
    run_delta(k3, [1] * n, 4, 4, True, start_given=False)
    if n == 1:
        run_delta(k3, [90], 2, 2, False, start_given=False)


def test_delta_rule_in_pieces_matches_whole(k3):
    """A prompt in one call, and the same in pieces through the carried state: prompt
    chunks, then single tokens."""
    H, lens = 4, [150]
    q, k, v, g, beta = delta_inputs(lens, H, H, True, 11)
    op = k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=D), 1, 150)
    whole, state = torch.empty(150, H, D, dtype=torch.bfloat16, device="cuda"), op.new_state(1)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    op(q, k, v, g, beta, whole, None, state, slots=one)
    parts, S = torch.empty_like(whole), op.new_state(1)
    for lo, hi in [(0, 64), (64, 70), (70, 147), (147, 148), (148, 149), (149, 150)]:
        op(q[lo:hi], k[lo:hi], v[lo:hi], g[lo:hi], beta[lo:hi], parts[lo:hi], S, S, slots=one)
    ref, ref_S = delta64(q, k, v, g, beta, torch.zeros_like(S).double(), lens, None, 1, D ** -0.5)
    check_delta(whole, state, ref, ref_S, "whole")
    check_delta(parts, S, ref, ref_S, "pieces")


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("lens,H,Hq", [([2500], 25, 5), ([1500, 0, 1101, 333], 19, 19), ([64 * 24], 75, 75)])
def test_delta_rule_in_stretches(k3, lens, H, Hq, channel):
    """Few long sequences: chains and the preparation of what follows go side by side."""
    run_delta(k3, lens, H, Hq, channel, seed=17, in_place=len(lens) == 1)


@pytest.mark.parametrize("channel", [False, True])
def test_delta_rule_stretches_bit_for_bit(k3, channel):
    """However a long sequence is walked, whole chunks at a time, the bits are the same."""
    T, H = 4096, 27
    q, k, v, g, beta = delta_inputs([T], H, H, channel, 23)
    op = k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=D if channel else 1), 1, T)
    got = []
    for cuts in ([0, T], [0, 64, 1024, 1216, T], [0, T]):
        out, state = torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda"), op.new_state(1)
        for t0, t1 in zip(cuts, cuts[1:]):
            op(q[t0:t1], k[t0:t1], v[t0:t1], g[t0:t1], beta[t0:t1], out[t0:t1], state, state,
               seq_start=torch.tensor([0, t1 - t0], dtype=torch.int32, device="cuda"))
        assert k3.k3moe_device_status(op.ws) == (0, 0)
        got.append((out, state))
    for out, state in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(state, got[0][1])


def test_delta_rule_repeats_bit_for_bit(k3):
    for lens in ([1] * 20, [300, 77, 1]):
        a = run_delta(k3, lens, 4, 2, True, seed=3)
        b = run_delta(k3, lens, 4, 2, True, seed=3)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens", [[1, 1, 1], [100, 80, 90]])
def test_delta_rule_reports_bad_sequences(k3, lens):
    """A slot or offset pair outside its range sets the status bit and skips that sequence;
    the others are computed."""
    H, n, T = 2, 3, sum(lens)
    q, k, v, g, beta = delta_inputs(lens, H, H, False, 5)
    op = k3.DeltaRule(k3.k3moe_delta_config(H, H), n, T)
    pool = 0.5 * torch.randn(4, H, D, D, device="cuda")
    t0 = np.concatenate([[0], np.cumsum(lens)])
    ref_out, ref_S = delta64(q, k, v, g, beta, pool[:3].double(), lens, None, 1, D ** -0.5)

    def go(start, slots):
        dst, out = torch.zeros_like(pool), torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
        op(q, k, v, g, beta, out, pool, dst, seq_start=torch.tensor(start, device="cuda").int(),
           slots=torch.tensor(slots, device="cuda").int())
        return (*k3.k3moe_device_status(op.ws), out, dst)

    for bad in (-1, 4, 1 << 30):
        rc, code, out, dst = go(t0, [0, bad, 2])
        assert rc == 6 and code == k3.DEV_BAD_INDEX
        assert (dst[1] == 0).all() and (out[t0[1]:t0[2]] == 0).all()
        for i in (0, 2):
            check_delta(out[t0[i]:t0[i + 1]], dst[i:i + 1], ref_out[t0[i]:t0[i + 1]], ref_S[i:i + 1])
    rc, code, out, dst = go([0, lens[0], T + 1, T], [0, 1, 2])         # the second ends past T
    assert rc == 6 and code == k3.DEV_BAD_OFFSETS
    check_delta(out[:lens[0]], dst[:1], ref_out[:lens[0]], ref_S[:1])
    assert (dst[1:] == 0).all()
    rc, code, out, dst = go([0, lens[0], -5, T], [0, 1, 2])
    assert rc == 6 and code == k3.DEV_BAD_OFFSETS and (dst[1:] == 0).all()
    assert go(t0, [0, 1, 2])[:2] == (0, 0)


def test_delta_rule_keeps_sequences_apart(k3):
    """NaN in one sequence's tokens or state stays in that sequence (a chunk's padding reads
    the neighbour's tokens, which take no part)."""
    for lens in ([2, 3, 1], [70, 65, 90]):
        H = 2
        q, k, v, g, beta = delta_inputs(lens, H, H, True, 9)
        q, k, v = q.clone(), k.clone(), v.clone()
        t0 = np.concatenate([[0], np.cumsum(lens)])
        for t in (q, k, v, g, beta):
            t[t0[1]:t0[2]] = float("nan")
        op = k3.DeltaRule(k3.k3moe_delta_config(H, H, gate_dim=D), 3, sum(lens))
        pool = 0.5 * torch.randn(3, H, D, D, device="cuda")
        dst, out = torch.zeros_like(pool), torch.zeros(sum(lens), H, D, dtype=torch.bfloat16, device="cuda")
        op(q, k, v, g, beta, out, pool, dst, seq_start=torch.tensor(t0, device="cuda").int())
        assert k3.k3moe_device_status(op.ws) == (0, 0)
        for i in (0, 2):
            sl = slice(t0[i], t0[i + 1])
            ro, rs = delta64(q[sl], k[sl], v[sl], g[sl], beta[sl], pool[i:i + 1].double(), [lens[i]], None, 1, D ** -0.5)
            check_delta(out[sl], dst[i:i + 1], ro, rs)
        assert torch.isnan(out[t0[1]:t0[2]]).all() and torch.isnan(dst[1]).any()
