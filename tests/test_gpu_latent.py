"""The latent attention's operators on the GPU against their definitions in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, a float rounding; a bf16 result is off by 2^-8 of
itself at most):
  norm: the mean of squares is a sum of positive terms, at most 64 roundings deep (a thread's 32,
    its warp's 5, up to 16 warps, the division), halved by the root; root, division and the products up to total
    add at most 12, the sigmoid (expf 2, sum, division) 5: y is within 50 u of itself, and total by 50 u |y| + u |total|.
    With bf16 sums the sigmoid's exponent t = z log2 e is rounded once, to |t| u, which moves 2^t by |t| ln 2 u = |z| u of itself;
    constant 1, 2^t 4, sum 1, reciprocal 2: 3 + |z| more than the 5 above.
    out adds as much again from its own norm and what total's error makes of it.
  head projection: a float sum of K products; a tensor core may truncate: at most 2^-23 of the running
    sum an addition, with signs that vary: 4 sqrt(K) 2^-23 of sum |w x| (four standard deviations of a random
    walk whose every step is the worst one).
  write: as norm for c; a rotated column has two products of a cosine or sine off by 2^-21 at most (an
    angle off by 2^-24 of a turn is 2^-21.3 radians).
  attention: a score is a float sum as above, off by d = 4 sqrt(columns) 2^-23 scale sum |q k|, and the
    exponent of a weight by 2^-21 more for each unit of the score; the weights exp(s - m) are off by e^(2d) - 1 <= 3d and rounded to
    bf16, so out is off by (2^-8 + 3d + 4 sqrt(keys) 2^-23) sum p |v|, lse by d + 2^-20 (1 + |lse|).
"""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
C, R, K, V = 512, 64, 128, 128
ROW = C + R
U, BF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def k3():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_expert_k3moe_gb300 import build as kbuild
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    return k3


def randn(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def within(got, ref, tol, what=""):
    if got.dtype == torch.bfloat16:
        tol = tol + BF * (ref.abs() + tol)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got.double() - ref).abs() / (tol + 1e-30)
    assert (off <= 1).all(), f"{what}: {int((off > 1).sum())} of {off.numel()} outside, worst {off.max():.2f}"


# ----------------------------------------------------------------------------- norm

NORM = [  # T, N, group, gate, x f32, sum f32, residual, scale, post, pre, pad
    (1, 7168, 0, "none", False, False, True, True, True, True, 0),
    (1, 8, 0, "none", False, True, False, False, True, False, 0),
    (3, 8, 0, "silu", True, False, True, True, True, True, 8),
    (5, 128, 128, "sigmoid", False, False, False, False, True, False, 0),
    (7, 64, 64, "silu", False, False, True, False, True, True, 16),
    (33, 1024, 256, "silu", False, True, True, True, True, True, 0),
    (130, 7168, 128, "sigmoid", False, False, False, False, True, False, 0),
    (9, 2048, 0, "none", True, True, True, False, True, True, 24),
    (11, 2056, 0, "sigmoid", False, False, True, True, True, True, 0),
    (6, 4096, 64, "none", False, False, True, True, True, True, 0),
    (4, 4104, 0, "silu", True, True, True, True, True, True, 8),
    (3, 16384, 0, "silu", True, True, True, True, True, True, 0),
    (2, 16384, 256, "sigmoid", False, False, True, True, True, True, 0),
    (257, 264, 0, "none", False, False, True, True, False, True, 0),
    (19, 520, 0, "silu", False, True, True, True, False, False, 0),
    (1000, 24, 0, "none", False, False, False, False, True, True, 0),
    (1300, 7168, 128, "sigmoid", False, False, False, False, True, False, 0),     # many long rows: a block takes several
    (901, 7168, 0, "none", False, False, True, True, True, True, 8),
    (700, 4104, 0, "silu", True, True, True, True, True, True, 16),
    (650, 8192, 256, "silu", True, True, True, False, True, True, 0),
    (1111, 2056, 0, "sigmoid", False, True, False, True, True, True, 0),
    (620, 5120, 64, "none", True, False, True, False, True, False, 8),
    (777, 6000, 0, "sigmoid", False, False, True, True, False, True, 0),
    (640, 2568, 0, "sigmoid", True, True, True, True, True, True, 8),
    (1400, 4104, 0, "silu", True, True, True, True, True, True, 16),              # and several of the shorter ones on an SM
    (1900, 2568, 0, "sigmoid", True, True, True, True, True, True, 8),
    (2500, 2056, 0, "sigmoid", False, True, False, True, True, True, 0),
    (2500, 2048, 64, "silu", False, False, False, False, True, False, 24),
    (5600, 1024, 256, "none", True, False, True, True, True, True, 0),
    (7400, 520, 0, "silu", False, False, True, False, False, True, 0),
]


def norm64(x, gate, act, post, group, alpha, scale, residual, pre, eps):
    """(total, y alone, out) in 64 bits."""
    y = x.double()
    if post is not None:
        z = y.unflatten(-1, (-1, group))
        y = (z / (z.pow(2).mean(-1, keepdim=True) + eps).sqrt() * post.double()).flatten(-2)
    if gate is not None:
        z = gate.double()
        y = y * torch.special.expit(z) * (z if act == "silu" else 1.0)
    y = alpha * y * (scale.double() if scale is not None else 1.0)
    total = y + (residual.double() if residual is not None else 0.0)
    r = (total.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    return total, y, (total * r * pre.double() if pre is not None else None), r


def check_norm(total, out, ref, pre, gate=None):
    want, y, want_out, r = ref
    tol = 50 * U * y.abs() + U * want.abs()
    if gate is not None and total is not None and total.dtype == torch.bfloat16:
        tol = tol + (3 + gate.double().abs()) * U * y.abs()
    if total is not None:
        within(total, want, tol, "total")
    if out is not None:
        # a total off by e moves the mean of squares by 2 total e: as much again of the root mean square
        rms = (tol * tol).mean(-1, keepdim=True).sqrt()
        within(out, want_out, (tol * r + (rms * r + 50 * U) * want.abs() * r) * pre.double().abs(), "out")


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(str(v) for v in c))
def test_norm(k3, case):
    T, N, group, gate, xf, sf, has_res, has_scale, post, pre, pad = case
    r, alpha, eps = randn(T + N), -0.75, 1e-5
    xt, st = (torch.float32 if f else torch.bfloat16 for f in (xf, sf))
    x = (3 * r(T, N + pad)).to(xt)[:, :N]
    g = (4 * r(T, N + pad)).bfloat16()[:, :N] if gate != "none" else None
    res = (2 * r(T, N + 2 * pad)).to(st)[:, :N] if has_res else None
    op = k3.Norm(k3.k3moe_norm_config(N, group, post, pre, gate, xf, sf, eps, alpha))
    op.post_gain, op.scale, op.pre_gain = r(group or N) if post else None, r(N) if has_scale else None, r(N) if pre else None
    wide = torch.full((T, N + pad), 7.5, dtype=st, device="cuda")
    wide_out = torch.full((T, N + pad), 7.5, dtype=torch.bfloat16, device="cuda")
    total, out = wide[:, :N], wide_out[:, :N] if pre else None
    op(x, out=out, gate=g, residual=res, total=total)
    ref = norm64(x, g, gate, op.post_gain, group or N, alpha, op.scale, res, op.pre_gain, eps)
    check_norm(total, out, ref, op.pre_gain, g)
    assert (wide[:, N:] == 7.5).all() and (wide_out[:, N:] == 7.5).all()
    if pre:                                                # the sum need not be written
        alone = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        op(x, out=alone, gate=g, residual=res)
        assert torch.equal(alone, out)
    if has_res:                                            # the residual in place
        again = res.clone()
        op(x, out=out, gate=g, residual=again, total=again)
        assert torch.equal(again, total)


def test_norm_edges(k3):
    """Zero rows, rows that no square survives, and a NaN that stays in its row; T = 0."""
    N = 1024
    op = k3.Norm(k3.k3moe_norm_config(N, eps=1e-6))
    op.post_gain, op.pre_gain = torch.ones(N, device="cuda"), torch.ones(N, device="cuda")
    x = randn(1)(5, N).bfloat16()
    x[1] = 0
    x[3, 17] = float("nan")
    res, out = torch.zeros_like(x), torch.empty_like(x)
    total = torch.empty_like(x)
    op(x, out=out, residual=res, total=total)
    assert (total[1] == 0).all() and (out[1] == 0).all()
    assert torch.isnan(total[3]).all() and torch.isnan(out[3]).all()
    keep = [0, 2, 4]
    check_norm(total[keep], out[keep], norm64(x[keep], None, "none", op.post_gain, N, 1.0, None, None, op.pre_gain, 1e-6), op.pre_gain)
    op(x[:0], out=out[:0])
    gated = k3.Norm(k3.k3moe_norm_config(N, post_norm=0, pre_norm=0, gate="silu"))
    gate = torch.full_like(x, -200.0)                      # its exponential overflows; the gate is zero
    x[3] = 1
    assert (gated(x, gate=gate, total=total) == 0).all()
    assert torch.equal(gated(x, gate=-gate, total=total), (x.float() * 200).bfloat16())


def test_norm_in_place(k3):
    """total and out over x, the gate and the residual, where type and stride are the same."""
    T, N = 37, 2064
    r = randn(5)
    op = k3.Norm(k3.k3moe_norm_config(N, gate="silu"))
    op.post_gain, op.scale, op.pre_gain = r(N), r(N), r(N)
    x, gate, res = (r(T, N).bfloat16() for _ in range(3))
    total, out = torch.empty_like(x), torch.empty_like(x)
    op(x, out=out, gate=gate, residual=res, total=total)
    for names in (("x", "gate"), ("gate", "x"), ("residual", "x"), ("x", "residual")):
        given = dict(x=x.clone(), gate=gate.clone(), residual=res.clone())
        op(**given, total=given[names[0]], out=given[names[1]])
        assert torch.equal(given[names[0]], total) and torch.equal(given[names[1]], out), names


@pytest.mark.parametrize("T", [1, 3])
def test_forward_reads_what_a_norm_wrote(k3, T):
    """The experts' mat-vec path reads its tokens ahead of its wait for the routing; not those a norm may still be
    writing.  The buffer is poisoned before the norm that writes it."""
    d, E, f = 1024, 64, 256
    g = torch.Generator("cuda").manual_seed(T)
    m = k3.MoELayer(k3.k3moe_config(d=d, f=f, n_experts=E, top_k=4, n_shared=1), T)
    codes = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")  # noqa: E731
    scale = lambda *s: torch.full(s, 121, dtype=torch.uint8, device="cuda")  # noqa: E731
    w = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).bfloat16()  # noqa: E731
    m.pack_experts(0, E, codes(E, f, d // 2), scale(E, f, d // 32), codes(E, f, d // 2), scale(E, f, d // 32), codes(E, d, f // 2), scale(E, d, f // 32))
    m.w_router, m.sh_w1, m.sh_w3, m.sh_w2 = w(E, d), w(1, f, d), w(1, f, d), w(1, d, f)
    op = k3.Norm(k3.k3moe_norm_config(d, post_norm=0))
    op.pre_gain = torch.ones(d, device="cuda")
    h, x, out = torch.randn(T, d, device="cuda").bfloat16(), torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d, device="cuda")
    op(h, out=x)
    m.route(x)
    torch.cuda.synchronize()
    m.forward(x, out)
    torch.cuda.synchronize()
    want = out.clone()
    for _ in range(50):
        x.fill_(float("nan"))
        op(h, out=x)
        m.forward(x, out)
        assert torch.equal(out, want)


# ----------------------------------------------------------------------------- a head's own projection

@pytest.mark.parametrize("T,H,K_,N,pad", [(1, 56, 128, 512, 0), (1, 1, 8, 1, 0), (2, 3, 64, 129, 8), (16, 5, 200, 128, 0), (17, 2, 512, 130, 64),
                                          (64, 4, 136, 72, 8), (65, 3, 512, 128, 0), (333, 7, 512, 128, 64), (130, 1, 72, 8192, 0)])
def test_head_linear(k3, T, H, K_, N, pad):
    r = randn(T + K_)
    x = r(T, H, K_ + pad).bfloat16()[..., :K_]
    w = (r(H, N, K_) / K_ ** 0.5).bfloat16()
    op = k3.HeadLinear(k3.k3moe_head_linear_config(H, N, K_), T)
    op.w = w
    wide = torch.full((T, H, N + pad), 7.5, dtype=torch.bfloat16, device="cuda")
    y = op(x, wide[..., :N])
    ref = torch.einsum("thk,hnk->thn", x.double(), w.double())
    mag = torch.einsum("thk,hnk->thn", x.double().abs(), w.double().abs())
    within(y, ref, 4 * K_ ** 0.5 * 2.0 ** -23 * mag)
    assert (wide[..., N:] == 7.5).all()
    assert torch.equal(op(x, torch.empty_like(y)), y)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- the cache's write

def rotate64(x, positions, freq, how):
    x = x.double()
    if how == "none":
        return x
    a = positions.double()[:, None] * freq
    a = a[:, None] if x.dim() == 3 else a
    if how == "pairs":
        u, v = x[..., 0::2], x[..., 1::2]
    else:
        u, v = x[..., :R // 2], x[..., R // 2:]
    p, q = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    return torch.stack([p, q], -1).flatten(-2) if how == "pairs" else torch.cat([p, q], -1)


def rope_tol(x, how):
    """2^-21 of the two columns that a rotated one is made of, and three roundings of them."""
    a = x.double().abs()
    s = (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1) if how == "pairs" else (a[..., :R // 2] + a[..., R // 2:]).repeat(*[1] * (x.dim() - 1), 2)
    return (2.0 ** -21 + 3 * U) * s


@pytest.mark.parametrize("how,norm,page", [("pairs", 1, 64), ("halves", 1, 16), ("none", 1, 256), ("pairs", 0, 32), ("halves", 0, 128)])
@pytest.mark.parametrize("T", [1, 7, 130])
def test_write(k3, T, how, norm, page):
    H = 5
    r = randn(T + page)
    op = k3.LatentAttention(k3.k3moe_latent_config(H, page_size=page, rope=how, norm=norm, norm_eps=1e-5), 0, T)
    op.gain = r(C) if norm else None
    op.inv_freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    wide = r(T, ROW + 24).bfloat16()
    c, q = wide[:, 8:8 + ROW], r(T, H, K + R).bfloat16()
    g = torch.Generator().manual_seed(T)
    positions = torch.randint(0, 1 << 20, (T,), generator=g).int().cuda()
    positions[0] = 0 if T > 1 else 1048575
    n_pages = -(-T // page) + 2
    slots = torch.randperm(n_pages * page, generator=g)[:T].cuda()
    if T > 5:
        slots[3] = -1
    cache = op.new_cache(n_pages) + 7.5
    rows, q_rope = torch.full((T, ROW + 8), 7.5, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, R, dtype=torch.bfloat16, device="cuda")
    op.write(c, positions, cache=cache, slots=slots, rows=rows[:, :ROW], q=q[..., K:], q_rope=q_rope)
    x = c[:, :C].double()
    want = x / (x.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * op.gain.double() if norm else x
    within(rows[:, :C], want, 50 * U * want.abs() if norm else 0 * want, "c")
    within(rows[:, C:ROW], rotate64(c[:, C:], positions, op.inv_freq, how), rope_tol(c[:, C:], how) if how != "none" else 0 * x[:, :R], "r")
    within(q_rope, rotate64(q[..., K:], positions, op.inv_freq, how), rope_tol(q[..., K:], how) if how != "none" else 0.0, "q")
    flat, written = cache.view(-1, ROW), torch.zeros(n_pages * page, dtype=torch.bool, device="cuda")
    for t in range(T):
        if slots[t] >= 0:
            assert torch.equal(flat[slots[t]], rows[t, :ROW])
            written[slots[t]] = True
    assert (flat[~written] == 7.5).all() and (rows[:, ROW:] == 7.5).all()
    beside, kept_q = wide[:, :8].clone(), q.clone()        # in place
    op.write(c, positions, rows=c, q=q[..., K:], q_rope=q[..., K:])
    assert torch.equal(c, rows[:, :ROW]) and torch.equal(q[..., K:], q_rope) and torch.equal(q[..., :K], kept_q[..., :K])
    assert torch.equal(wide[:, :8], beside)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_write_far_positions_and_bad_slots(k3):
    T, page = 4, 16
    op = k3.LatentAttention(k3.k3moe_latent_config(1, page_size=page, rope="halves", norm=0), 0, T)
    op.inv_freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    c = randn(3)(T, ROW).bfloat16()
    positions = torch.tensor([2 ** 31 - 1, -5, 2 ** 30 + 1, 12345678], dtype=torch.int32, device="cuda")
    cache = op.new_cache(2)
    slots = torch.tensor([32, 31, 1 << 40, -(1 << 40)], device="cuda")
    rows = torch.empty_like(c)
    op.write(c, positions, cache=cache, slots=slots, rows=rows)
    # 64-bit angles of 2^31 are off by 2^-22 themselves
    within(rows[:, C:], rotate64(c[:, C:], positions, op.inv_freq, "halves"), 2 * rope_tol(c[:, C:], "halves"), "r")
    assert torch.equal(cache.view(-1, ROW)[31], rows[1]) and not cache.view(-1, ROW)[:31].any()
    assert k3.k3moe_device_status(op.ws) == (6, 0x1)        # slots 32 and 2^40 are past the cache
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- attention

def attention64(q, k, v, scale, causal):
    """(out, lse, tolerance of out, of lse) of q [n][H][c], k [m][H or 1][c], v [m][H or 1][d]."""
    n, m, H = q.shape[0], k.shape[0], q.shape[1]
    q, k, v = q.double(), k.double().expand(-1, H, -1), v.double().expand(-1, H, -1)
    z = torch.einsum("qhc,khc->hqk", q, k) * scale
    d = 4 * q.shape[2] ** 0.5 * 2.0 ** -23 * scale * torch.einsum("qhc,khc->hqk", q.abs(), k.abs()) + 2.0 ** -21 * z.abs()
    sees = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        sees = torch.arange(m, device=q.device)[None] <= torch.arange(n, device=q.device)[:, None] + m - n
    z = torch.where(sees, z, -float("inf"))
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None]).nan_to_num(0.0)
    d = torch.where(sees, d, 0.0).amax(-1) if m else torch.zeros_like(lse)
    out = torch.einsum("hqk,khd->qhd", p, v)
    tol = (BF + 3 * d + 4 * max(m, 1) ** 0.5 * 2.0 ** -23).t()[..., None] * torch.einsum("hqk,khd->qhd", p, v.abs())
    return out, lse.t(), tol, (d + 2.0 ** -20 * (1 + lse.abs())).t()


def check_attention(out, lse, ref, what):
    want, want_lse, tol, tol_lse = ref
    within(out, want, tol, f"{what} out")
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isneginf(lse), empty), f"{what}: rows without a key"
    assert (out[empty] == 0).all()
    within(lse[~empty], want_lse[~empty], tol_lse[~empty], f"{what} lse")


class Cached:
    """Sequences' rows in shuffled pages; what no sequence owns is NaN."""

    def __init__(self, queries, lens, H, page, seed, pad=0, spoil=float("nan"), q_scale=1.0):
        r = randn(seed)
        g = torch.Generator().manual_seed(seed)
        need = [-(-x // page) for x in lens]
        self.n_pages = sum(need) + 3
        order = torch.randperm(self.n_pages, generator=g).int()
        self.cache = torch.full((self.n_pages, page, ROW), spoil, dtype=torch.bfloat16, device="cuda")
        self.pages = torch.full((len(lens), max(need + [1]) + 1), 1 << 30, dtype=torch.int32)
        self.rows, at = [], 0
        for i, (m, x) in enumerate(zip(need, lens)):
            mine = order[at:at + m]
            self.pages[i, :m] = mine
            at += m
            rows = r(x, ROW).bfloat16()
            self.rows.append(rows)
            j = torch.arange(x)
            self.cache[mine.long()[j // page].cuda(), (j % page).cuda()] = rows
        self.pages = self.pages.cuda()
        T = sum(queries)
        self.q = (q_scale * r(T, H, ROW + pad)).bfloat16()[..., :ROW]
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.start = torch.tensor([0, *itertools.accumulate(queries)], dtype=torch.int32, device="cuda")
        self.queries, self.lens, self.H, self.page, self.T = queries, lens, H, page, T
        self.out = torch.full((T, H, C), 7.5, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, H), 7.5, device="cuda")

    def holder(self, k3, **kw):
        cfg = k3.k3moe_latent_config(self.H, page_size=self.page, **kw)
        return k3.LatentAttention(cfg, len(self.lens), self.T), cfg

    def __call__(self, op, **kw):
        return op.attend(self.q, self.cache, self.pages, self.kv_len, self.out, **{"seq_start": self.start, "lse": self.lse, **kw})

    def check(self, cfg, skip=()):
        t = 0
        for i, n in enumerate(self.queries):
            s = slice(t, t + n)
            t += n
            if n == 0 or i in skip:
                continue
            k = self.rows[i][:, None]
            check_attention(self.out[s], self.lse[s], attention64(self.q[s], k, k[..., :C], cfg.scale, cfg.causal), f"sequence {i}")


ATTEND = [  # queries, kv lengths, heads, page, causal, pad
    ([1], [1], 1, 16, 1, 0),
    ([1], [0], 8, 16, 1, 0),
    ([1], [777], 56, 64, 1, 0),
    ([1, 1, 1], [64, 128, 127], 16, 64, 1, 8),
    ([1, 1, 1, 1], [129, 0, 1, 255], 3, 32, 1, 0),
    ([1, 0, 3, 2], [300, 10, 5, 1], 13, 16, 1, 0),              # drafts, one with more queries than rows
    ([4, 1, 7], [1000, 333, 260], 28, 128, 1, 64),
    ([5, 2], [513, 6], 64, 256, 0, 0),
    ([1, 2], [200, 900], 128, 64, 1, 0),
    ([1], [9001], 65, 16, 1, 0),
    ([33], [140], 8, 64, 1, 0),
    ([70, 3], [70, 129], 5, 32, 1, 0),
    ([1] * 40, [(37 * i) % 513 for i in range(40)], 8, 64, 1, 0),
    ([2], [40000], 16, 64, 1, 0),
    ([1] * 3, [20000, 5, 7000], 200, 64, 1, 0),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{sum(c[0])}x{c[2]}-{max(c[1])}-{c[3]}")
def test_attend(k3, case):
    queries, lens, H, page, causal, pad = case
    c = Cached(queries, lens, H, page, sum(lens) + H, pad)
    op, cfg = c.holder(k3, causal=causal)
    c(op)
    c.check(cfg)
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(2):                                     # and again, bit for bit
        c(op)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    if max(queries) == 1:                                  # without offsets, without lse
        c(op, seq_start=None, lse=None)
        assert torch.equal(c.out, out)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("q_scale", [0.0, 8.0])
def test_attend_flat_and_sharp(k3, q_scale):
    """Equal weights of all rows; and scores of tens to hundreds, so that the running maximum moves."""
    c = Cached([1, 2], [3000, 1100], 16, 64, 7, q_scale=q_scale)
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)


def test_attend_growing_scores(k3):
    """Every later row outdoes all before it: each tile rescales what was summed."""
    c = Cached([1], [2000], 8, 64, 9)
    c.q[:] = 0
    c.q[..., 0] = 64
    ramp = torch.arange(2000, device="cuda") * 0.25
    c.rows[0][:, 0] = ramp.bfloat16()
    at = torch.arange(2000, device="cuda")
    c.cache[c.pages[0].long()[at // 64], at % 64] = c.rows[0]
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)
    c.rows[0][:, 0] = -ramp.bfloat16()                     # and the first one does
    c.cache[c.pages[0].long()[at // 64], at % 64] = c.rows[0]
    c(op)
    c.check(cfg)


def test_attend_reports_what_does_not_fit(k3):
    c = Cached([1, 1, 1, 1], [100, 100, 200, 100], 8, 64, 11)
    op, cfg = c.holder(k3)
    good = c.pages.clone()
    for bad in (-1, c.n_pages, 1 << 30, -(1 << 31)):
        c.pages[2, 1] = bad
        c(op)
        rows = c.rows[2].clone()
        c.rows[2][64:128] = 0                               # the page reads as zeros
        c.check(cfg)
        c.rows[2] = rows
        assert k3.k3moe_device_status(op.ws) == (6, 0x1)
    c.pages.copy_(good)
    for name, at, bad in (("kv_len", 1, -1), ("kv_len", 1, 64 * c.pages.shape[1] + 1), ("start", 2, 0), ("start", 2, 5)):
        t = getattr(c, name)
        kept = t.clone()
        t[at] = bad
        c.out[:], c.lse[:] = 7.5, 7.5
        c(op)
        lost = {"kv_len": [1], "start": [1] if bad == 0 else [1, 2]}[name]
        if name == "start" and bad == 0:                    # then the third begins at the first token: only what is plain is compared
            c.check(cfg, skip=[0, 1, 2])
        else:
            c.check(cfg, skip=lost)
            assert (c.out[1] == 7.5).all() and (c.lse[1] == 7.5).all()
        assert k3.k3moe_device_status(op.ws) == (6, 0x2)
        t.copy_(kept)
    c(op)
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attend_what_is_not_seen_does_not_matter(k3, value):
    """Rows behind the last, and the later rows of a draft, whatever they hold."""
    c = Cached([3, 1], [150, 70], 8, 64, 13, spoil=value)
    op, cfg = c.holder(k3)
    at = 149                                               # the draft's last row: seen by its last query alone
    c.cache[c.pages[0, at // 64].long(), at % 64] = value
    c(op)
    c.rows[0][at] = 0
    k = c.rows[0][:149, None]
    for j in range(2):
        ref = attention64(c.q[j:j + 1], k[:148 + j], k[:148 + j, :, :C], cfg.scale, 0)
        check_attention(c.out[j:j + 1], c.lse[j:j + 1], ref, f"query {j}")
    assert torch.isnan(c.out[2]).any(-1).all()
    k = c.rows[1][:, None]
    check_attention(c.out[3:4], c.lse[3:4], attention64(c.q[3:4], k, k[..., :C], cfg.scale, 1), "the other")


def test_attend_captured(k3):
    """A captured call replays on new lengths, pages and queries."""
    c = Cached([1, 1, 1], [500, 64, 3], 16, 64, 17)
    op, cfg = c.holder(k3)
    graph = k3._capture(lambda x, out: c(op), c.q, c.out)
    for lens in ([10, 500, 65], [513, 2, 1]):
        d = Cached([1, 1, 1], lens, 16, 64, sum(lens))
        c.pages[:] = -1
        n = min(c.n_pages, d.n_pages)
        w = min(c.pages.shape[1], d.pages.shape[1])
        if d.n_pages > c.n_pages:
            continue
        c.cache[:n].copy_(d.cache[:n])
        c.pages[:, :w].copy_(d.pages[:, :w])
        c.q.copy_(d.q)
        c.kv_len.copy_(d.kv_len)
        graph.replay()
        c.rows = d.rows
        c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_attend_on_a_side_stream(k3):
    c = Cached([1] * 5, [100, 2000, 30, 700, 1], 16, 64, 19)
    op, cfg = c.holder(k3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c(op, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.check(cfg)


@pytest.mark.parametrize("queries,lens", [([1, 1, 1], [64, 20000, 900]), ([2, 3], [500, 700])])
def test_attend_nan_queries(k3, queries, lens):
    """A NaN in a query is all of its outputs, however many parts its rows are cut into, and nothing of another's."""
    c = Cached(queries, lens, 16, 64, 43)
    op, cfg = c.holder(k3)
    c(op)
    out, lse = c.out.clone(), c.lse.clone()
    bad = torch.zeros(c.T, 16, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[-1, 15] = bad[0, 0] = True
    c.q[bad] = float("nan")
    c(op)
    assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
    assert torch.equal(c.out[~bad], out[~bad]) and torch.equal(c.lse[~bad], lse[~bad])


@pytest.mark.parametrize("n_seq", [128, 129, 200, 500])
def test_attend_many_sequences(k3, n_seq):
    """Empty ones, drafts, ones without rows, in more than a warp and more than a block looks over at once."""
    queries = [(0, 1, 1, 2, 1, 5)[i % 6] for i in range(n_seq)]
    lens = [(41 * i) % 300 if i % 7 else 0 for i in range(n_seq)]
    c = Cached(queries, lens, 16, 64, n_seq)
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)
    c.start[n_seq // 2 + 1] = -3                           # two that do not fit leave the others' to do, cut in other places
    c.out[:] = 7.5
    c(op)
    a, b = sum(queries[:n_seq // 2]), sum(queries[:n_seq // 2 + 2])
    assert (c.out[a:b] == 7.5).all()
    c.check(cfg, skip=[n_seq // 2, n_seq // 2 + 1])
    assert k3.k3moe_device_status(op.ws) == (6, 0x2)


@pytest.mark.parametrize("n_seq,tables", [(40, 50000), (200, 10000)])
def test_attend_wide_tables(k3, n_seq, tables):
    """Tables so wide that the tiles of all sequences would not be counted in 32 bits, were they full."""
    queries = [8] * n_seq
    c = Cached(queries, [(77 * i) % 700 for i in range(n_seq)], 64, 256, n_seq + 1)
    assert n_seq * sum(queries) * c.H / 64 * tables * 4 > 2 ** 31
    wide = torch.full((n_seq, tables), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :c.pages.shape[1]] = c.pages
    c.pages = wide
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_write_and_attend_far_rows(k3):
    """A cache whose last rows are past 2^32 bytes and 2^31 elements: written, read, and a spoiled one added."""
    H, n_pages = 8, 70000
    cfg = k3.k3moe_latent_config(H, page_size=64, rope="none", norm=0)
    op = k3.LatentAttention(cfg, 2, 130)
    cache = torch.empty(n_pages, 64, ROW, dtype=torch.bfloat16, device="cuda")
    r = randn(51)
    rows, q = r(130, ROW).bfloat16(), r(2, H, ROW).bfloat16()
    pages = torch.tensor([[n_pages - 1, 3, n_pages - 2], [n_pages - 3, 0, 0]], dtype=torch.int32, device="cuda")
    at = torch.arange(130, device="cuda")
    slots = pages[0].long()[at // 64] * 64 + at % 64
    op.write(rows, cache=cache, slots=slots)
    op.write(rows[:5].contiguous(), cache=cache, slots=(n_pages - 3) * 64 + at[:5])
    assert torch.equal(cache[n_pages - 1], rows[:64]) and torch.equal(cache[n_pages - 2, :2], rows[128:])
    out, lse = torch.empty(2, H, C, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, device="cuda")
    op.attend(q, cache, pages, torch.tensor([130, 5], dtype=torch.int32, device="cuda"), out, lse=lse)
    for i, n in enumerate((130, 5)):
        k = rows[:n, None]
        check_attention(out[i:i + 1], lse[i:i + 1], attention64(q[i:i + 1], k, k[..., :C], cfg.scale, 1), f"sequence {i}")
    cache[n_pages - 2, 1, 7] = float("inf")                # the last row of one sequence that two queries share: the second sees it
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    op.attend(q, cache, pages[:1], torch.tensor([130], dtype=torch.int32, device="cuda"), out, seq_start=start, lse=lse)
    k = rows[:129, None]
    check_attention(out[:1], lse[:1], attention64(q[:1], k, k[..., :C], cfg.scale, 1), "before it")
    assert not torch.isfinite(out[1, :, 7]).any()
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_attend_twice_at_once(k3):
    """Two holders on two streams, beside each other; and two captured graphs of one holder, in turn."""
    c, d = Cached([1] * 4, [3000, 500, 0, 77], 56, 64, 31), Cached([3, 1], [900, 4000], 16, 64, 32)
    (op, cfg), (op2, cfg2) = c.holder(k3), d.holder(k3)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        c(op, stream=streams[0])
        d(op2, stream=streams[1])
    torch.cuda.synchronize()
    c.check(cfg)
    d.check(cfg2)
    e = Cached([2] * 2, [1500, 33], 56, 64, 33)
    graphs = k3._capture(lambda x, out: c(op), c.q, c.out), k3._capture(lambda x, out: e(op), e.q, e.out)
    for g in graphs + graphs:
        g.replay()
    c.check(cfg)
    e.check(cfg)


PROMPT = [  # queries, keys (None: the queries' own), heads, causal, padded strides
    ([1], None, 1, 1, False),
    ([2], [5], 3, 1, True),
    ([127, 128, 129], None, 4, 1, False),
    ([64, 0, 1, 300], [64, 10, 700, 290], 3, 1, True),          # a prefix, an empty sequence, more queries than keys
    ([255, 257], [255, 257], 2, 0, False),
    ([256], [1000], 5, 1, False),
    ([5, 3], [0, 2], 2, 1, False),                              # rows that see nothing
    ([7, 9], [0, 300], 2, 0, True),
    ([1000], None, 2, 1, True),
    ([513, 1030], None, 1, 1, False),
    ([1] * 9, [1, 2, 64, 127, 128, 129, 511, 512, 513], 8, 1, False),
    ([3000], None, 1, 1, False),
    ([17], [5000], 2, 1, False),                                # few queries, many keys: parts of the keys
    ([200, 3], [6000, 0], 3, 1, True),
    ([1, 130], [4097, 4000], 1, 0, False),
    ([5, 40, 0, 7], [5, 3000, 100, 8], 1, 1, False),            # one long among short ones: parts that have no keys
    ([260], [2600], 5, 1, False),
]


class Expanded:
    def __init__(self, queries, keys, H, padded, seed, q_scale=1.0):
        r = randn(seed)
        self.queries, self.keys = queries, keys or queries
        T, S = sum(queries), sum(self.keys)
        pad = 8 if padded else 0
        self.q = (q_scale * r(T, H, K + R + 2 * pad)).bfloat16()[..., :K + R]
        self.kv = r(S, H, K + V + pad).bfloat16()[..., :K + V]
        self.rope = r(S, R + 3 * pad).bfloat16()[:, :R]
        starts = lambda x: torch.tensor([0, *itertools.accumulate(x)], dtype=torch.int32, device="cuda")  # noqa: E731
        self.start, self.kv_start = starts(queries), starts(self.keys) if keys else None
        self.out = torch.full((T, H, V), 7.5, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, H), 7.5, device="cuda")
        self.H, self.T = H, T

    def holder(self, k3, **kw):
        cfg = k3.k3moe_latent_config(self.H, **kw)
        return k3.LatentAttention(cfg, len(self.queries), self.T), cfg

    def __call__(self, op, **kw):
        return op.prompt(self.q, self.kv, self.rope, self.out, **{"seq_start": self.start, "kv_start": self.kv_start, "lse": self.lse, **kw})

    def check(self, cfg, skip=()):
        t = s = 0
        for i, (n, m) in enumerate(zip(self.queries, self.keys)):
            if n and i not in skip:
                kv = self.kv[s:s + m]
                k = torch.cat([kv[..., :K], self.rope[s:s + m, None].expand(-1, self.H, -1)], -1)
                check_attention(self.out[t:t + n], self.lse[t:t + n], attention64(self.q[t:t + n], k, kv[..., K:], cfg.scale, cfg.causal),
                                f"sequence {i}")
            t, s = t + n, s + m


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: f"{sum(c[0])}x{c[2]}-{sum(c[1] or c[0])}-{c[3]}")
def test_prompt(k3, case):
    queries, keys, H, causal, padded = case
    c = Expanded(queries, keys, H, padded, sum(queries) + H)
    op, cfg = c.holder(k3, causal=causal)
    c(op)
    c.check(cfg)
    out, lse = c.out.clone(), c.lse.clone()
    c(op, lse=None)
    assert torch.equal(c.out, out)
    c(op)
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    if len(queries) == 1:                                  # one sequence needs no offsets
        c(op, seq_start=None, kv_start=None)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("queries,keys", [([300], [300]), ([40], [6000])])
def test_prompt_nan_queries(k3, queries, keys):
    c = Expanded(queries, keys, 2, False, 44)
    op, cfg = c.holder(k3)
    c(op)
    out, lse = c.out.clone(), c.lse.clone()
    bad = torch.zeros(c.T, 2, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[17, 0] = bad[-1, 1] = True
    c.q[bad] = float("nan")
    c(op)
    assert torch.isnan(c.out[bad]).all() and torch.isnan(c.lse[bad]).all()
    assert torch.equal(c.out[~bad], out[~bad]) and torch.equal(c.lse[~bad], lse[~bad])


@pytest.mark.parametrize("n_seq", [33, 384, 500])
def test_prompt_many_sequences(k3, n_seq):
    queries = [(0, 1, 7, 30)[i % 4] for i in range(n_seq)]
    c = Expanded(queries, [(13 * i) % 150 if i % 5 else 0 for i in range(n_seq)], 3, True, n_seq)
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_prompt_twice_at_once(k3):
    """Two holders on two streams beside each other, one of them with its keys in parts."""
    c, d = Expanded([300, 500], None, 8, False, 41), Expanded([20], [6000], 4, False, 42)
    (op, cfg), (op2, cfg2) = c.holder(k3), d.holder(k3)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        c(op, stream=streams[0])
        d(op2, stream=streams[1])
    torch.cuda.synchronize()
    c.check(cfg)
    d.check(cfg2)


@pytest.mark.parametrize("q_scale", [0.0, 8.0])
def test_prompt_flat_and_sharp(k3, q_scale):
    c = Expanded([700, 300], [900, 300], 2, False, 5, q_scale)
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)


def test_prompt_growing_scores(k3):
    for sign in (1, -1):
        c = Expanded([1200], None, 2, False, 6)
        c.q[:] = 0
        c.q[..., 0] = 32
        c.kv[..., 0] = (sign * 0.25 * torch.arange(1200, device="cuda"))[:, None].bfloat16()
        op, cfg = c.holder(k3)
        c(op)
        c.check(cfg)


def test_prompt_reports_what_does_not_fit(k3):
    c = Expanded([60, 70, 80], [60, 170, 80], 2, False, 8)
    op, cfg = c.holder(k3)
    for name, at, bad, lost in (("start", 3, 211, [2]), ("start", 0, -1, [0]), ("kv_start", 3, 311, [2]), ("kv_start", 2, 30, [1, 2])):
        t = getattr(c, name)
        kept = t.clone()
        t[at] = bad
        c.out[:], c.lse[:] = 7.5, 7.5
        c(op)
        c.check(cfg, skip=lost)
        i = lost[0]
        s = slice(sum(c.queries[:i]), sum(c.queries[:i + 1]))
        assert (c.out[s] == 7.5).all() and (c.lse[s] == 7.5).all()
        assert k3.k3moe_device_status(op.ws) == (6, 0x2)
        t.copy_(kept)
    c(op)
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


def test_prompt_leaves_other_rows(k3):
    """Tokens before the first sequence and behind the last stay as they are, whatever lies there."""
    c = Expanded([50, 200, 100, 30], None, 3, False, 10)
    for t in (c.q, c.kv, c.rope):
        t[:50], t[350:] = float("nan"), float("inf")
    op, cfg = c.holder(k3)
    c(op, seq_start=c.start[1:4].contiguous())
    assert (c.out[:50] == 7.5).all() and (c.out[350:] == 7.5).all() and (c.lse[:50] == 7.5).all() and (c.lse[350:] == 7.5).all()
    c.check(cfg, skip=[0, 3])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [100, 2000, 2850, 2997])
def test_prompt_parts_what_is_not_seen_does_not_matter(k3, value, at):
    """As below, with the keys in parts: a value reaches the queries that see it whichever part it is in."""
    c = Expanded([150], [3000], 2, False, 13)
    op, cfg = c.holder(k3)
    c(op)
    out, lse = c.out.clone(), c.lse.clone()
    c.kv[at, :, K] = value
    c(op)
    first = max(0, at - 2850)                              # the first query that sees it
    assert torch.equal(c.out[:first], out[:first]) and torch.equal(c.lse, lse) and torch.equal(c.out[first:, :, 1:], out[first:, :, 1:])
    assert not torch.isfinite(c.out[first:, :, 0]).any()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["key", "value", "rope"])
@pytest.mark.parametrize("at", [5, 127, 130, 299])
def test_prompt_what_is_not_seen_does_not_matter(k3, which, value, at):
    """A spoiled token reaches no query before its own, nor another sequence."""
    c = Expanded([300, 100], None, 2, False, 12)
    op, cfg = c.holder(k3)
    c(op)
    out, lse = c.out.clone(), c.lse.clone()
    if which == "rope":
        c.rope[at] = value
    else:
        c.kv[at, :, K if which == "value" else 3] = value
    c(op)
    seen = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    seen[at:300] = True
    assert torch.equal(c.out[~seen], out[~seen]) and torch.equal(c.lse[~seen], lse[~seen])
    if which == "value":
        assert not torch.isfinite(c.out[seen][..., 0]).any()
        assert torch.equal(c.out[seen][..., 1:], out[seen][..., 1:]) and torch.equal(c.lse, lse)
    elif value != value:
        assert torch.isnan(c.out[seen]).all()


def test_prompt_captured(k3):
    """A captured call replays on new inputs and lengths."""
    c = Expanded([100, 200], [150, 250], 2, False, 14)
    op, cfg = c.holder(k3)
    graph = k3._capture(lambda x, out: c(op), c.q, c.out)
    d = Expanded([260, 40], [300, 100], 2, False, 15)
    for name in ("q", "kv", "rope", "start", "kv_start"):
        getattr(c, name).copy_(getattr(d, name))
    graph.replay()
    c.queries, c.keys = d.queries, d.keys
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- together

def test_both_forms_agree_as_a_layer(k3):
    """A prompt and drafted tokens of two sequences, expanded; the same tokens through the written cache, absorbed.
    Rows, q and the projections are rounded to bf16 alike but for the absorbed queries and the attended latents:
    two roundings more, 2^-8 each of a head's 2-norm, and the outputs' own in both."""
    H, page, lens, step = 8, 32, [90, 33], 3
    r = randn(23)
    cfg = k3.k3moe_latent_config(H, page_size=page, rope="pairs", causal=1)
    T = sum(lens) + 2 * step
    op = k3.LatentAttention(cfg, 2, T)
    op.gain, op.inv_freq = 1 + 0.1 * r(C), 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    wk, wv = (r(H, K, C) / C ** 0.5).bfloat16(), (r(H, V, C) / C ** 0.5).bfloat16()
    expand = k3.Linear(k3.k3moe_linear_config(H * (K + V), C), T)
    expand.w = torch.cat([wk, wv], 1).reshape(H * (K + V), C).contiguous()
    absorb, value = k3.HeadLinear(k3.k3moe_head_linear_config(H, C, K), T), k3.HeadLinear(k3.k3moe_head_linear_config(H, V, C), T)
    absorb.w, value.w = wk.transpose(1, 2).contiguous(), wv
    whole = [n + step for n in lens]
    start = torch.tensor([0, *itertools.accumulate(whole)], dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(n) for n in whole]).int().cuda()
    q, c = r(T, H, K + R).bfloat16(), r(T, ROW).bfloat16()
    pages = torch.tensor([[3, 0, 5], [2, 4, -1]], dtype=torch.int32, device="cuda")
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(whole)]).cuda()
    slots = pages[seq, (positions // page).long()].long() * page + positions % page
    cache = op.new_cache(6)
    rows = op.write(c, positions, cache=cache, slots=slots, rows=torch.empty_like(c), q=q[..., K:], q_rope=q[..., K:])
    kv = expand(rows[:, :C], torch.empty(T, H * (K + V), dtype=torch.bfloat16, device="cuda")).view(T, H, K + V)
    expanded = op.prompt(q, kv, rows[:, C:], torch.empty(T, H, V, dtype=torch.bfloat16, device="cuda"), seq_start=start)
    last = torch.cat([torch.arange(n - step, n) + s for n, s in zip(whole, start.tolist())]).cuda()
    qa = torch.empty(2 * step, H, ROW, dtype=torch.bfloat16, device="cuda")
    absorb(q[last][..., :K], qa[..., :C])
    qa[..., C:] = q[last][..., K:]
    o = op.attend(qa, cache, pages, torch.tensor(whole, dtype=torch.int32, device="cuda"), torch.empty(2 * step, H, C, dtype=torch.bfloat16, device="cuda"),
                  seq_start=torch.tensor([0, step, 2 * step], dtype=torch.int32, device="cuda"))
    absorbed = value(o, torch.empty(2 * step, H, V, dtype=torch.bfloat16, device="cuda"))
    want = expanded[last].double()
    err = (absorbed.double() - want).norm(dim=-1) / want.norm(dim=-1)
    assert torch.isfinite(absorbed).all() and (err <= 6 * BF).all(), err.max()
    for holder in (op, expand, absorb, value):
        assert k3.k3moe_device_status(holder.ws) == (0, 0)
