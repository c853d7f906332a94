"""What is measured of the token-mixer operators: the gated delta rule (``k3moe_delta_rule``) and the
linear projection with its epilogue (``k3moe_linear``).

``run`` computes one pass.  Where ``own`` is false it is the plain form, in elementary torch operations
and 32 bits; where it is true it is the framework's own call on the same inputs.  ``exact`` computes the
same from the definitions in 64 bits: the delta rule token by token, the projection as one product.

Gated delta rule, per sequence and value head, state S [D][D] (keys x values):
    S = diag(exp(g_t)) S;  u = beta_t (v_t - S^T k_t);  S = S + k_t u^T;  o_t = scale * S^T q_t
with q and k divided by sqrt(sum x^2 + eps), the decay g per head or per key channel.
Linear: y = act(x W^T + bias) + residual.
"""
import math

import torch

own = False

D = 128                     # key and value width of a head
EPS = 1e-6
SCALE = D ** -0.5


def listed():
    return [
        # ---- gated delta rule
        # one user's next token: 56 heads of 128 (a hidden width of 7168), one launch's latency
        dict(name="delta_step_1", op="delta", n_seq=1, tokens=1, heads=56, qk_heads=56, channel=True),
        # a decode batch: one token for each of 96 sequences, q and k heads shared by two value heads
        dict(name="delta_step_96", op="delta", n_seq=96, tokens=96, heads=32, qk_heads=16, channel=False),
        # drafted tokens: 37 sequences of a few tokens each, ragged
        dict(name="delta_draft_37", op="delta", n_seq=37, tokens=149, heads=56, qk_heads=56, channel=True),
        # a ragged batch of prompts, odd lengths, shared q and k heads
        dict(name="delta_ragged_11", op="delta", n_seq=11, tokens=6007, heads=32, qk_heads=16, channel=False),
        # one long prompt, decay per channel
        dict(name="delta_prompt_8192", op="delta", n_seq=1, tokens=8192, heads=56, qk_heads=56, channel=True),
        # a full prefill batch, decay per head
        dict(name="delta_batch_16384", op="delta", n_seq=8, tokens=16384, heads=56, qk_heads=56, channel=False),
        # ---- linear
        # one token into the latent width, SiLU
        dict(name="linear_t1", op="linear", T=1, K=7168, N=3584, act="silu", bias=True, residual=False, f32=False, pad=0),
        # a decode batch through the output projection onto the residual stream
        dict(name="linear_t48", op="linear", T=48, K=3584, N=7168, act="none", bias=False, residual=True, f32=False, pad=0),
        # odd sizes: a gate of 4999 columns in f32 from a slice of a wider row
        dict(name="linear_t333", op="linear", T=333, K=1992, N=4999, act="logsigmoid", bias=True, residual=False, f32=True, pad=56),
        # a prompt through the output projection: bias and residual
        dict(name="linear_t4096", op="linear", T=4096, K=7168, N=7168, act="none", bias=True, residual=True, f32=False, pad=0),
        # the largest: a prefill batch through a fused projection with GELU
        dict(name="linear_t16384", op="linear", T=16384, K=3584, N=14336, act="gelu", bias=True, residual=False, f32=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: every length, head layout, gate and epilogue they stand for."""
    if rng.random() < 0.5:
        kind = rng.choice(["step", "draft", "prompt"])
        qk = rng.choice([3, 8, 16, 28, 56])
        heads = qk * (rng.choice([1, 2, 3]) if qk <= 16 else 1)
        if kind == "step":
            n = _log(rng, 1, 96)
            tokens = n
        elif kind == "draft":
            n = _log(rng, 1, 64)
            tokens = n + rng.randrange(0, 7 * n + 1)
        else:
            n = _log(rng, 1, 12)
            tokens = max(n, _log(rng, 40, 8192))
        return dict(op="delta", n_seq=n, tokens=tokens, heads=heads, qk_heads=qk, channel=rng.random() < 0.5)
    T, K = _log(rng, 1, 8192), 8 * _log(rng, 16, 896)
    N = _log(rng, 100, 7168)
    return dict(op="linear", T=T, K=K, N=N, act=rng.choice(["none", "relu", "silu", "gelu", "sigmoid", "logsigmoid"]),
                bias=rng.random() < 0.5, residual=rng.random() < 0.5, f32=rng.random() < 0.5, pad=8 * rng.randrange(0, 9))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _lengths(case, seed):
    """n_seq lengths of at least one token that sum to `tokens`."""
    n, T = case["n_seq"], case["tokens"]
    g = torch.Generator()
    g.manual_seed(int(seed) * 31 + 5)
    if T == n or n == 1:
        return [T // n] * n
    cuts = torch.sort(torch.rand(n - 1, generator=g)).values * (T - n)
    cuts = [0] + [int(c) for c in cuts] + [T - n]
    return [cuts[i + 1] - cuts[i] + 1 for i in range(n)]


def _delta_inputs(case, seed):
    """Activations as the projections leave them: q, k, v after SiLU in one fused row, decays with time
    constants from ten to a thousand tokens per head and channel, step sizes in (0, 1), a carried state."""
    g = _gen(seed)
    T, H, Hq, n = case["tokens"], case["heads"], case["qk_heads"], case["n_seq"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    qkv = torch.nn.functional.silu(r(T, (2 * Hq + H) * D)).bfloat16()
    G = D if case["channel"] else 1
    rate = torch.rand(H, 1, generator=g, device="cuda") * 15 + 1
    dt = torch.exp(torch.rand(H, G, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    inv = dt + torch.log(-torch.expm1(-dt))
    gate = -rate * torch.nn.functional.softplus(0.5 * r(T, H, G) + inv)
    beta = torch.sigmoid(r(T, H))
    slots = torch.randperm(n + 3, generator=g, device="cuda")[:n].int()
    state = 0.3 * r(n + 3, H, D, D)
    lens = _lengths(case, seed)
    start = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:2 * Hq * D].view(T, Hq, D)
    v = qkv[:, 2 * Hq * D:].view(T, H, D)
    return dict(q=q, k=k, v=v, g=gate, beta=beta, slots=slots, state=state, start=start, lens=lens)


def _linear_inputs(case, seed):
    g = _gen(seed)
    T, K, N = case["T"], case["K"], case["N"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = r(T, K + case["pad"]).bfloat16()[:, :K]
    w = (r(N, K) / math.sqrt(K)).bfloat16()
    kind = torch.float32 if case["f32"] else torch.bfloat16
    return dict(x=x, w=w, bias=0.5 * r(N) if case["bias"] else None, residual=r(T, N).to(kind) if case["residual"] else None)


def prepare(case, seed):
    s = _delta_inputs(case, seed) if case["op"] == "delta" else _linear_inputs(case, seed)
    s["case"] = case
    if own:
        import sparse_moe_expert_k3moe_gb300 as k3
        if case["op"] == "delta":
            cfg = k3.k3moe_delta_config(n_heads=case["heads"], n_qk_heads=case["qk_heads"], head_dim=D,
                                        gate_dim=D if case["channel"] else 1, qk_norm=1, norm_eps=EPS, scale=SCALE)
            s["op"] = k3.DeltaRule(cfg, case["n_seq"], case["tokens"])
            s["out"] = torch.empty(case["tokens"], case["heads"], D, dtype=torch.bfloat16, device="cuda")
            s["state_out"] = torch.zeros_like(s["state"])
        else:
            cfg = k3.k3moe_linear_config(n=case["N"], k=case["K"], act=case["act"], y_f32=case["f32"])
            s["op"] = k3.Linear(cfg, case["T"])
            s["op"].w, s["op"].bias = s["w"], s["bias"]
            s["out"] = torch.empty(case["T"], case["N"], dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms, 32 bits

def _padded(s, x, L):
    """x [T][...] as [n_seq][L][...], zeros after each sequence's end."""
    n = len(s["lens"])
    at = s["start"][:-1, None].long() + torch.arange(L, device="cuda")[None]
    ok = torch.arange(L, device="cuda")[None] < (s["start"][1:] - s["start"][:-1])[:, None]
    y = x[at.clamp(max=x.shape[0] - 1)]
    return torch.where(ok.view(n, L, *([1] * (x.dim() - 1))), y, torch.zeros((), dtype=x.dtype, device="cuda")), ok


def _delta_plain(s):
    """Chunks of 16 tokens: the pairwise products within each chunk for all chunks at once, then the
    state from chunk to chunk."""
    case = s["case"]
    H, Hq, n = case["heads"], case["qk_heads"], case["n_seq"]
    C = min(16, max(s["lens"]))
    nc = -(-max(s["lens"]) // C)
    L = nc * C

    def heads(x, ok_too=False):                                    # [n][nc][H][C][..]
        y, ok = _padded(s, x, L)
        y = y.float()
        if y.shape[2] != H:
            y = y.repeat_interleave(H // Hq, dim=2)
        return y.view(n, nc, C, H, -1).transpose(2, 3), ok

    q, k, v, g = (heads(s[m])[0] for m in ("q", "k", "v", "g"))
    b = heads(s["beta"].unsqueeze(-1))[0]
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS) * SCALE
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    G = torch.cumsum(g, dim=3)                                      # [..][C][1 or D]
    if g.shape[-1] == 1:
        E = torch.exp(torch.clamp(G - G.transpose(3, 4), max=0.0))
        A, P = (k @ k.transpose(3, 4)) * E, (q @ k.transpose(3, 4)) * E
    else:
        E = torch.exp(torch.clamp(G.unsqueeze(4) - G.unsqueeze(3), max=0.0)) * k.unsqueeze(3)   # [..][t][i][D]
        A, P = (E @ k.unsqueeze(-1)).squeeze(-1), (E @ q.unsqueeze(-1)).squeeze(-1)
        del E
    A, P = torch.tril(A * b, -1), torch.tril(P)
    eye = torch.eye(C, device="cuda")
    inv, A2 = eye - A, A @ A                                        # (I + A)^-1 of a nilpotent A: (I - A)(I + A^2)(I + A^4)(I + A^8)
    inv = inv @ (eye + A2)
    A4 = A2 @ A2
    inv = inv @ (eye + A4)
    inv = inv @ (eye + A4 @ A4)
    Tm = inv * b.transpose(3, 4)
    kd, qd = k * torch.exp(G), q * torch.exp(G)
    kl = k * torch.exp(G[..., -1:, :] - G)
    end = torch.exp(G[..., -1, :]).unsqueeze(-1)                    # [..][1 or D][1]
    S = s["state"][s["slots"].long()]
    outs = []
    for c in range(nc):
        U = Tm[:, c] @ (v[:, c] - kd[:, c] @ S)
        outs.append(qd[:, c] @ S + P[:, c] @ U)
        S = end[:, c] * S + kl[:, c].transpose(2, 3) @ U
    o = torch.stack(outs, 1).transpose(2, 3).reshape(n, L, H, D)
    ok = torch.arange(L, device="cuda")[None] < (s["start"][1:] - s["start"][:-1])[:, None]
    state = torch.zeros_like(s["state"])
    state[s["slots"].long()] = S
    return {"out": o[ok].bfloat16(), "state": state}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * (0.5 ** 0.5)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "logsigmoid":
        return torch.clamp(z, max=0) - torch.log1p(torch.exp(-torch.abs(z)))
    return z


def _linear_plain(s):
    case = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _act(z, case["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z if case["f32"] else z.bfloat16()


def run(state):
    s = state
    if not own:
        return _delta_plain(s) if s["case"]["op"] == "delta" else _linear_plain(s)
    if s["case"]["op"] == "delta":
        s["op"](s["q"], s["k"], s["v"], s["g"], s["beta"], s["out"], s["state"], s["state_out"], seq_start=s["start"], slots=s["slots"])
        return {"out": s["out"], "state": s["state_out"]}
    return s["op"](s["x"], s["out"], residual=s["residual"])


def work(case):
    if case["op"] == "delta":
        T, H, Hq, n = case["tokens"], case["heads"], case["qk_heads"], case["n_seq"]
        G = D if case["channel"] else 1
        token = 2 * 2 * D * Hq + 2 * D * H + 4 * G * H + 4 * H + 2 * D * H
        return {"bytes": T * token + n * H * 2 * 4 * D * D, "flops": T * H * 7 * D * D}
    T, K, N = case["T"], case["K"], case["N"]
    size = 4 if case["f32"] else 2
    return {"bytes": 2 * T * K + 2 * N * K + T * N * size * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
            "flops": 2 * T * N * K}


# ----------------------------------------------------------------------------- the definitions, 64 bits

def _delta_exact(case, seed):
    s = _delta_inputs(case, seed)
    H, Hq, lens = case["heads"], case["qk_heads"], s["lens"]
    rep = H // Hq
    out = torch.zeros(case["tokens"], H, D, dtype=torch.float64, device="cuda")
    state = torch.zeros(s["state"].shape, dtype=torch.float64, device="cuda")
    S = s["state"].double()[s["slots"].long()]
    first = s["start"][:-1].long()
    order = sorted(range(len(lens)), key=lambda i: -lens[i])          # longest first: the live ones are a prefix
    idx = torch.tensor(order, device="cuda")
    S, first = S[idx], first[idx]
    for t in range(lens[order[0]]):
        live = sum(1 for i in order if lens[i] > t)
        at = first[:live] + t
        q, k = s["q"][at].double(), s["k"][at].double()
        q = (q / (q.pow(2).sum(-1, keepdim=True) + EPS).sqrt() * SCALE).repeat_interleave(rep, 1)
        k = (k / (k.pow(2).sum(-1, keepdim=True) + EPS).sqrt()).repeat_interleave(rep, 1)
        W = S[:live] * s["g"][at].double().exp().unsqueeze(-1)
        u = s["beta"][at].double().unsqueeze(-1) * (s["v"][at].double() - torch.einsum("nhk,nhkv->nhv", k, W))
        W = W + k.unsqueeze(-1) * u.unsqueeze(-2)
        S[:live] = W
        out[at] = torch.einsum("nhk,nhkv->nhv", q, W)
    state[s["slots"].long()[idx]] = S
    return {"out": out, "state": state}


def exact(case, seed):
    if case["op"] == "delta":
        return _delta_exact(case, seed)
    s = _linear_inputs(case, seed)
    if 2.0 * case["T"] * case["K"] * case["N"] > 6e12:
        return None                                                 # over 20 seconds in 64 bits
    z = torch.matmul(s["x"].double(), s["w"].double().T)
    if s["bias"] is not None:
        z += s["bias"].double()
    act = case["act"]
    if act == "relu":
        z = z.clamp(min=0)
    elif act == "silu":
        z = z * torch.special.expit(z)
    elif act == "gelu":
        z = z * torch.special.ndtr(z)
    elif act == "sigmoid":
        z = torch.special.expit(z)
    elif act == "logsigmoid":
        z = -torch.logaddexp(torch.zeros_like(z), -z)
    return z if s["residual"] is None else z + s["residual"].double()
