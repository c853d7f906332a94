"""What is measured of the latent attention's operators: a block's norms with its gate and residual
scale (``k3moe_norm``), the projections of each head (``k3moe_head_linear``), the write of the latent
cache (``k3moe_latent_write``), attention over it in the absorbed form (``k3moe_latent_attend``) and over
expanded keys and values (``k3moe_latent_prompt``).

``run`` computes one pass.  Where ``own`` is false it is the plain form, in elementary torch operations
and 32 bits (angles in 64); where it is true it is the framework's own call on the same inputs.
``exact`` computes the same from the definitions in 64 bits.

Norm, a row of N:  y = x / sqrt(mean x^2 + eps) * post_gain (over the row, or over each head's 128),
    y *= act(gate), total = residual + alpha * scale * y, out = total / sqrt(mean total^2 + eps) * pre_gain.
Head projection:   y[t][h] = W[h] x[t][h].
Latent write:      row = [c / sqrt(mean c^2 + eps) * gain, rotate(r, position)] of a token's [c, r]; the
    row goes to the token's slot of the cache, and q's 64 last columns of every head are rotated.
Absorbed:          s_j = scale q . row_j over a sequence's cached rows, out = sum softmax(s)_j c_j,
    lse = log sum exp(s); the i-th of n queries sees all rows but the n - 1 - i last.
Expanded:          the same with keys [k_j of the head, r_j] and values v_j of the head.
"""
import math

import torch

own = False

C, R = 512, 64              # a token's latent and its rotated part
ROW = C + R
K, V = 128, 128             # a head's keys (beside R) and values in the expanded form
EPS = 1e-6
SCALE = (K + R) ** -0.5
BASE = 50000.0              # of the rotation's frequencies


def listed():
    return [
        # ---- norms around a block
        # one user's next token: the block's output normed, scaled onto the residual, normed for the next block
        dict(name="norm_t1", op="norm", T=1, N=7168, heads=False, gate="none", x_f32=False, sum_f32=False, residual=True, pre=True),
        # a prompt through the gated norm of each head after the token mixer
        dict(name="norm_heads_t8192", op="norm", T=8192, N=7168, heads=True, gate="sigmoid", x_f32=False, sum_f32=False, residual=False, pre=False),
        # ---- a head's own projection
        # one token's queries into the latent
        dict(name="head_t1", op="head", T=1, H=56, K=128, N=512),
        # a decode batch of odd size: the attended latents back to values
        dict(name="head_t333", op="head", T=333, H=56, K=512, N=128),
        # ---- the cache's write
        # a decode batch's tokens, far positions
        dict(name="write_t37", op="write", T=37, H=56, page=64, rope="pairs"),
        # a prompt's tokens
        dict(name="write_t8192", op="write", T=8192, H=56, page=64, rope="halves"),
        # ---- absorbed attention over the cache
        # one user, a short context: latency
        dict(name="attend_1", op="attend", n_seq=1, tokens=1, H=56, longest=777, even=True, page=64),
        # one user, a long context: work split over it
        dict(name="attend_long", op="attend", n_seq=1, tokens=1, H=56, longest=131071, even=True, page=64),
        # a decode batch of ragged contexts
        dict(name="attend_96", op="attend", n_seq=96, tokens=96, H=56, longest=8192, even=False, page=64),
        # drafted tokens, small pages, few heads
        dict(name="attend_draft_11", op="attend", n_seq=11, tokens=40, H=16, longest=5003, even=False, page=16),
        # ---- expanded attention
        # a ragged batch of short prompts, some behind a cached prefix
        dict(name="prompt_ragged_7", op="prompt", n_seq=7, tokens=3001, H=16, prefix=700),
        # one long prompt
        dict(name="prompt_8192", op="prompt", n_seq=1, tokens=8192, H=56, prefix=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges."""
    op = rng.choice(["norm", "head", "write", "attend", "attend", "prompt", "prompt"])
    if op == "norm":
        heads = rng.random() < 0.4
        N = 128 * _log(rng, 1, 64) if heads else 8 * _log(rng, 16, 1024)
        residual = rng.random() < 0.6
        T = min(_log(rng, 1, 8192), 8192 * 3584 // N)
        return dict(op=op, T=max(T, 1), N=N, heads=heads, gate=rng.choice(["none", "sigmoid", "silu"]), x_f32=rng.random() < 0.3,
                    sum_f32=rng.random() < 0.3, residual=residual, pre=residual and rng.random() < 0.7)
    if op == "head":
        K_, N = rng.choice([(128, 512), (512, 128), (64, 192), (192, 72)])
        return dict(op=op, T=_log(rng, 1, 333), H=rng.choice([3, 8, 16, 28, 56]), K=K_, N=N)
    if op == "write":
        return dict(op=op, T=_log(rng, 1, 8192), H=rng.choice([3, 8, 16, 28, 56]), page=rng.choice([16, 32, 64, 128]),
                    rope=rng.choice(["none", "pairs", "halves"]))
    if op == "attend":
        n = _log(rng, 1, 96)
        tokens = n + (rng.randrange(0, 3 * n + 1) if rng.random() < 0.4 else 0)
        longest = _log(rng, 16, 131071 if n == 1 else 8192)
        H = rng.choice([1, 8, 13, 16, 28, 56, 64, 128])
        while tokens * longest * H > 96 * 4096 * 56:
            longest = longest * 2 // 3
        return dict(op=op, n_seq=n, tokens=tokens, H=H, longest=max(longest, 16), even=rng.random() < 0.3, page=rng.choice([16, 32, 64, 128]))
    n = _log(rng, 1, 12)
    tokens, prefix, H = max(n, _log(rng, 1, 8192)), rng.choice([0, 0, _log(rng, 1, 4096)]), rng.choice([1, 3, 8, 16, 28, 56])
    while tokens * (tokens + 2 * prefix * n) * H > 8192 * 8192 * 56 or tokens > 4096 and prefix * n > 8192:
        prefix //= 2
    return dict(op="prompt", n_seq=n, tokens=tokens, H=H, prefix=prefix)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6271 + 29)
    return g


def _cuts(n, T, seed, least=1):
    """n lengths of at least `least` that sum to T."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 37 + 3)
    spare = T - least * n
    if spare <= 0 or n == 1:
        return [T // n] * n
    cuts = torch.sort(torch.rand(n - 1, generator=g)).values * spare
    cuts = [0] + [int(c) for c in cuts] + [spare]
    return [cuts[i + 1] - cuts[i] + least for i in range(n)]


def _starts(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def _norm_inputs(case, seed):
    g = _gen(seed)
    T, N = case["T"], case["N"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kx, ks = (torch.float32 if case[m] else torch.bfloat16 for m in ("x_f32", "sum_f32"))
    width = 128 if case["heads"] else N
    s = dict(x=(0.7 * r(T, N)).to(kx), gate=r(T, N).bfloat16() if case["gate"] != "none" else None,
             post_gain=1 + 0.1 * r(width), residual=None, scale=None, pre_gain=None, ks=ks)
    if case["residual"]:
        s["residual"] = (3 * r(T, N)).to(ks)
        s["scale"] = 0.5 + 0.1 * r(N)
    if case["pre"]:
        s["pre_gain"] = 1 + 0.1 * r(N)
    return s


def _head_inputs(case, seed):
    """x and y are a head's columns of wider rows, as they are in a layer's queries."""
    g = _gen(seed)
    T, H, K_, N = case["T"], case["H"], case["K"], case["N"]
    x = torch.randn(T, H, K_ + 64, generator=g, device="cuda").bfloat16()[..., :K_]
    return dict(x=x, w=(torch.randn(H, N, K_, generator=g, device="cuda") / math.sqrt(K_)).bfloat16())


def _freq():
    return BASE ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") * 2 / R)


def _write_inputs(case, seed):
    g = _gen(seed)
    T, H, page = case["T"], case["H"], case["page"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if T > 2 * page:                                             # a prompt: whole pages in turn
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda")
        slots = order[at // page] * page + at % page
        positions = (torch.randint(0, 100000, (1,), generator=g, device="cuda") + at).int()
    else:
        positions = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").int()
    return dict(c=r(T, ROW).bfloat16(), q=r(T, H, K + R).bfloat16(), gain=1 + 0.1 * r(C), positions=positions, slots=slots,
                cache=r(pages, page, ROW).bfloat16(), freq=_freq())


def _attend_inputs(case, seed):
    g = _gen(seed)
    T, H, n, page = case["tokens"], case["H"], case["n_seq"], case["page"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    queries = _cuts(n, T, seed)
    gl = torch.Generator()
    gl.manual_seed(int(seed) * 41 + 7)
    if case["even"]:
        lens = [case["longest"]] * n
    else:                                                        # half of them long, some short
        u = torch.rand(n, generator=gl)
        lens = [max(1, int(case["longest"] * float(x) ** 0.9)) for x in u]
        lens[int(u.argmax())] = case["longest"]
    lens = [max(x, y) for x, y in zip(lens, queries)]
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 5
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((n, max(need) + 2), -1, dtype=torch.int32, device="cuda")     # what lies behind a sequence is no page
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    cache = torch.empty(n_pages, page, ROW, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (page * ROW))
    for i in range(0, n_pages, step):
        cache[i:i + step] = r(min(step, n_pages - i), page, ROW).bfloat16()
    return dict(q=r(T, H, ROW).bfloat16(), cache=cache, table=table, lens=lens, queries=queries, kv=torch.tensor(lens, device="cuda").int(),
                start=_starts(queries))


def _prompt_inputs(case, seed):
    g = _gen(seed)
    T, H, n = case["tokens"], case["H"], case["n_seq"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    queries = _cuts(n, T, seed)
    keys = [x + (case["prefix"] * i // max(n - 1, 1) if n > 1 else case["prefix"]) for i, x in enumerate(queries)]
    S = sum(keys)
    rows = r(S, ROW).bfloat16()
    return dict(q=r(T, H, K + R).bfloat16(), kv=r(S, H, K + V).bfloat16(), rope=rows[:, C:], queries=queries, keys=keys,
                start=_starts(queries), kv_start=_starts(keys))


INPUTS = dict(norm=_norm_inputs, head=_head_inputs, write=_write_inputs, attend=_attend_inputs, prompt=_prompt_inputs)


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    s["case"] = case
    op = case["op"]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op == "write":
        s["rows"], s["q_rope"] = torch.empty(case["T"], ROW, **bf), torch.empty(case["T"], case["H"], ROW, **bf)[..., C:]
    if not own:
        return s
    import sparse_moe_expert_k3moe_gb300 as k3
    if op == "norm":
        s["op"] = k3.Norm(k3.k3moe_norm_config(case["N"], group=128 if case["heads"] else 0, gate=case["gate"], pre_norm=case["pre"],
                                               x_f32=case["x_f32"], sum_f32=case["sum_f32"], eps=EPS, alpha=0.75))
        s["op"].post_gain, s["op"].scale, s["op"].pre_gain = s["post_gain"], s["scale"], s["pre_gain"]
        s["total"] = torch.empty(case["T"], case["N"], dtype=s["ks"], device="cuda")
        s["out"] = torch.empty(case["T"], case["N"], **bf) if case["pre"] else None
    elif op == "head":
        s["op"] = k3.HeadLinear(k3.k3moe_head_linear_config(case["H"], case["N"], case["K"]), case["T"])
        s["op"].w = s["w"]
        s["out"] = torch.empty(case["T"], case["H"], case["N"] + 64, **bf)[..., :case["N"]]
    else:
        cfg = k3.k3moe_latent_config(case["H"], page_size=case.get("page", 64), rope=case.get("rope", "none"), norm_eps=EPS, scale=SCALE)
        tokens = case["T"] if op == "write" else case["tokens"]
        s["op"] = k3.LatentAttention(cfg, case.get("n_seq", 0), tokens)
        if op == "write":
            s["op"].gain, s["op"].inv_freq = s["gain"], s["freq"]
        else:
            s["out"] = torch.empty(tokens, case["H"], C if op == "attend" else V, **bf)
            s["lse"] = torch.empty(tokens, case["H"], dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms, 32 bits

def _norm_plain(s):
    case = s["case"]
    x = s["x"].float()
    y = x.view(case["T"], -1, 128) if case["heads"] else x
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post_gain"]
    y = y.reshape(x.shape)
    if s["gate"] is not None:
        z = s["gate"].float()
        w = 1 / (1 + torch.exp(-z))
        y = y * (w if case["gate"] == "sigmoid" else z * w)
    y = 0.75 * y
    if s["scale"] is not None:
        y = y * s["scale"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"total": y.to(s["ks"])}
    if case["pre"]:
        out["out"] = (y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["pre_gain"]).bfloat16()
    return out


def _head_plain(s):
    return torch.bmm(s["x"].float().transpose(0, 1), s["w"].float().transpose(1, 2)).transpose(0, 1).contiguous().bfloat16()


def _rotate(x, positions, freq, how):
    """x [T][..][64] in 32 bits, rotated by angles taken in 64."""
    if how == "none":
        return x
    a = torch.remainder(positions.double()[:, None] * freq, 2 * math.pi)
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    if x.dim() == 3:
        cos, sin = cos[:, None], sin[:, None]
    if how == "pairs":
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    u, v = x[..., :R // 2], x[..., R // 2:]
    return torch.cat([u * cos - v * sin, v * cos + u * sin], -1)


def _write_plain(s):
    how = s["case"]["rope"]
    c = s["c"][:, :C].float()
    c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * s["gain"]
    rows = torch.cat([c, _rotate(s["c"][:, C:].float(), s["positions"], s["freq"], how)], -1).bfloat16()
    s["cache"].view(-1, ROW)[s["slots"]] = rows
    return {"rows": rows, "cache": s["cache"], "q_rope": _rotate(s["q"][..., K:].float(), s["positions"], s["freq"], how).bfloat16()}


def _softmax(s):
    """(weights, log of the sum) over the last axis."""
    m = s.max(-1, keepdim=True).values
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    return e / z, (m + torch.log(z)).squeeze(-1)


def _seen(queries, keys):
    """[queries][keys]: which keys each query sees."""
    return torch.arange(keys, device="cuda")[None] <= torch.arange(queries, device="cuda")[:, None] + (keys - queries)


def _attend_plain(s):
    """Sequences of alike lengths together, their rows gathered page by page."""
    case = s["case"]
    n, H, page, lens, queries = case["n_seq"], case["H"], case["page"], s["lens"], s["queries"]
    out = torch.empty(case["tokens"], H, C, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(case["tokens"], H, dtype=torch.float32, device="cuda")
    first = [0]
    for x in queries:
        first.append(first[-1] + x)
    order = sorted(range(n), key=lambda i: (queries[i], lens[i]))
    while order:
        nq = queries[order[0]]
        group = [i for i in order if queries[i] == nq][:16]
        order = [i for i in order if i not in group]
        L = max(lens[i] for i in group)
        idx = torch.tensor(group, device="cuda")
        rows = s["cache"][s["table"][idx, :-(-L // page)].long().clamp(min=0)].view(len(group), -1, ROW)[:, :L].float()
        rows = torch.where((torch.arange(L, device="cuda")[None] < s["kv"][idx, None])[..., None], rows, 0.0)
        at = torch.tensor([[first[i] + j for j in range(nq)] for i in group], device="cuda")
        q = s["q"][at].float().view(len(group), nq * H, ROW)
        z = (torch.bmm(q, rows.transpose(1, 2)) * SCALE).view(len(group), nq, H, L)
        sees = torch.arange(L, device="cuda") < (s["kv"][idx, None] - nq + 1 + torch.arange(nq, device="cuda")[None])[..., None]
        p, ls = _softmax(torch.where(sees[:, :, None], z, -math.inf))
        out[at] = torch.bmm(p.view(len(group), nq * H, L), rows[..., :C]).view(len(group), nq, H, C).bfloat16()
        lse[at] = ls
    return {"out": out, "lse": lse}


def _prompt_plain(s):
    case = s["case"]
    H = case["H"]
    out = torch.empty(case["tokens"], H, V, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(case["tokens"], H, dtype=torch.float32, device="cuda")
    t0 = k0 = 0
    for nq, nk in zip(s["queries"], s["keys"]):
        sees = _seen(nq, nk)
        step = max(1, (1 << 28) // (nq * nk))
        for h in range(0, H, step):
            q = s["q"][t0:t0 + nq, h:h + step].float().transpose(0, 1)
            kv = s["kv"][k0:k0 + nk, h:h + step].float().transpose(0, 1)
            k = torch.cat([kv[..., :K], s["rope"][k0:k0 + nk].float()[None].expand(kv.shape[0], -1, -1)], -1)
            z = torch.where(sees, torch.bmm(q, k.transpose(1, 2)) * SCALE, -math.inf)
            p, ls = _softmax(z)
            out[t0:t0 + nq, h:h + step] = torch.bmm(p, kv[..., K:]).transpose(0, 1).bfloat16()
            lse[t0:t0 + nq, h:h + step] = ls.t()
        t0, k0 = t0 + nq, k0 + nk
    return {"out": out, "lse": lse}


PLAIN = dict(norm=_norm_plain, head=_head_plain, write=_write_plain, attend=_attend_plain, prompt=_prompt_plain)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return PLAIN[op](s)
    if op == "norm":
        s["op"](s["x"], out=s["out"], gate=s["gate"], residual=s["residual"], total=s["total"])
        return {"total": s["total"], "out": s["out"]} if s["case"]["pre"] else {"total": s["total"]}
    if op == "head":
        return s["op"](s["x"], s["out"])
    if op == "write":
        s["op"].write(s["c"], s["positions"], cache=s["cache"], slots=s["slots"], rows=s["rows"], q=s["q"][..., K:], q_rope=s["q_rope"])
        return {"rows": s["rows"], "cache": s["cache"], "q_rope": s["q_rope"]}
    if op == "attend":
        s["op"].attend(s["q"], s["cache"], s["table"], s["kv"], s["out"], seq_start=s["start"], lse=s["lse"])
    else:
        s["op"].prompt(s["q"], s["kv"], s["rope"], s["out"], seq_start=s["start"], kv_start=s["kv_start"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _lens_of(case):
    """Lengths that a case's work is counted with: those of a seed of its own."""
    n, T = case["n_seq"], case["tokens"]
    queries = _cuts(n, T, 1)
    if case["op"] == "prompt":
        return queries, [x + (case["prefix"] * i // max(n - 1, 1) if n > 1 else case["prefix"]) for i, x in enumerate(queries)]
    longest = case["longest"]
    lens = [longest] * n if case["even"] else [max(1, round(longest * ((i + 0.5) / n) ** 0.9)) for i in range(n - 1)] + [longest]
    return queries, [max(x, y) for x, y in zip(lens, queries)]


def work(case):
    op = case["op"]
    if op == "norm":
        T, N = case["T"], case["N"]
        sx, ss = (4 if case[m] else 2 for m in ("x_f32", "sum_f32"))
        row = sx + ss + (2 if case["gate"] != "none" else 0) + (ss if case["residual"] else 0) + (2 if case["pre"] else 0)
        return {"bytes": T * N * row, "flops": 10 * T * N}
    if op == "head":
        T, H, K_, N = case["T"], case["H"], case["K"], case["N"]
        return {"bytes": 2 * H * (K_ * N + T * (K_ + N)), "flops": 2 * T * H * K_ * N}
    if op == "write":
        T, H = case["T"], case["H"]
        return {"bytes": T * (3 * 2 * ROW + 2 * 2 * R * H + 12), "flops": T * (4 * ROW + 3 * R * H)}
    queries, lens = _lens_of(case)
    H = case["H"]
    seen = sum(q * k - q * (q - 1) // 2 for q, k in zip(queries, lens))
    if op == "attend":
        return {"bytes": 2 * ROW * sum(lens) + case["tokens"] * H * (2 * ROW + 2 * C + 4), "flops": 2 * seen * H * (ROW + C)}
    return {"bytes": sum(lens) * 2 * (H * (K + V) + R) + case["tokens"] * H * (2 * (K + R + V) + 4), "flops": 2 * seen * H * (K + R + V)}


# ----------------------------------------------------------------------------- the definitions, 64 bits

def _norm_exact(case, s):
    x = s["x"].double()
    rms = lambda t: (t.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()  # noqa: E731
    if case["heads"]:
        y = (x.unflatten(-1, (-1, 128)) * rms(x.unflatten(-1, (-1, 128))) * s["post_gain"].double()).flatten(-2)
    else:
        y = x * rms(x) * s["post_gain"].double()
    if case["gate"] != "none":
        z = s["gate"].double()
        y = y * torch.special.expit(z) * (z if case["gate"] == "silu" else 1.0)
    total = 0.75 * y * (s["scale"].double() if s["scale"] is not None else 1.0)
    if s["residual"] is not None:
        total = total + s["residual"].double()
    return {"total": total, "out": total * rms(total) * s["pre_gain"].double()} if case["pre"] else {"total": total}


def _write_exact(case, s):
    freq = torch.exp(-torch.arange(R // 2, dtype=torch.float64, device="cuda") * (2 * math.log(BASE) / R))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * freq)

    def rotate(x):
        x = x.double()
        if case["rope"] == "none":
            return x
        pairs = x.unflatten(-1, (-1, 2)) if case["rope"] == "pairs" else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_complex(pairs.contiguous()) * (turn if x.dim() == 2 else turn[:, None])
        z = torch.view_as_real(z)
        return (z if case["rope"] == "pairs" else z.transpose(-1, -2)).flatten(-2)

    c = s["c"][:, :C].double()
    rows = torch.cat([c * s["gain"].double() / (c.square().sum(-1, keepdim=True) / C + EPS).sqrt(), rotate(s["c"][:, C:])], -1)
    cache = s["cache"].double()
    cache.view(-1, ROW).index_copy_(0, s["slots"], rows)
    return {"rows": rows, "cache": cache, "q_rope": rotate(s["q"][..., K:])}


def _attend_exact(case, s):
    out, lse, t0 = [], [], 0
    for i, (nq, L) in enumerate(zip(s["queries"], s["lens"])):
        at = torch.arange(L, device="cuda")
        rows = s["cache"][s["table"][i, at // case["page"]].long(), at % case["page"]].double()
        z = SCALE * torch.einsum("qhc,lc->qhl", s["q"][t0:t0 + nq].double(), rows)
        for j in range(nq):
            z[j, :, L - (nq - 1 - j):] = -math.inf
        lse.append(torch.logsumexp(z, -1))
        out.append(torch.einsum("qhl,lc->qhc", torch.exp(z - lse[-1][..., None]), rows[:, :C]))
        t0 += nq
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _prompt_exact(case, s):
    out = torch.empty(case["tokens"], case["H"], V, dtype=torch.float64, device="cuda")
    lse = torch.empty(case["tokens"], case["H"], dtype=torch.float64, device="cuda")
    t0 = k0 = 0
    for nq, nk in zip(s["queries"], s["keys"]):
        rope = s["rope"][k0:k0 + nk].double()
        for h in range(case["H"]):
            kv = s["kv"][k0:k0 + nk, h].double()
            for a in range(0, nq, 2048):                           # a block of queries against what its last one sees
                b = min(nq, a + 2048)
                seen = nk - nq + b
                q = s["q"][t0 + a:t0 + b, h].double()
                z = (q[:, :K] @ kv[:seen, :K].T + q[:, K:] @ rope[:seen].T) * SCALE
                z.masked_fill_(torch.ones(b - a, seen, dtype=torch.bool, device="cuda").triu(seen - (b - a) + 1), -math.inf)
                ls = torch.logsumexp(z, -1)
                out[t0 + a:t0 + b, h] = torch.exp(z - ls[:, None]) @ kv[:seen, K:]
                lse[t0 + a:t0 + b, h] = ls
        t0, k0 = t0 + nq, k0 + nk
    return {"out": out, "lse": lse}


def exact(case, seed):
    op, s = case["op"], INPUTS[case["op"]](case, seed)
    if op == "head":
        return torch.einsum("thk,hnk->thn", s["x"].double(), s["w"].double())
    return dict(norm=_norm_exact, write=_write_exact, attend=_attend_exact, prompt=_prompt_exact)[op](case, s)
