"""Refusals and sizes of the latent attention's entry points (no GPU needed): every check is on
the host and comes before any CUDA call."""
import ctypes
import struct

import pytest

from sparse_moe_expert_k3moe_gb300 import build as kbuild

A = 0x10000000      # a fake, 256-aligned address: never dereferenced on the host
B, C = A + (1 << 20), A + (2 << 20)
BIG = 1 << 40
OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def k3():
    kbuild.build()
    import sparse_moe_expert_k3moe_gb300 as k3
    k3.lib()
    return k3


def vp(a):
    return ctypes.c_void_p(a) if a else None


def norm(k3, nc=None, T=4, x=A, xs=256, gate=B, gs=256, post=A, res=C, rs=256, scale=A, total=C + 4096, ts=256, pre=A, out=C + 8192, os=256):
    nc = nc or k3.k3moe_norm_config(256, 128, gate="silu")
    return k3.lib().k3moe_norm(ctypes.byref(nc), T, vp(x), xs, vp(gate), gs, vp(post), vp(res), rs, vp(scale), vp(total), ts, vp(pre),
                               vp(out), os, None)


def test_norm_refusals(k3):
    cfg = lambda n=256, *a, **kw: k3.k3moe_norm_config(n, *a, **{"gate": "silu", **kw})  # noqa: E731
    for nc in (cfg(0), cfg(-8), cfg(256, -1), cfg(gate=3), cfg(gate=-1), cfg(post_norm=2), cfg(pre_norm=2), cfg(eps=0.0), cfg(eps=NAN),
               cfg(eps=INF), cfg(alpha=INF), cfg(alpha=NAN)):
        assert norm(k3, nc) == EINVAL
    bad = cfg()
    bad.x_f32 = 2
    assert norm(k3, bad) == EINVAL
    for nc in (cfg(260), cfg(16392), cfg(256, 32), cfg(256, 192), cfg(320, 128), cfg(256, 512)):
        assert norm(k3, nc) == ESHAPE
    assert norm(k3, T=-1) == norm(k3, T=(1 << 20) + 1) == ESHAPE
    assert norm(k3, x=0) == norm(k3, post=0) == norm(k3, pre=0) == norm(k3, out=0) == norm(k3, gate=0) == EINVAL
    assert norm(k3, cfg(gate="none")) == norm(k3, cfg(pre_norm=0)) == EINVAL        # a gate, an out that the config has not
    assert norm(k3, cfg(pre_norm=0), out=0, total=0) == EINVAL
    for name in ("xs", "gs", "rs", "ts", "os"):
        assert norm(k3, **{name: 248}) == norm(k3, **{name: 260}) == norm(k3, **{name: 1 << 40}) == ESHAPE
    assert norm(k3, total=C, ts=264) == EINVAL                        # the residual itself, with another stride
    assert norm(k3, cfg(sum_f32=True), total=A) == EINVAL             # x itself, with another type
    assert norm(k3, cfg(sum_f32=True), out=C) == norm(k3, total=B, ts=264) == norm(k3, total=C + 8192) == EINVAL
    for name in ("x", "gate", "post", "res", "scale", "total", "pre", "out"):
        assert norm(k3, **{name: A + 8}) == EALIGN
    assert k3.lib().k3moe_norm(None, 1, vp(A), 8, None, 0, None, None, 0, None, vp(B), 8, None, None, 0, None) == EINVAL
    assert norm(k3, T=0, x=0, gate=0, total=0, out=0) == OK            # nothing to do


def head(k3, hc=None, T=4, x=A, xs=1024, xh=128, w=A, y=B, ys=4096, yh=512, ws=A, wb=BIG):
    hc = hc or k3.k3moe_head_linear_config(8, 512, 128)
    return k3.lib().k3moe_head_linear(ctypes.byref(hc), T, vp(x), xs, xh, vp(w), vp(y), ys, yh, vp(ws), wb, None)


def test_head_linear_refusals(k3):
    cfg = k3.k3moe_head_linear_config
    for hc in (cfg(0, 512, 128), cfg(8, 0, 128), cfg(8, 512, 0), cfg(-1, 512, 128)):
        assert head(k3, hc) == EINVAL
    for hc in (cfg(1025, 512, 128), cfg(8, 8193, 128), cfg(8, 512, 520), cfg(8, 512, 124)):
        assert head(k3, hc) == ESHAPE
        with pytest.raises(k3.K3MoEError):
            k3.k3moe_head_linear_workspace_bytes(hc, 4)
    assert head(k3, T=-1) == head(k3, T=(1 << 20) + 1) == ESHAPE
    assert head(k3, x=0) == head(k3, w=0) == head(k3, y=0) == EINVAL
    assert head(k3, xs=1016) == head(k3, xs=1028) == head(k3, xh=120) == head(k3, xh=132, xs=8192) == head(k3, xh=136) == ESHAPE
    assert head(k3, ys=4095) == head(k3, yh=511) == head(k3, yh=513) == head(k3, ys=1 << 40) == head(k3, xs=1 << 40) == ESHAPE
    assert head(k3, x=A + 8) == head(k3, w=A + 8) == head(k3, y=B + 1) == EALIGN
    assert head(k3, ws=0) == head(k3, ws=A + 8) == head(k3, wb=256) == EWORKSPACE
    assert k3.lib().k3moe_head_linear(None, 1, vp(A), 8, 8, vp(A), vp(B), 8, 8, vp(A), BIG, None) == EINVAL
    assert head(k3, T=0, x=0, w=0, y=0, ws=0) == OK


def latent_configs(k3):
    cfg = lambda n=8, **kw: k3.k3moe_latent_config(n, **kw)  # noqa: E731
    invalid = [cfg(0), cfg(-1), cfg(rank=0), cfg(rope_dim=0), cfg(key_dim=0), cfg(value_dim=0), cfg(page_size=0), cfg(rope=3), cfg(rope=-1),
               cfg(norm=2), cfg(norm_eps=0.0), cfg(norm_eps=NAN), cfg(scale=0.0), cfg(scale=-1.0), cfg(scale=INF), cfg(causal=2)]
    shapes = [cfg(1025), cfg(rank=256), cfg(rope_dim=32), cfg(key_dim=64), cfg(value_dim=64), cfg(page_size=8), cfg(page_size=48),
              cfg(page_size=512)]
    return [(c, EINVAL) for c in invalid] + [(c, ESHAPE) for c in shapes]


def write(k3, lc=None, T=4, c=A, cs=576, gain=A, pos=A, freq=A, rows=B, rs=576, cache=C, n_pages=4, slots=A, q=A, qs=1536, qh=192, o=A, os=1536,
          oh=192, ws=A, wb=BIG):
    lc = lc or k3.k3moe_latent_config(8)
    return k3.lib().k3moe_latent_write(ctypes.byref(lc), T, vp(c), cs, vp(gain), vp(pos), vp(freq), vp(rows), rs, vp(cache), n_pages, vp(slots),
                                       vp(q), qs, qh, vp(o), os, oh, vp(ws), wb, None)


def test_latent_write_refusals(k3):
    for lc, want in latent_configs(k3):
        assert k3.k3moe_latent_validate_config(lc) == want and write(k3, lc) == want
        with pytest.raises(k3.K3MoEError):
            k3.k3moe_latent_workspace_bytes(lc, 1, 1)
    assert k3.k3moe_latent_validate_config(k3.k3moe_latent_config(8, norm=0, norm_eps=0.0)) == OK
    assert write(k3, T=-1) == write(k3, T=(1 << 20) + 1) == ESHAPE
    for name in ("c", "gain", "pos", "freq", "slots", "cache", "q", "o"):
        assert write(k3, **{name: 0}) == EINVAL
    assert write(k3, rows=0, cache=0, slots=0, q=0, o=0) == EINVAL     # nothing to write to
    assert write(k3, cs=568) == write(k3, cs=580) == write(k3, rs=568) == write(k3, rs=1 << 40) == write(k3, n_pages=0) == ESHAPE
    assert write(k3, qs=1400) == write(k3, qh=56) == write(k3, qh=196) == write(k3, os=1404) == write(k3, oh=60) == ESHAPE
    assert write(k3, rows=A, rs=584) == write(k3, os=1544) == write(k3, oh=184) == EINVAL   # c, q themselves, with other strides
    for name, by in (("c", 8), ("gain", 8), ("pos", 2), ("freq", 4), ("rows", 8), ("cache", 8), ("slots", 4), ("q", 8), ("o", 8)):
        assert write(k3, **{name: C + by}) == EALIGN
    assert write(k3, ws=0) == write(k3, ws=A + 8) == write(k3, wb=256) == EWORKSPACE
    assert write(k3, T=0, c=0, ws=0) == OK


def attend(k3, lc=None, n=3, T=10, start=A, q=A, qs=4608, qh=576, cache=C, n_pages=4, pages=A, max_pages=2, lens=A, out=B, lse=A, ws=A, wb=BIG):
    lc = lc or k3.k3moe_latent_config(8)
    return k3.lib().k3moe_latent_attend(ctypes.byref(lc), n, T, vp(start), vp(q), qs, qh, vp(cache), n_pages, vp(pages), max_pages, vp(lens),
                                        vp(out), vp(lse), vp(ws), wb, None)


def test_latent_attend_refusals(k3):
    for lc, want in latent_configs(k3):
        assert attend(k3, lc) == want
    assert attend(k3, n=-1) == attend(k3, T=-1) == attend(k3, n=(1 << 16) + 1) == attend(k3, T=(1 << 20) + 1) == ESHAPE
    assert attend(k3, n=0) == ESHAPE and attend(k3, n=0, T=0) == OK and attend(k3, T=0, q=0, ws=0) == OK
    assert attend(k3, start=0) == EINVAL                              # 3 sequences, 10 tokens, no offsets
    for name in ("q", "cache", "pages", "lens", "out"):
        assert attend(k3, **{name: 0}) == EINVAL
    assert attend(k3, qs=4600) == attend(k3, qs=4612) == attend(k3, qh=568) == attend(k3, qh=584) == attend(k3, qs=1 << 40) == ESHAPE
    assert attend(k3, n_pages=0) == attend(k3, max_pages=0) == attend(k3, n_pages=1 << 25) == attend(k3, max_pages=1 << 25) == ESHAPE
    for name, by in (("q", 8), ("cache", 8), ("out", 8), ("start", 2), ("pages", 2), ("lens", 2), ("lse", 2)):
        assert attend(k3, **{name: C + by}) == EALIGN
    need = k3.k3moe_latent_workspace_bytes(k3.k3moe_latent_config(8), 3, 10)
    assert attend(k3, ws=0) == attend(k3, ws=A + 8) == attend(k3, wb=need - 1) == EWORKSPACE


def prompt(k3, lc=None, n=3, T=10, S=12, start=A, kstart=A, q=A, qs=1536, qh=192, kv=C, ks=2048, kh=256, rope=A, rs=576, out=B, lse=A, ws=A,
           wb=BIG):
    lc = lc or k3.k3moe_latent_config(8)
    return k3.lib().k3moe_latent_prompt(ctypes.byref(lc), n, T, S, vp(start), vp(kstart), vp(q), qs, qh, vp(kv), ks, kh, vp(rope), rs, vp(out),
                                        vp(lse), vp(ws), wb, None)


def test_latent_prompt_refusals(k3):
    for lc, want in latent_configs(k3):
        assert prompt(k3, lc) == want
    assert prompt(k3, n=-1) == prompt(k3, T=-1) == prompt(k3, S=-1) == prompt(k3, n=(1 << 16) + 1) == prompt(k3, T=(1 << 20) + 1) == ESHAPE
    assert prompt(k3, S=(1 << 20) + 1) == prompt(k3, n=0) == ESHAPE and prompt(k3, n=0, T=0) == prompt(k3, T=0, q=0, ws=0) == OK
    assert prompt(k3, start=0) == prompt(k3, kstart=0) == prompt(k3, n=1, kstart=0) == EINVAL
    for name in ("q", "kv", "rope", "out"):
        assert prompt(k3, **{name: 0}) == EINVAL
    assert prompt(k3, qs=1528) == prompt(k3, qs=1540) == prompt(k3, qh=184) == prompt(k3, qh=200) == ESHAPE
    assert prompt(k3, ks=2040) == prompt(k3, kh=248) == prompt(k3, kh=260, ks=8192) == prompt(k3, rs=56) == prompt(k3, rs=68) == ESHAPE
    for name, by in (("q", 8), ("kv", 8), ("rope", 8), ("out", 8), ("start", 2), ("kstart", 2), ("lse", 2)):
        assert prompt(k3, **{name: C + by}) == EALIGN
    need = k3.k3moe_latent_workspace_bytes(k3.k3moe_latent_config(8), 3, 10)
    assert prompt(k3, ws=0) == prompt(k3, ws=A + 8) == prompt(k3, wb=need - 1) == EWORKSPACE


def test_calls_by_words(k3):
    """The same entries with their arguments as 64-bit words: the same statuses, and refusals of what the words cannot be."""
    call = k3.lib().k3moe_call
    words = lambda *w: ctypes.c_char_p(struct.pack(f"{len(w)}q", *w))  # noqa: E731
    nc, lc = k3.k3moe_norm_config(256), k3.k3moe_latent_config(8)
    at, la = ctypes.addressof(nc), ctypes.addressof(lc)
    args = [at, 0, A, 256, 0, 256, A, C, 256, A, C + 4096, 256, A, C + 8192, 256, 0]
    assert call(words(0, 16, *args)) == OK                 # no rows
    assert call(words(0, 16, 0, *args[1:])) == EINVAL      # no config
    assert call(words(0, 16, at, 4, A + 2, *args[3:])) == EALIGN
    assert call(words(0, 15, *args)) == EINVAL
    assert call(words(0, 17, *args, 0)) == EINVAL
    for entry in (-1, 5, 1 << 32):
        assert call(words(entry, 16, *args)) == EINVAL
    assert call(None) == EINVAL
    for T in (1 << 31, 1 << 32, -(1 << 31) - 1, (1 << 32) + 1):     # would be another number in 32 bits
        assert call(words(0, 16, at, T, *args[2:])) == ESHAPE
    hc = k3.k3moe_head_linear_config(8, 512, 128)
    args = [ctypes.addressof(hc), 0, A, 1024, 128, A, B, 4096, 512, A, BIG, 0]
    assert call(words(1, 12, *args)) == OK
    args[1], args[10] = 4, 0
    assert call(words(1, 12, *args)) == EWORKSPACE
    args[10] = -1                                          # no size
    assert call(words(1, 12, *args)) == ESHAPE
    args = [la, 0, A, 576, A, A, A, B, 576, C, 4, A, A, 1536, 192, A, 1536, 192, A, BIG, 0]
    assert call(words(2, 21, *args)) == OK
    assert call(words(2, 21, la, 4, A, 575, *args[4:])) == ESHAPE
    args = [la, 3, 0, A, A, 4608, 576, C, 4, A, 2, A, B, A, A, BIG, 0]
    assert call(words(3, 17, *args)) == OK
    assert call(words(3, 17, la, 3, 10, A, 0, *args[5:])) == EINVAL
    args = [la, 3, 0, 12, A, A, A, 1536, 192, C, 2048, 256, A, 576, B, A, A, BIG, 0]
    assert call(words(4, 19, *args)) == OK
    assert call(words(4, 19, la, 3, 10, -1, *args[4:])) == ESHAPE


def test_latent_workspace_covers_every_smaller_call(k3):
    for H in (1, 8, 56, 200):
        size = lambda n, T: k3.k3moe_latent_workspace_bytes(k3.k3moe_latent_config(H), n, T)  # noqa: E731,B023
        grid = [(n, T) for n in (0, 1, 2, 7, 40, 300) for T in (0, 1, 3, 64, 300, 5000)]
        for n, T in grid:
            for m, U in grid:
                if m <= n and U <= T:
                    assert size(m, U) <= size(n, T), (H, m, U, n, T)
    for bad in ((-1, 4), (4, -1), ((1 << 16) + 1, 4), (1, (1 << 20) + 1)):
        with pytest.raises(k3.K3MoEError):
            k3.k3moe_latent_workspace_bytes(k3.k3moe_latent_config(8), *bad)
    with pytest.raises(k3.K3MoEError):
        k3.k3moe_head_linear_workspace_bytes(k3.k3moe_head_linear_config(8, 8, 8), -1)


def refuses(call, good, bad):
    for name, value in bad:
        with pytest.raises(ValueError):
            call(**{**good, name: value})


def test_holders_refuse_what_does_not_fit(k3):
    """The holders check what a pointer cannot say: types, shapes, strides, devices."""
    torch = pytest.importorskip("torch")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    op = k3.Norm(k3.k3moe_norm_config(256, gate="silu"), device="cpu")
    op.post_gain, op.pre_gain = torch.ones(256), torch.ones(256)
    good = dict(x=bf(4, 256), out=bf(4, 256), gate=bf(4, 256), residual=bf(4, 256), total=bf(4, 256))
    refuses(op, good, [("x", torch.zeros(4, 256)), ("out", bf(5, 256)), ("gate", bf(256, 4).t()), ("residual", torch.zeros(4, 256)),
                       ("total", bf(4, 248)), ("x", bf(4, 512)[:, ::2])])
    op.pre_gain = torch.ones(128)
    refuses(op, good, [("x", good["x"])])
    op = k3.HeadLinear(k3.k3moe_head_linear_config(8, 64, 128), 4, device="cpu")
    op.w = bf(8, 64, 128)
    good = dict(x=bf(4, 8, 128), y=bf(4, 8, 64))
    refuses(op, good, [("x", bf(5, 8, 128)), ("x", bf(4, 8, 64)), ("x", torch.zeros(4, 8, 128)), ("y", bf(4, 64, 8).transpose(1, 2))])
    op.w = bf(8, 128, 64)
    refuses(op, good, [("x", good["x"])])
    op = k3.LatentAttention(k3.k3moe_latent_config(8), 3, 10, device="cpu")
    op.gain, op.inv_freq = torch.ones(512), torch.ones(32, dtype=torch.float64)
    cache = op.new_cache(4)
    assert tuple(cache.shape) == (4, 64, 576) and not cache.any()
    good = dict(c=bf(10, 576), positions=i32(10), cache=cache, slots=torch.zeros(10, dtype=torch.int64), rows=bf(10, 576), q=bf(10, 8, 64),
                q_rope=bf(10, 8, 64))
    refuses(op.write, good, [("c", bf(11, 576)), ("c", bf(10, 512)), ("positions", i32(9)), ("positions", torch.zeros(10)),
                             ("cache", cache[..., :512]), ("slots", i32(10)), ("rows", torch.zeros(10, 576)), ("q", bf(10, 4, 64)),
                             ("q_rope", bf(10, 64, 8).transpose(1, 2))])
    op.inv_freq = torch.ones(32)
    refuses(op.write, good, [("c", good["c"])])
    good = dict(q=bf(10, 8, 576), cache=cache, pages=i32(3, 2), kv_len=i32(3), out=bf(10, 8, 512), seq_start=i32(4), lse=torch.zeros(10, 8))
    refuses(op.attend, good, [("q", bf(11, 8, 576)), ("q", bf(10, 8, 512)), ("cache", cache[:, :32]), ("pages", i32(2, 3).t()), ("pages", i32(2, 2)),
                              ("kv_len", i32(4)), ("out", bf(10, 8, 576)[..., :512]), ("seq_start", i32(3)), ("lse", torch.zeros(8, 10).t()),
                              ("lse", bf(10, 8))])
    good = dict(q=bf(10, 8, 192), kv=bf(12, 8, 256), rope_key=bf(12, 64), out=bf(10, 8, 128), seq_start=i32(4), kv_start=i32(4),
                lse=torch.zeros(10, 8))
    refuses(op.prompt, good, [("q", bf(10, 8, 128)), ("kv", bf(12, 4, 256)), ("rope_key", bf(10, 64)), ("rope_key", torch.zeros(12, 64)),
                              ("out", bf(10, 8, 256)[..., :128]), ("seq_start", i32(5)), ("kv_start", i32(3)), ("lse", torch.zeros(10, 8, 1))])
