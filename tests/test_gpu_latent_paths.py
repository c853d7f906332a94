"""The latent attention's operators on the paths that go by the number of blocks: query blocks sorted by their length, several
whole ones on an SM, the head projection's ring used over; captured calls that replay on other lengths; and rows
whose scores leave nothing.  Definitions, tolerances and inputs are those of test_gpu_latent.py."""
import itertools

import pytest

from test_gpu_latent import C, K, R, ROW, Cached, Expanded, attention64, check_attention, k3, randn, within  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ----------------------------------------------------------------------------- scores that leave nothing

LOWEST = -3.3895313892515355e38                                # bf16's


@pytest.mark.parametrize("value", [-float("inf"), LOWEST])
@pytest.mark.parametrize("masked,more,other", [(1, 300, 700), (64, 3, 700), (200, 300, 700), (130, 20000, 700), (64, 3, 60), (130, 100, 60), (200, 150, 60)])
def test_attend_first_rows_of_no_weight(k3, masked, more, other, value):
    """A sequence's first rows hold minus infinity, or the lowest value, in a rotated column and finite values in c: their scores are
    minus infinity (4 times the lowest passes float's), their weights zero, and the rows behind them, whose scores are
    about -173, have all the weight; with a short other sequence one SM has all of them."""
    c = Cached([1, 2], [masked + more, other], 16, 64, masked + more)
    c.q[..., C] = 4
    rows = c.rows[0]
    rows[:masked, C], rows[masked:, C] = value, -600
    at = torch.arange(masked + more, device="cuda")
    c.cache[c.pages[0].long()[at // 64], at % 64] = rows
    op, cfg = c.holder(k3)
    c(op)
    k = rows[masked:, None]
    check_attention(c.out[:1], c.lse[:1], attention64(c.q[:1], k, k[..., :C], cfg.scale, 1), "masked")
    c.check(cfg, skip=[0])
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("value", [-float("inf"), LOWEST])
@pytest.mark.parametrize("masked,more", [(1, 300), (128, 40), (200, 300), (130, 6000)])
def test_prompt_first_keys_of_no_weight(k3, masked, more, value):
    c = Expanded([40, 30], [masked + more, 30], 2, False, masked + more)
    c.q[..., K] = 4
    c.rope[:masked, 0], c.rope[masked:masked + more, 0] = value, -600
    op, cfg = c.holder(k3)
    c(op)
    kv = c.kv[masked:masked + more]
    k = torch.cat([kv[..., :K], c.rope[masked:masked + more, None].expand(-1, 2, -1)], -1)
    check_attention(c.out[:40], c.lse[:40], attention64(c.q[:40], k, kv[..., K:], cfg.scale, 1), "masked")
    c.check(cfg, skip=[0])
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- holders

def test_holder_made_on_a_busy_stream(k3):
    """A holder serves every stream from the first call on, whatever the stream it was made on is still busy with: what
    the call reports stays reported."""
    c = Cached([1], [100], 8, 64, 61)
    c.pages[0, 1] = -1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                         # about a tenth of a second
    op, cfg = c.holder(k3)
    c(op, stream=side)
    torch.cuda.synchronize()
    assert k3.k3moe_device_status(op.ws) == (6, 0x1)
    c.rows[0][64:] = 0                                      # the page reads as zeros
    c.check(cfg)


# ----------------------------------------------------------------------------- absorbed

@pytest.mark.parametrize("width,lens", [
    (330, ([500, 64, 3, 0], [3, 20000, 65, 700], [20000, 0, 1, 64], [9000, 9001, 63, 1], [1, 2, 3, 4])),        # cut, and joined
    (4, ([200, 64, 3, 0], [0, 129, 256, 255], [1, 2, 3, 4]))])                                                   # whole
def test_attend_captured_follows(k3, width, lens):
    """One captured call replays on other lengths, pages, queries and offsets: other cuts, other blocks to join."""
    queries = [[1, 0, 2, 1], [2, 1, 1, 0], [0, 0, 4, 0], [1, 1, 1, 1], [0, 3, 0, 1]]
    first = Cached(queries[0], lens[0], 56, 64, 91)
    op, cfg = first.holder(k3)
    room = 400
    cache = torch.zeros(room, 64, ROW, dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros(4, width, dtype=torch.int32, device="cuda")
    q, start, kv_len = torch.zeros_like(first.q), torch.zeros_like(first.start), torch.zeros_like(first.kv_len)
    out, lse = torch.empty_like(first.out), torch.empty_like(first.lse)

    def put(d):
        assert d.n_pages <= room and d.pages.shape[1] - 1 <= width and d.T == 4
        cache.fill_(float("nan"))
        cache[:d.n_pages].copy_(d.cache)
        pages.fill_(-1)
        w = min(width, d.pages.shape[1])                   # the last column of theirs is no page
        pages[:, :w].copy_(d.pages[:, :w])
        for mine, other in ((q, d.q), (start, d.start), (kv_len, d.kv_len)):
            mine.copy_(other)
        out.fill_(7.5)
        lse.fill_(7.5)

    put(first)
    graph = k3._capture(lambda x, y: op.attend(x, cache, pages, kv_len, y, seq_start=start, lse=lse), q, out)
    for i in [*range(len(lens)), 0]:
        d = Cached(queries[i], lens[i], 56, 64, 91 + i)
        put(d)
        graph.replay()
        d.out, d.lse = out, lse
        d.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("n,H,longest", [(96, 128, 192), (200, 128, 120), (130, 100, 64)])
def test_attend_whole_blocks_in_turn(k3, n, H, longest):
    """Short tables and more query blocks of 64 than SMs, none cut: an SM has several, one after the other."""
    queries = [(1, 1, 2, 0, 3)[i % 5] for i in range(n)]
    lens = [(37 * i) % (longest + 1) if i else longest for i in range(n)]
    c = Cached(queries, lens, H, 64, n + H)
    blocks, tiles = -(-c.T * H // 64), c.pages.shape[1]
    assert blocks > sms() and tiles * (-(-blocks // sms()) - 0.5 * blocks / sms()) <= 6.5
    op, cfg = c.holder(k3)
    c(op)
    c.check(cfg)
    out, lse = c.out.clone(), c.lse.clone()
    c(op)
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("lens", [[300, 20000, 5, 700], [60, 130, 5, 100]])
def test_attend_leaves_other_rows(k3, lens):
    """Tokens before the first sequence and behind the last stay as they are, whatever their queries hold."""
    c = Cached([3, 2, 4, 5], lens, 16, 64, 63)
    op, cfg = c.holder(k3)
    c.q[:3], c.q[9:] = float("nan"), float("inf")
    op.attend(c.q, c.cache, c.pages[1:3].contiguous(), c.kv_len[1:3].contiguous(), c.out, seq_start=c.start[1:4].contiguous(), lse=c.lse)
    assert (c.out[:3] == 7.5).all() and (c.out[9:] == 7.5).all() and (c.lse[:3] == 7.5).all() and (c.lse[9:] == 7.5).all()
    c.check(cfg, skip=[0, 3])
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- expanded, sorted

RAGGED = [429, 1, 700, 429, 0, 942, 500], [429, 101, 900, 929, 50, 1442, 100]     # prefixes, an empty one, more queries than keys
SORTED = [  # queries, keys, heads, causal
    (*RAGGED, 16, 1),
    (*RAGGED, 16, 0),
    ([300] * 8, None, 16, 1),                                  # alike
    ([256] * 8, [256, 0, 600, 256, 256, 0, 600, 1], 16, 1),    # some without keys
    ([1] * 128, [(11 * i) % 140 for i in range(128)], 3, 1),
    ([3] * 127, [(29 * i) % 300 for i in range(127)], 3, 0),
    ([0, 5, 1, 0] * 32, [(7 * i) % 90 for i in range(128)], 3, 1),     # half of the places have no block
    ([2000, 40], [2000, 2000], 17, 1),
    ([5000], None, 8, 1),
]


def in_order(c):
    """Asserts what a call has to have for its query blocks to be sorted."""
    blocks, S = c.T // 256 + min(len(c.queries), c.T), sum(c.keys)
    assert blocks * c.H > sms() and blocks <= 128 and len(c.queries) <= 128 and S * c.H * (K + R + R) * 2 <= 64 << 20


@pytest.mark.parametrize("case", SORTED, ids=lambda c: f"{len(c[0])}-{sum(c[0])}x{c[2]}-{sum(c[1] or c[0])}-{c[3]}")
def test_prompt_sorted(k3, case):
    queries, keys, H, causal = case
    c = Expanded(queries, keys, H, True, sum(queries) + H)
    in_order(c)
    op, cfg = c.holder(k3, causal=causal)
    c(op)
    c.check(cfg)
    out, lse = c.out.clone(), c.lse.clone()
    c(op)
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


@pytest.mark.parametrize("name,at,bad,lost", [("start", 3, -1, [2, 3]), ("start", 7, 3002, [6]), ("kv_start", 1, 1 << 30, [0, 1]), ("kv_start", 6, -7, [5, 6])])
def test_prompt_sorted_reports_what_does_not_fit(k3, name, at, bad, lost):
    c = Expanded(*RAGGED, 16, False, 77)
    in_order(c)
    op, cfg = c.holder(k3)
    getattr(c, name)[at] = bad
    c(op)
    c.check(cfg, skip=lost)
    first = list(itertools.accumulate([0, *c.queries]))
    for i in lost:
        assert (c.out[first[i]:first[i + 1]] == 7.5).all() and (c.lse[first[i]:first[i + 1]] == 7.5).all()
    assert k3.k3moe_device_status(op.ws) == (6, 0x2)


def test_prompt_sorted_captured(k3):
    """A captured call replays on other lengths: another order."""
    c = Expanded(*RAGGED, 16, False, 78)
    op, cfg = c.holder(k3)
    graph = k3._capture(lambda x, out: c(op), c.q, c.out)
    d = Expanded([1, 1500, 0, 300, 300, 899, 1], [700, 1500, 0, 251, 300, 1000, 200], 16, False, 79)
    assert d.T == c.T and sum(d.keys) == sum(c.keys)
    for name in ("q", "kv", "rope", "start", "kv_start"):
        getattr(c, name).copy_(getattr(d, name))
    c.out.fill_(7.5)
    c.lse.fill_(7.5)
    graph.replay()
    c.queries, c.keys = d.queries, d.keys
    c.check(cfg)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- a head's own projection

@pytest.mark.parametrize("T,H,K_,N,xpad,ypad", [
    (333, 56, 512, 128, 64, 64),                               # 176 tokens a block, five places of the ring for eight chunks
    (512, 56, 512, 128, 0, 8),                                 # 256 a block, four places
    (500, 56, 512, 128, 8, 1),                                 # a ragged last tile, y's heads at odd places
    (250, 28, 512, 600, 0, 0),
    (240, 100, 512, 127, 16, 0),
    (600, 56, 512, 128, 0, 0),                                 # more blocks than SMs: three places, two blocks an SM
    (1000, 56, 512, 129, 64, 0),                               # two places
    (1000, 60, 328, 72, 8, 3),
    (4096, 56, 512, 128, 0, 64),
])
def test_head_linear_ring(k3, T, H, K_, N, xpad, ypad):
    """Rings with fewer places than there are chunks of K, and blocks of up to 256 tokens."""
    r = randn(T + H)
    x = r(T, H, K_ + xpad).bfloat16()[..., :K_]
    w = (r(H, N, K_) / K_ ** 0.5).bfloat16()
    op = k3.HeadLinear(k3.k3moe_head_linear_config(H, N, K_), T)
    op.w = w
    wide = torch.full((T, H, N + ypad), 7.5, dtype=torch.bfloat16, device="cuda")
    y = op(x, wide[..., :N])
    for t in range(0, T, 1024):
        a, b = x[t:t + 1024].double(), w.double()
        ref, mag = torch.einsum("thk,hnk->thn", a, b), torch.einsum("thk,hnk->thn", a.abs(), b.abs())
        within(y[t:t + 1024], ref, 4 * K_ ** 0.5 * 2.0 ** -23 * mag)
    assert (wide[..., N:] == 7.5).all()
    for _ in range(2):
        assert torch.equal(op(x, torch.full_like(y, 7.5)), y)
    assert k3.k3moe_device_status(op.ws) == (0, 0)


# ----------------------------------------------------------------------------- large values

@pytest.mark.parametrize("power", [100, -60])
def test_attention_of_large_and_small_values(k3, power):
    """Values 2^power as large have outputs 2^power as large, bit for bit: weights and sums are the same, and nothing overflows within
    the documented bound (2^119 / 2000 rows, 2^97 / 900 keys of values below 8, so 2^80 there) or is lost: products are of
    weights above 2^-30 and values above 2^-90."""
    c = Cached([1, 2], [2000, 70], 16, 64, 5)
    op, _ = c.holder(k3)
    c.q[..., :C] = 0                                       # scores are of the rotated columns alone
    c(op)
    out, lse = c.out.clone(), c.lse.clone()
    c.cache[..., :C] *= 2.0 ** power
    c(op)
    assert torch.equal(c.out.double(), out.double() * 2.0 ** power) and torch.equal(c.lse, lse)
    power = min(power, 80)
    e = Expanded([100, 300], [900, 300], 2, False, 6)
    op, _ = e.holder(k3)
    e(op)
    out, lse = e.out.clone(), e.lse.clone()
    e.kv[..., K:] *= 2.0 ** power
    e(op)
    assert torch.equal(e.out.double(), out.double() * 2.0 ** power) and torch.equal(e.lse, lse)
