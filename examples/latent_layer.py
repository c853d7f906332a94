"""A latent-attention decoder layer from the library's operators, then the routed experts, each on the
residual stream:

    h = norm(x)       q = h Wq^T       [c, r] = h Wc^T       z = h Wz^T
    row = [norm(c), rotate(r)] into the sequence's pages, q's last columns rotated
    prompts:  k, v = row's c Wkv^T;  o = softmax(q . [k, r]) v
    steps:    o = Wv (softmax([Wk^T q, q_r] . rows) rows' c), over the pages
    x <- x + scale * norm(o Wo^T) * sigmoid(z),   h = norm(x),   x <- x + MoE(h)

Run it for a prompt batch followed by single-token steps, the steps as one CUDA graph:

    python examples/latent_layer.py

The weights are random.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_moe_expert_k3moe_gb300 as k3  # noqa: E402

C, R, K, V = 512, 64, 128, 128                                # latent, rotated part, a head's keys and values


class LatentLayer:
    """One layer for up to n_seq sequences of up to max_len tokens, T_max tokens a call."""

    def __init__(self, d, heads, moe_cfg, n_seq, max_len, T_max, page_size=64, device="cuda"):
        dev, H = device, heads
        self.heads, self.page, self.n_seq = H, page_size, n_seq
        lin = lambda n, k: k3.Linear(k3.k3moe_linear_config(n, k), T_max, dev)  # noqa: E731
        self.q, self.c, self.z, self.o = lin(H * (K + R), d), lin(C + R, d), lin(d, d), lin(d, H * V)
        self.kv = lin(H * (K + V), C)
        self.absorb = k3.HeadLinear(k3.k3moe_head_linear_config(H, C, K), T_max, dev)
        self.value = k3.HeadLinear(k3.k3moe_head_linear_config(H, V, C), T_max, dev)
        self.attn = k3.LatentAttention(k3.k3moe_latent_config(H, page_size=page_size, rope="pairs"), n_seq, T_max, dev)
        self.before = k3.Norm(k3.k3moe_norm_config(d, post_norm=0), dev)
        self.between = k3.Norm(k3.k3moe_norm_config(d, gate="sigmoid"), dev)
        self.moe = k3.MoELayer(moe_cfg, T_max, dev)
        each = -(-max_len // page_size)
        self.cache = self.attn.new_cache(n_seq * each)
        # any order will do: here the sequences' pages take turns
        self.pages = torch.arange(n_seq * each, dtype=torch.int32, device=dev).view(each, n_seq).t().contiguous()
        self.lens = torch.zeros(n_seq, dtype=torch.int32, device=dev)
        self._every = torch.arange(n_seq, device=dev)
        new = lambda *s, dtype=torch.bfloat16: torch.empty((T_max, *s), dtype=dtype, device=dev)  # noqa: E731
        self._h, self._z, self._y, self._c = new(d), new(d), new(d), new(C + R)
        self._q, self._qa, self._kv = new(H, K + R), new(H, C + R), new(H, K + V)
        self._lat, self._o, self._moe = new(H, C), new(H, V), new(d, dtype=torch.float32)

    def randomise(self, seed=0):
        gn = torch.Generator("cpu").manual_seed(seed)
        dev = self.cache.device
        w = lambda *s: (torch.randn(*s, generator=gn) / s[-1] ** 0.5).bfloat16().to(dev)  # noqa: E731
        for op in (self.q, self.c, self.z, self.o):
            op.w = w(op.lc.n, op.lc.k)
        up = w(self.heads, K + V, C)                          # one matrix, as it is and a head at a time
        self.kv.w = up.view(-1, C)
        self.absorb.w, self.value.w = up[:, :K].transpose(1, 2).contiguous(), up[:, K:].contiguous()
        d = self.o.lc.n
        gain = lambda n: 1 + 0.1 * torch.randn(n, generator=gn).to(dev)  # noqa: E731
        self.attn.gain, self.before.pre_gain, self.between.post_gain, self.between.pre_gain = gain(C), gain(d), gain(d), gain(d)
        self.between.scale = 0.5 * gain(d)
        self.attn.inv_freq = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device=dev) * 2 / R)
        c, m = self.moe.cfg, self.moe
        codes = lambda *s: torch.randint(0, 256, s, generator=gn, dtype=torch.uint8).to(dev)  # noqa: E731
        scale = lambda *s: torch.full(s, 121, dtype=torch.uint8, device=dev)         # 2^-6  # noqa: E731
        E, f = c.n_experts, c.f
        m.pack_experts(0, E, codes(E, f, d // 2), scale(E, f, d // 32), codes(E, f, d // 2), scale(E, f, d // 32),
                       codes(E, d, f // 2), scale(E, d, f // 32))
        m.w_router = w(E, d)
        if c.n_shared:
            m.sh_w1, m.sh_w3, m.sh_w2 = w(c.n_shared, f, d), w(c.n_shared, f, d), w(c.n_shared, d, f)
        return self

    def _half(self, x, attend):
        """x [T][d] bf16, changed in place, around attend(q [T][H][..], rows' input c) -> o [T][H][V]."""
        T = x.shape[0]
        h = self.before(x, out=self._h[:T])
        q = self.q(h, self._q[:T].view(T, -1)).view(T, self.heads, K + R)
        o = attend(q, self.c(h, self._c[:T]))
        y, z = self.o(o.view(T, -1), self._y[:T]), self.z(h, self._z[:T])
        self.between(y, out=self._h[:T], gate=z, residual=x, total=x)
        x += self.moe(self._h[:T], self._moe[:T])
        return x

    def _slots(self, sequences, positions):
        """The rows of the cache for tokens of these sequences at these positions.  -1, which writes nothing, for one that no page holds:
        a captured step may be replayed once too often, and an index out of range ends the process."""
        page = torch.div(positions, self.page, rounding_mode="floor").long()
        held = (page >= 0) & (page < self.pages.shape[1]) & (sequences >= 0) & (sequences < self.n_seq)
        rows = self.pages[torch.where(held, sequences, 0), torch.where(held, page, 0)].long() * self.page + positions % self.page
        return torch.where(held, rows, -1)

    def prompt(self, x, seq_start, positions, sequences):
        """Prompts of all sequences, from position 0 on: x [T][d]; positions, sequences [T] of each token."""
        slots = self._slots(sequences, positions)

        def attend(q, c):
            T = q.shape[0]
            self.attn.write(c, positions, cache=self.cache, slots=slots, rows=c, q=q[..., K:], q_rope=q[..., K:])
            kv = self.kv(c[:, :C], self._kv[:T].view(T, -1)).view(T, self.heads, K + V)
            return self.attn.prompt(q, kv, c[:, C:], self._o[:T], seq_start=seq_start)

        self.lens.copy_(seq_start[1:] - seq_start[:-1])
        return self._half(x, attend)

    def step(self, x):
        """One token of each sequence: x [n_seq][d].  A sequence whose pages are full is left out, and
        k3moe_device_status(attn.ws) says so."""
        positions = self.lens.clone()
        slots = self._slots(self._every, positions)
        self.lens += 1

        def attend(q, c):
            T = q.shape[0]
            qa = self._qa[:T]
            self.attn.write(c, positions, cache=self.cache, slots=slots, q=q[..., K:], q_rope=qa[..., C:])
            self.absorb(q[..., :K], qa[..., :C])
            return self.value(self.attn.attend(qa, self.cache, self.pages, self.lens, self._lat[:T]), self._o[:T])

        return self._half(x, attend)

    def capture(self, x):
        """One step on the fixed buffer x as a CUDA graph.  The step that warms up is taken back: the row it wrote is
        written again before it is read."""
        kept, kept_x = self.lens.clone(), x.clone()
        side = torch.cuda.Stream(device=x.device)
        side.wait_stream(torch.cuda.current_stream(x.device))
        with torch.cuda.stream(side):
            self.step(x)
        torch.cuda.current_stream(x.device).wait_stream(side)
        self.lens.copy_(kept)
        x.copy_(kept_x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(x)
        return graph


def places(lens, device="cuda"):
    """(seq_start, positions, sequences) of packed sequences."""
    start = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32, device=device)
    positions = torch.cat([torch.arange(n) for n in lens]).int().to(device)
    return start, positions, torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).to(device)


def main():
    d, heads, lens, steps = 3584, 56, [1500, 37, 700, 64], 32
    cfg = k3.k3moe_config(d=d, f=1024, n_experts=64, top_k=8, n_shared=1)
    layer = LatentLayer(d, heads, cfg, len(lens), max(lens) + steps + 1, sum(lens)).randomise()
    x = torch.randn(sum(lens), d, device="cuda").bfloat16()
    at = places(lens)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    layer.prompt(x.clone(), *at)
    t0.record()
    y = layer.prompt(x, *at)
    t1.record()
    torch.cuda.synchronize()
    print(f"prompts of {lens} tokens: {t0.elapsed_time(t1) * 1e3:.0f} us")
    token = y[at[0][1:].long() - 1].contiguous()                      # each sequence's last row goes on
    graph = layer.capture(token)
    graph.replay()
    t0.record()
    for _ in range(steps - 1):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    print(f"{steps} steps of {len(lens)} tokens: {t0.elapsed_time(t1) / (steps - 1) * 1e3:.1f} us a step")
    for op in (layer.q, layer.c, layer.z, layer.o, layer.kv, layer.absorb, layer.value, layer.attn, layer.moe):
        assert k3.k3moe_device_status(op.ws) == (0, 0)


if __name__ == "__main__":
    main()
