"""A decoder layer from the library's operators: the token mixer's projections and the gated
delta rule, then the routed experts, each on the residual stream.

    q, k, v = silu(x Wqkv^T)      g = logsigmoid(x Wg^T + bg)      b = sigmoid(x Wb^T)
    o = delta rule of (q, k, v, g, b) on each sequence's state
    x <- x + o Wo^T               x <- x + MoE(x)

Run it for a prompt batch followed by single-token steps, the steps as one CUDA graph:

    python examples/decoder_layer.py

The weights are random; the normalisations that a model has before each half are left out.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_moe_expert_k3moe_gb300 as k3  # noqa: E402


class DecoderLayer:
    """One layer for up to n_seq sequences and T_max tokens a call; sequence i keeps its state
    in slot i of `state`."""

    def __init__(self, d, heads, qk_heads, moe_cfg, n_seq, T_max, device="cuda"):
        self.heads, self.qk_heads, self.D = heads, qk_heads, 128
        D, dev = self.D, device
        self.qkv = k3.Linear(k3.k3moe_linear_config((2 * qk_heads + heads) * D, d, "silu"), T_max, dev)
        self.gate = k3.Linear(k3.k3moe_linear_config(heads * D, d, "logsigmoid", y_f32=True), T_max, dev)
        self.beta = k3.Linear(k3.k3moe_linear_config(heads, d, "sigmoid", y_f32=True), T_max, dev)
        self.mix = k3.DeltaRule(k3.k3moe_delta_config(heads, qk_heads, gate_dim=D), n_seq, T_max, dev)
        self.proj = k3.Linear(k3.k3moe_linear_config(d, heads * D), T_max, dev)
        self.moe = k3.MoELayer(moe_cfg, T_max, dev)
        self.state = self.mix.new_state(n_seq)
        new = lambda n, dtype: torch.empty((T_max, n), dtype=dtype, device=dev)  # noqa: E731
        self._qkv, self._o = new(self.qkv.lc.n, torch.bfloat16), new(heads * D, torch.bfloat16)
        self._g, self._b = new(heads * D, torch.float32), new(heads, torch.float32)
        self._y = new(d, torch.float32)

    def randomise(self, seed=0):
        gn = torch.Generator("cpu").manual_seed(seed)
        dev = self.state.device
        w = lambda *s: (torch.randn(*s, generator=gn) / s[-1] ** 0.5).bfloat16().to(dev)  # noqa: E731
        for op in (self.qkv, self.gate, self.beta, self.proj):
            op.w = w(op.lc.n, op.lc.k)
        self.gate.bias = 4.0 + torch.rand(self.gate.lc.n, generator=gn).to(dev)      # slow decays
        c, m = self.moe.cfg, self.moe
        codes = lambda *s: torch.randint(0, 256, s, generator=gn, dtype=torch.uint8).to(dev)  # noqa: E731
        scale = lambda *s: torch.full(s, 121, dtype=torch.uint8, device=dev)         # 2^-6  # noqa: E731
        E, d, f = c.n_experts, c.d, c.f
        m.pack_experts(0, E, codes(E, f, d // 2), scale(E, f, d // 32), codes(E, f, d // 2), scale(E, f, d // 32),
                       codes(E, d, f // 2), scale(E, d, f // 32))
        m.w_router = w(E, d)
        if c.n_shared:
            m.sh_w1, m.sh_w3, m.sh_w2 = w(c.n_shared, f, d), w(c.n_shared, f, d), w(c.n_shared, d, f)
        return self

    def __call__(self, x, seq_start=None):
        """x [T][d] bf16, changed in place; seq_start [n_seq+1] int32, or None for one token of
        each sequence."""
        T, D, H, Hq = x.shape[0], self.D, self.heads, self.qk_heads
        qkv = self.qkv(x, self._qkv[:T])
        q = qkv[:, :Hq * D].view(T, Hq, D)
        k = qkv[:, Hq * D:2 * Hq * D].view(T, Hq, D)
        v = qkv[:, 2 * Hq * D:].view(T, H, D)
        g = self.gate(x, self._g[:T]).view(T, H, D)
        o = self._o[:T]
        self.mix(q, k, v, g, self.beta(x, self._b[:T]), o.view(T, H, D), self.state, self.state, seq_start=seq_start)
        self.proj(o, x, residual=x)
        x += self.moe(x, self._y[:T])
        return x

    def capture(self, x):
        """One step (a token of each sequence) on the fixed buffer x as a CUDA graph.  The step
        that warms up is taken back: the states are as before."""
        kept, kept_x = self.state.clone(), x.clone()
        side = torch.cuda.Stream(device=x.device)
        side.wait_stream(torch.cuda.current_stream(x.device))
        with torch.cuda.stream(side):
            self(x)
        torch.cuda.current_stream(x.device).wait_stream(side)
        self.state.copy_(kept)
        x.copy_(kept_x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self(x)
        return graph


def main():
    d, heads, qk_heads, lens, steps = 3584, 32, 16, [1500, 37, 700, 64], 32
    cfg = k3.k3moe_config(d=d, f=1024, n_experts=64, top_k=8, n_shared=1)
    layer = DecoderLayer(d, heads, qk_heads, cfg, len(lens), sum(lens)).randomise()
    x = torch.randn(sum(lens), d, device="cuda").bfloat16()
    start = torch.tensor([0, *torch.tensor(lens).cumsum(0)], dtype=torch.int32, device="cuda")
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    layer(x.clone(), start)
    layer.state.zero_()
    t0.record()
    y = layer(x, start)
    t1.record()
    torch.cuda.synchronize()
    print(f"prompts of {lens} tokens: {t0.elapsed_time(t1) * 1e3:.0f} us")
    token = y[start[1:].long() - 1].contiguous()                      # each sequence's last row goes on
    graph = layer.capture(token)
    graph.replay()
    t0.record()
    for _ in range(steps):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    print(f"{steps} steps of {len(lens)} tokens: {t0.elapsed_time(t1) / steps * 1e3:.1f} us a step")
    for op in (layer.qkv, layer.gate, layer.beta, layer.proj, layer.mix, layer.moe):
        assert k3.k3moe_device_status(op.ws) == (0, 0)


if __name__ == "__main__":
    main()
