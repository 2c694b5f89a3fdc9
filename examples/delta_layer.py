"""A delta-attention layer from the library's operators, in 8 bits where the weights are.

    hidden, residual -> norm (int8) -> packed input projection (int8) -> gated delta rule
                     -> output gate -> row quantisation -> output projection (int8)

The same call takes a decode batch (one token a sequence) and packed prompts of any
lengths; every sequence keeps its state in a slot of a pool.  Run it:

    python examples/delta_layer.py            # a small layer, checked against float64
    python examples/delta_layer.py --full     # 96 heads of 128, 49376 x 7168 and 7168 x 12288, timed
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import skinny_bf16_split_gb300 as dep  # noqa: E402


class DeltaLayer:
    """heads x dim query, key, value and gate channels, a rank-dim decay and a write strength a head:
    (4 * heads * dim + dim + heads) rows of input projection.  heads is a multiple of 8, which keeps the rows
    of the packed projection, and so q, k and v in them, 16-byte aligned."""

    def __init__(self, hidden, heads, dim, slots, max_rows=256, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.heads, self.dim, self.inner = heads, dim, heads * dim
        self.norm_weight = (1 + 0.1 * rnd(hidden)).bfloat16()
        # weights in 8 bits with a scale for each output channel: rows, quantised like any rows
        w_in = (rnd(4 * self.inner + dim + heads, hidden) * hidden ** -0.5).bfloat16()
        w_out = (rnd(hidden, self.inner) * self.inner ** -0.5).bfloat16()
        self.in_proj = dep.Int8Projection(*dep.quantize_rows(w_in), max_rows=max_rows)
        self.out_proj = dep.Int8Projection(*dep.quantize_rows(w_out), max_rows=max_rows)
        self.decay_up = (rnd(self.inner, dim) * dim ** -0.5).bfloat16()
        self.rate = torch.exp(torch.linspace(-2.5, 1.0, heads, device=device))
        self.state = torch.zeros(slots, heads, dim, dim, device=device)

    def forward(self, hidden, residual, slots, cu_seqlens=None):
        """hidden, residual: bfloat16 [tokens, hidden] (residual is updated in place); slots: int32, a
        sequence's place in the pool; cu_seqlens: int32 bounds of the sequences, or None for one token each."""
        T, H, D, I = hidden.shape[0], self.heads, self.dim, self.inner
        x, x_scale = dep.add_rms_norm(hidden, self.norm_weight, residual, quant="int8")
        packed = self.in_proj.run(x, x_scale)
        q, k, v, gate, low, beta = packed.split([I, I, I, I, D, H], 1)
        g = -torch.nn.functional.softplus((low @ self.decay_up.t()).float()).view(T, H, D) * self.rate[:, None]
        o = dep.gated_delta_rule(q.view(T, H, D), k.view(T, H, D), v.view(T, H, D), g, torch.sigmoid(beta.float()),
                                 self.state, cu_seqlens=cu_seqlens, n_seq=slots.shape[0], slots=slots, l2norm=True)
        y, y_scale = dep.quantize_rows(o.view(T, I) * torch.sigmoid(gate))
        return self.out_proj.run(y, y_scale)

    def reference(self, hidden, residual, state, lengths):
        """forward() in float64 but for the stored roundings, token by token; returns (out, states)."""
        H, D, I = self.heads, self.dim, self.inner
        h = (hidden.float() + residual.float()).bfloat16().double()
        p = h * self.norm_weight.double()
        top = p.abs().amax(1, keepdim=True)
        x = torch.round(127 * p / top) * (top / 127 / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt())
        w_in, w_out = (m.weight.double() * m.weight_scale.double()[:, None] for m in (self.in_proj, self.out_proj))
        packed = (x @ w_in.t()).bfloat16()
        q, k, v, gate, low, beta = packed.split([I, I, I, I, D, H], 1)
        a = torch.exp(-torch.nn.functional.softplus((low @ self.decay_up.t()).float()).view(-1, H, D)
                      * self.rate[:, None]).double()
        unit = lambda t: t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
        q, k, v = (t.double().reshape(-1, H, D) for t in (q, k, v))
        q, k, b = unit(q) * D ** -0.5, unit(k), torch.sigmoid(beta.float()).double()
        o, S, t = torch.empty_like(v), state.double().clone(), 0
        for s, n in enumerate(lengths):
            for _ in range(n):
                St = S[s] * a[t][:, None, :]
                u = b[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", St, k[t]))
                S[s] = St + u[:, :, None] * k[t][:, None, :]
                o[t] = torch.einsum("hvk,hk->hv", S[s], q[t])
                t += 1
        y = (o.bfloat16().view(-1, I) * torch.sigmoid(gate)).double()
        top = y.abs().amax(1, keepdim=True)
        return (torch.round(127 * y / top) * (top / 127)) @ w_out.t(), S


def tokens(n, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(n, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))


def check():
    layer = DeltaLayer(256, 8, 64, slots=5)
    lengths, slots = [37, 1, 20], torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 37, 38, 58], dtype=torch.int32, device="cuda")
    x, r = tokens(58, 256, 1)
    want, S = layer.reference(x, r, torch.zeros(3, 8, 64, 64, device="cuda"), lengths)
    out = layer.forward(x, r, slots, cu)  # the prompts
    print("prompts: relative error %.4f" % ((out.double() - want).norm() / want.norm()))
    x, r = tokens(3, 256, 2)
    want, _ = layer.reference(x, r, S, [1, 1, 1])
    out = layer.forward(x, r, slots)  # one more token each
    print("decode:  relative error %.4f" % ((out.double() - want).norm() / want.norm()))


def full():
    layer = DeltaLayer(7168, 96, 128, slots=64)
    for name, n, cu in (("1 token", 1, None), ("64 tokens of 64 users", 64, None), ("a prompt of 1024", 1024, [0, 1024])):
        x, r = tokens(n, 7168, 3)
        slots = torch.arange(n if cu is None else 1, dtype=torch.int32, device="cuda")
        cu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        layer.forward(x, r, slots, cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(x, r, slots, cu)
        graph.replay()
        torch.cuda.synchronize()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / 20 * 1e3:.1f} us a layer, as a CUDA graph")


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--full", action="store_true")
    full() if ap.parse_args().full else check()
