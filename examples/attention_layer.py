"""A softmax-attention layer from the library's operators, in 8 bits where the weights are.

    hidden, residual -> norm (int8) -> packed input projection (int8) -> heads' norm and rotation, keys and
                     values to their pages -> attention over the pages -> gate a head -> row quantisation
                     -> output projection (int8)

The same call takes a decode batch (one token a sequence), packed prompts of any lengths and trees of
drafted tokens.  Run it:

    python examples/attention_layer.py          # a small layer, checked against float64
    python examples/attention_layer.py --full   # 96 heads of 128 over 8, 14560 x 7168 and 7168 x 12288, timed
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import skinny_bf16_split_gb300 as dep  # noqa: E402


class Pages:
    """Which pages of a pool the sequences have, and how long they are (on the host)."""

    def __init__(self, pages, page_size, width):
        self.free, self.page_size, self.width = list(range(pages - 1, -1, -1)), page_size, width
        self.pages, self.length = {}, {}

    def extend(self, new):
        """`new`: {sequence: tokens to add}.  Returns what a layer's call takes of it, on the device: the
        slots of the new tokens, the sequences' page table, lengths and first tokens."""
        slots, table, cu = [], [], [0]
        for s, n in new.items():
            at = self.length.get(s, 0)
            own = self.pages.setdefault(s, [])
            while len(own) * self.page_size < at + n:
                own.append(self.free.pop())
            slots += [own[j // self.page_size] * self.page_size + j % self.page_size for j in range(at, at + n)]
            self.length[s] = at + n
            table.append(own + [-1] * (self.width - len(own)))
            cu.append(cu[-1] + n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"slots": i32(slots), "page_table": i32(table), "kv_lens": i32([self.length[s] for s in new]), "cu_seqlens": i32(cu)}

    def drop(self, s, n):
        """Forget the last n tokens of a sequence (drafts that were not taken)."""
        self.length[s] -= n
        own = self.pages[s]
        while (len(own) - 1) * self.page_size >= self.length[s]:
            self.free.append(own.pop())
            if not own:
                break


class AttentionLayer:
    """heads query heads and kv_heads key and value heads of dim channels, and a gate for each query head:
    (heads + 2 kv_heads) dim + heads rows of input projection, filled up with `spare` more.  heads + spare is a
    multiple of 8, which keeps the rows of the packed projection, and so q, k and v in them, 16-byte aligned."""

    def __init__(self, hidden, heads, kv_heads, dim, pages, page_size, spare=0, max_rows=256, base=5e5, factor=1.0,
                 original=None, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.inner = heads, kv_heads, dim, heads * dim
        self.norm_weight = (1 + 0.1 * rnd(hidden)).bfloat16()
        self.q_weight, self.k_weight = ((1 + 0.1 * rnd(dim)).bfloat16() for _ in range(2))
        w_in = (rnd((heads + 2 * kv_heads) * dim + heads + spare, hidden) * hidden ** -0.5).bfloat16()
        w_out = (rnd(hidden, self.inner) * self.inner ** -0.5).bfloat16()
        self.in_proj = dep.Int8Projection(*dep.quantize_rows(w_in), max_rows=max_rows)
        self.out_proj = dep.Int8Projection(*dep.quantize_rows(w_out), max_rows=max_rows)
        self.freqs, self.amplitude = dep.rotary_freqs(dim, base, factor=factor, original=original, device=device)
        self.k_cache, self.v_cache = (torch.zeros(pages, page_size, kv_heads, dim, device=device, dtype=torch.bfloat16)
                                      for _ in range(2))

    def forward(self, hidden, residual, positions, slots, page_table, kv_lens, cu_seqlens, tree=None):
        """hidden, residual: bfloat16 [tokens, hidden] (residual is updated in place); positions: int32 [tokens];
        the rest as Pages.extend gives it; tree: int64 [tokens], which new tokens of its sequence each sees."""
        T, H, K, D, I = hidden.shape[0], self.heads, self.kv_heads, self.dim, self.inner
        x, x_scale = dep.add_rms_norm(hidden, self.norm_weight, residual, quant="int8")
        packed = self.in_proj.run(x, x_scale)
        q, k, v, gate = packed[:, : I + 2 * K * D + H].split([I, K * D, K * D, H], 1)
        q = dep.append_kv(k.view(T, K, D), v.view(T, K, D), self.k_cache, self.v_cache, slots, positions, self.freqs,
                          amplitude=self.amplitude, norm=True, k_weight=self.k_weight, q=q.view(T, H, D), q_weight=self.q_weight)
        o = dep.paged_attention(q, self.k_cache, self.v_cache, page_table, kv_lens, cu_seqlens=cu_seqlens, tree=tree)
        y, y_scale = dep.quantize_rows((o * torch.sigmoid(gate)[..., None]).view(T, I))
        return self.out_proj.run(y, y_scale)

    def reference(self, hidden, residual, positions, past, lengths, tree=None):
        """forward() in float64 but for the stored roundings; past: each sequence's (keys, values) so far, or
        None.  Returns (out, the sequences' keys and values)."""
        H, K, D, I = self.heads, self.kv_heads, self.dim, self.inner
        h = (hidden.float() + residual.float()).bfloat16().double()
        p = h * self.norm_weight.double()
        top = p.abs().amax(1, keepdim=True)
        x = torch.round(127 * p / top) * (top / 127 / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt())
        w_in, w_out = (m.weight.double() * m.weight_scale.double()[:, None] for m in (self.in_proj, self.out_proj))
        packed = (x @ w_in.t()).bfloat16()
        q, k, v, gate = packed[:, : I + 2 * K * D + H].split([I, K * D, K * D, H], 1)
        u = positions.double()[:, None, None] * self.freqs

        def turned(t, weight):
            t = t.double().reshape(len(t), -1, D)
            t = t / (t.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
            a, b = t.chunk(2, -1)
            return (self.amplitude * torch.cat((a * u.cos() - b * u.sin(), b * u.cos() + a * u.sin()), -1)).bfloat16().double()

        q, k, v = turned(q, self.q_weight), turned(k, self.k_weight), v.double().reshape(-1, K, D)
        o, kept, t = torch.empty_like(q), [], 0
        for s, n in enumerate(lengths):
            keys, values = (new[t: t + n] if past[s] is None else torch.cat((past[s][i], new[t: t + n])) for i, new in enumerate((k, v)))
            own = torch.arange(len(keys), device="cuda") - (len(keys) - n)
            seen = own <= torch.arange(n, device="cuda")[:, None]
            if tree is not None:
                seen = (own < 0) | (tree[t: t + n, None] >> own.clamp(min=0) & 1 == 1)
            for j in range(H):
                w = (q[t: t + n, j] @ keys[:, j * K // H].t() * D ** -0.5).masked_fill(~seen, -torch.inf).softmax(-1)
                o[t: t + n, j] = w @ values[:, j * K // H]
            kept.append((keys, values))
            t += n
        y = (o.bfloat16() * torch.sigmoid(gate)[..., None]).view(-1, I).double()
        top = y.abs().amax(1, keepdim=True)
        return (torch.round(127 * y / top) * (top / 127)) @ w_out.t(), kept


def tokens(n, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(n, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check():
    layer = AttentionLayer(256, 8, 2, 64, pages=40, page_size=16, factor=4.0, original=64)
    pages = Pages(40, 16, 12)
    x, r = tokens(58, 256, 1)
    place = i32([*range(37), 0, *range(20)])
    want, past = layer.reference(x, r, place, [None] * 3, [37, 1, 20])
    out = layer.forward(x, r, place, **pages.extend({"a": 37, "b": 1, "c": 20}))
    print("prompts: relative error %.4f" % ((out.double() - want).norm() / want.norm()))
    x, r = tokens(3, 256, 2)
    place = i32([37, 1, 20])
    want, past = layer.reference(x, r, place, past, [1, 1, 1])
    out = layer.forward(x, r, place, **pages.extend({"a": 1, "b": 1, "c": 1}))
    print("decode:  relative error %.4f" % ((out.double() - want).norm() / want.norm()))
    # a root, two drafts after it, and one after the second of these; nothing for c
    x, r = tokens(8, 256, 3)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1101] * 2, device="cuda")
    place = i32([38 + j for j in (0, 1, 1, 2)] + [2 + j for j in (0, 1, 1, 2)])
    want, _ = layer.reference(x, r, place, past[:2], [4, 4], tree)
    out = layer.forward(x, r, place, **pages.extend({"a": 4, "b": 4}), tree=tree)
    print("drafts:  relative error %.4f" % ((out.double() - want).norm() / want.norm()))


def full():
    context = 8192
    layer = AttentionLayer(7168, 96, 8, 128, pages=64 * (context // 64 + 8), page_size=64, spare=128)
    for name, n, seqs, tree in (("1 token", 1, 1, False), ("64 tokens of 64 users", 64, 64, False), ("8 trees of 16", 128, 8, True),
                                ("512 tokens of a prompt", 512, 1, False)):
        pages = Pages(64 * (context // 64 + 8), 64, context // 64 + 8)
        pages.extend({s: context for s in range(seqs)})
        x, r = tokens(n, 7168, 3)
        new = n // seqs
        at = pages.extend({s: new for s in range(seqs)})
        place = i32(list(range(context, context + new)) * seqs)
        words = torch.tensor([(2 << j) - 1 for j in range(new)] * seqs, device="cuda") if tree else None
        layer.forward(x, r, place, **at, tree=words)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(x, r, place, **at, tree=words)
        graph.replay()
        torch.cuda.synchronize()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{name} after {context}: {start.elapsed_time(end) / 20 * 1e3:.1f} us a layer, as a CUDA graph")


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--full", action="store_true")
    full() if ap.parse_args().full else check()
