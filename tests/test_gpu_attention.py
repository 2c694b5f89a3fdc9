"""Attention over a paged cache against the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), math.inf


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


class Case:
    """Sequences of (new tokens, positions before them), in pages that lie anywhere in the pool.
    Everything of the pool that belongs to no sequence is NaN."""

    def __init__(self, seqs, hq, hk, d, page, layout="token", seed=0, tree=False, scale=None, gap=(0, 0), extra=0):
        host = torch.Generator().manual_seed(seed)
        self.new = [n for n, _ in seqs]
        self.lens = [n + c for n, c in seqs]
        self.hq, self.hk, self.d, self.page = hq, hk, d, page
        self.scale = d ** -0.5 if scale is None else scale
        T = self.T = sum(self.new) + sum(gap)
        self.first = [gap[0] + sum(self.new[:i]) for i in range(len(seqs))]
        self.q = rnd(seed, T, hq * d + 16).bfloat16()[:, : hq * d].unflatten(1, (hq, d))
        need = [-(-n // page) for n in self.lens]
        pages = sum(need) + 3
        width = max(need + [1]) + extra
        if layout == "token":
            self.k, self.v = (torch.full((pages, page, hk, d), NAN, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        elif layout == "head":
            self.k, self.v = (torch.full((pages, hk, page, d), NAN, device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
        else:
            both = torch.full((pages, page, hk, 2 * d), NAN, device="cuda", dtype=torch.bfloat16)
            self.k, self.v = both[..., :d], both[..., d:]
        order = torch.randperm(pages, generator=host).tolist()
        self.table = torch.full((len(seqs), width + 2), -1, dtype=torch.int32)[:, 1: width + 1]
        for s, n in enumerate(need):
            for j in range(n):
                self.table[s, j] = order.pop()
        self.table = torch.full((len(seqs), width + 2), 12345, dtype=torch.int32).cuda()[:, 1: width + 1].copy_(self.table)
        # dense copies, [length, hk, d] for each sequence
        self.keys = [rnd(seed + 100 + s, n, hk, d).bfloat16() for s, n in enumerate(self.lens)]
        self.values = [rnd(seed + 900 + s, n, hk, d).bfloat16() for s, n in enumerate(self.lens)]
        self.tree = None
        if tree:
            words = torch.randint(-(1 << 63), (1 << 63) - 1, (T,), generator=host)
            self.tree = words.cuda()
        self.cu = torch.tensor([gap[0] + sum(self.new[:i]) for i in range(len(seqs) + 1)], dtype=torch.int32, device="cuda")
        self.kv = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.fill()

    def fill(self):
        for s, n in enumerate(self.lens):
            at = torch.arange(n, device="cuda")
            pg = self.table[s].long()[at // self.page]
            self.k[pg, at % self.page], self.v[pg, at % self.page] = self.keys[s], self.values[s]

    def seen(self, s):
        """[new, length] of what each new token of sequence s sees."""
        n, length = self.new[s], self.lens[s]
        own = torch.arange(length, device="cuda") - (length - n)
        if self.tree is None:
            return own[None] <= torch.arange(n, device="cuda")[:, None]
        words = self.tree[self.first[s]: self.first[s] + n]
        return (own < 0) | ((own < 64) & ((words[:, None] >> own.clamp(0, 63)) & 1 == 1))

    def run(self, dep, **kw):
        self.out = torch.full((self.T, self.hq * self.d + 8), NAN, device="cuda", dtype=torch.bfloat16)
        out = self.out[:, : self.hq * self.d].unflatten(1, (self.hq, self.d))
        self.lse = torch.full((self.T, self.hq), NAN, device="cuda")
        args = dict(cu_seqlens=self.cu, tree=self.tree, scale=self.scale, out=out, lse=self.lse)
        got = dep.paged_attention(self.q, self.k, self.v, self.table, self.kv, **{**args, **kw})
        torch.cuda.synchronize()
        assert self.out[:, self.hq * self.d:].isnan().all()
        return got

    def check(self, got, seen=None):
        for s, n in enumerate(self.new):
            f, G = self.first[s], self.hq // self.hk
            see = self.seen(s) if seen is None else seen[s]
            for h in range(self.hq):
                q, k, v = (x.double() for x in (self.q[f: f + n, h], self.keys[s][:, h // G], self.values[s][:, h // G]))
                x = (q @ k.T * self.scale).masked_fill(~see, -INF)
                lse = x.logsumexp(-1)
                p = torch.where(see, (x - lse[:, None]).exp(), 0.0)
                p = torch.where(lse[:, None] == -INF, 0.0, p)
                v = torch.where(see.any(0)[:, None], v, 0.0)
                want, size = p @ v, p @ v.abs()
                # A score: exact products, d sums in FP32 that may cut off (2^-23 of the sum of their sizes each)
                off = self.d * 2.0 ** -23 * self.scale * (q.abs() @ k.abs().T).masked_fill(~see, 0).amax(-1, keepdim=True) if see.shape[1] else torch.zeros(n, 1, device="cuda")
                # o: its rounding (2^-8), the rounding of every p (2^-8), every p's error from its score and from the
                # exponential and the sums (2^-20)
                bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * off + 2.0 ** -20) * size + 1e-38
                bad = ~((got[f: f + n, h].double() - want).abs() <= bound)
                assert not bad.any(), (s, h, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                       got[f: f + n, h][bad][:3].tolist(), want[bad][:3].tolist())
                g = self.lse[f: f + n, h].double()
                fine = torch.where(lse == -INF, g == -INF, (g - lse).abs() <= off[:, 0] + 2.0 ** -20 * (1 + lse.abs()))
                assert fine.all(), (s, h, g[~fine][:3].tolist(), lse[~fine][:3].tolist())


def go(dep, *a, **kw):
    c = Case(*a, **kw)
    c.check(c.run(dep))
    return c


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("context", [0, 1, 15, 63, 64, 126, 127, 128, 129, 255, 256, 257, 383, 1000])
def test_one_token(dep, d, context):
    go(dep, [(1, context)], 12, 1, d, 16, seed=context)


@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (3, 1), (20, 4), (14, 14), (96, 8), (40, 1), (130, 1), (257, 1), (300, 2)])
def test_head_layouts(dep, hq, hk):
    go(dep, [(1, 300), (3, 77)], hq, hk, 128, 16, seed=hq)


@pytest.mark.parametrize("n", [1, 2, 5, 10, 11, 16, 21, 22, 32, 33, 63, 64])
@pytest.mark.parametrize("context", [0, 3, 128, 300])
def test_trees(dep, n, context):
    go(dep, [(n, context), (1, 40), (n, context + 1)], 12, 1, 128, 16, seed=n + context, tree=True)


@pytest.mark.parametrize("n", [1, 2, 16, 43, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("context", [0, 5, 128, 200])
def test_causal(dep, n, context):
    go(dep, [(n, context)], 6, 2, 64 if n % 2 else 128, 24, "head", seed=n + context)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 16, 24, 64, 100, 128, 256, 1000])
@pytest.mark.parametrize("layout", ["token", "head", "rows"])
def test_pages(dep, page, layout):
    go(dep, [(4, 290), (1, 0), (2, 129)], 8, 2, 128, page, layout, seed=page, tree=page % 2 == 0)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_batches(dep, seed, d):
    g = torch.Generator().manual_seed(seed)
    n = int(torch.randint(1, 40, (1,), generator=g))
    tree = seed % 2 == 0
    seqs = [(int(torch.randint(0, 40 if tree else 90, (1,), generator=g)), int(torch.randint(0, 1500, (1,), generator=g)) if i % 5 else 0)
            for i in range(n)]
    hq, hk = [(96, 8), (20, 4), (14, 14)][seed % 3]
    go(dep, seqs, hq, hk, d, [16, 24, 64][seed % 3], ["token", "head", "rows"][seed % 3], seed=seed, tree=tree, gap=(seed, 3))


def test_many_short_sequences(dep):
    go(dep, [(1 + i % 3, i % 9) for i in range(1500)], 4, 2, 64, 4, seed=3)


def test_one_long_context(dep):
    go(dep, [(1, 70001)], 12, 1, 128, 64)
    go(dep, [(16, 40003)], 24, 2, 128, 128, tree=True)


def test_tokens_of_no_sequence_are_left(dep):
    c = go(dep, [(2, 30), (0, 50), (1, 10)], 4, 1, 64, 16, gap=(3, 2))
    for t in (0, 1, 2, 6, 7):
        assert c.out[t].isnan().all() and c.lse[t].isnan().all()
    assert not c.lse[3:6].isnan().any()


def test_equal_sequences_without_a_table_of_starts(dep):
    c = Case([(3, 50), (3, 7), (3, 200)], 4, 2, 128, 16)
    c.check(c.run(dep, cu_seqlens=None))


def test_rows_that_see_nothing(dep):
    c = Case([(5, 0), (5, 200), (64, 0)], 6, 2, 128, 16, tree=True)
    c.tree[1] = c.tree[6] = c.tree[20] = 0
    c.tree[10:] &= ~torch.tensor(0xFFFF, device="cuda")
    got = c.run(dep)
    c.check(got)
    assert (got[1] == 0).all() and (c.lse[1] == -INF).all() and (got[6] != 0).any()


def test_nothing_in_the_cache(dep):
    """Lengths of zero, tables of no width, caches of no pages."""
    c = Case([(2, 0), (1, 0)], 4, 2, 64, 16)
    for kw in (dict(kv=torch.zeros_like(c.kv)), dict(kv=c.kv - 100), dict(table=c.table[:, :0]),
               dict(table=torch.full_like(c.table, -1)), dict(table=torch.full_like(c.table, 1 << 30)), dict(pages=0)):
        out, lse = torch.full((3, 4, 64), NAN, device="cuda", dtype=torch.bfloat16), torch.full((3, 4), NAN, device="cuda")
        pages = kw.get("pages")
        dep.paged_attention(c.q, c.k[:pages], c.v[:pages], kw.get("table", c.table), kw.get("kv", c.kv), cu_seqlens=c.cu, out=out,
                            lse=lse)
        assert (out == 0).all() and (lse == -INF).all(), kw


def test_lengths_outside_the_table(dep):
    """kv_lens past the table is clipped; a sequence shorter than its new tokens has the last of them."""
    c = Case([(3, 45)], 4, 2, 128, 16)
    c.kv[0] = 10 ** 9
    c.table[0, 2] = c.table[0, 1]  # (48 positions: all three pages)
    c.keys[0][32:], c.values[0][32:] = c.keys[0][16:32].clone(), c.values[0][16:32].clone()
    c.check(c.run(dep))
    c = Case([(9, 0)], 4, 2, 128, 16)
    c.kv[0] = 4  # positions 0..3 are those of tokens 5..8
    see = torch.arange(9, device="cuda")[:, None] >= torch.arange(9, device="cuda")[None] + 5
    c.check(c.run(dep), [see])


def test_pages_outside_the_pool_are_not_seen(dep):
    c = Case([(2, 500), (1, 300)], 6, 2, 128, 16)
    seen = [c.seen(0), c.seen(1)]
    for s, j, page in ((0, 3, -1), (0, 4, 10 ** 6), (0, 31, -(2 ** 31)), (1, 0, c.k.shape[0])):
        c.table[s, j] = page
        seen[s][:, 16 * j: 16 * j + 16] = False
    c.check(c.run(dep), seen)


@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("tree", [False, True])
def test_what_is_not_seen_does_not_reach_a_row(dep, what, tree):
    """NaN and infinities in keys and values of new tokens that some rows see and others do not."""
    n = 20
    c = Case([(n, 150), (7, 130)], 12, 2, 128, 16, tree=tree, seed=5)
    want = c.run(dep).clone()
    lse = c.lse.clone()
    for s, j in ((0, 13), (1, 4)):
        at = c.lens[s] - c.new[s] + j
        c.values[s][at, 0, ::3] = what
        c.keys[s][at, 1, 5] = what
    c.fill()
    got = c.run(dep)
    for s, j in ((0, 13), (1, 4)):
        see = c.seen(s)[:, c.lens[s] - c.new[s] + j]
        for i in range(c.new[s]):
            t = c.first[s] + i
            if not see[i]:
                assert torch.equal(got[t], want[t]) and torch.equal(c.lse[t], lse[t]), (s, i)
            else:
                # values: their channels alone; the others as they were
                head = torch.arange(128, device="cuda")
                assert torch.equal(got[t, :6][:, head % 3 != 0], want[t, :6][:, head % 3 != 0])
                hit = got[t, :6][:, ::3]
                assert (hit.isnan() if math.isnan(what) else hit == what).all(), (s, i)
                if math.isnan(what):  # a NaN among the scores
                    assert got[t, 6:].isnan().all() and c.lse[t, 6:].isnan().all()


def test_values_of_the_context_that_are_not_finite(dep):
    c = Case([(3, 400)], 4, 1, 128, 16)
    want = c.run(dep).clone()
    c.values[0][77, 0, 9], c.values[0][301, 0, 10] = INF, NAN
    c.fill()
    got = c.run(dep)
    assert (got[:, :, 9] == INF).all() and got[:, :, 10].isnan().all()
    keep = [i for i in range(128) if i not in (9, 10)]
    assert torch.equal(got[..., keep], want[..., keep])


@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores(dep, d):
    """Scores that rise along the context, so that the running maximum moves all the time, and ones that fall."""
    for sign in (1, -1):
        c = Case([(2, 2000), (40, 700)], 12, 2, d, 16)
        for s in range(2):
            ramp = torch.linspace(0, 6, c.lens[s], device="cuda")[:, None, None] * sign
            c.keys[s] = (c.keys[s].float() * 0.2 + ramp).bfloat16()
        c.q[...] = (c.q.float() * 0.3 + 1).bfloat16()
        c.fill()
        c.check(c.run(dep))


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0, 40.0])
def test_scales(dep, scale):
    go(dep, [(2, 333), (5, 20)], 8, 2, 128, 16, scale=scale)


def test_scores_of_minus_infinity(dep):
    c = Case([(1, 20)], 2, 1, 64, 16)
    c.q[...] = 1.0
    c.keys[0][:10, 0, 0] = -INF
    c.fill()
    got = c.run(dep)
    seen = c.seen(0)
    seen[:, :10] = False
    c.keys[0][:10] = 0
    c.check(got, [seen])


def test_outputs_allocated_and_without_lse(dep):
    c = Case([(2, 40)], 4, 2, 128, 16)
    want = c.run(dep)
    got = dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu)
    assert torch.equal(got, want) and got.is_contiguous()
    none = dep.paged_attention(c.q[:0], c.k, c.v, c.table[:0], c.kv[:0])
    assert none.shape == (0, 4, 128)


def test_same_bits_every_time(dep):
    c = Case([(3, 5000), (1, 17), (16, 900)], 24, 2, 128, 16, tree=True)
    want, lse = c.run(dep).clone(), c.lse.clone()
    for _ in range(5):
        assert torch.equal(c.run(dep), want) and torch.equal(c.lse, lse)


def test_two_streams_at_once(dep):
    cases = [Case([(2, 3000), (1, 100)], 16, 2, 128, 16, seed=i) for i in range(2)]
    want = [c.run(dep).clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, stream=s) for c, s in zip(cases, streams)]
           for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))


def test_graphs(dep):
    """Two captured graphs at once on two streams, replayed with other lengths, tables and trees than captured."""
    cases = [Case([(4, 1000), (2, 300)], 16, 2, 128, 16, seed=i, tree=True) for i in range(2)]
    graphs, outs = [], []
    for c in cases:
        c.run(dep)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, tree=c.tree))
        graphs.append(g)
    for c in cases:  # shorter, split otherwise
        c.kv.copy_(torch.tensor([700, 40]))
        c.cu.copy_(torch.tensor([0, 1, 6]))
        c.tree.bitwise_not_()
    want = [dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, tree=c.tree) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_cache_past_32_bits(dep):
    pages, page, hk, d = 33000, 64, 8, 128
    k, v = (torch.empty(pages, page, hk, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    c = Case([(1, 200)], 16, 8, 128, 64)
    for j, pg in enumerate((32999, 5, 32768, 32767)):
        k[pg], v[pg] = c.k[c.table[0, j]], c.v[c.table[0, j]]
        c.table[0, j] = pg
    c.k, c.v = k, v
    c.check(c.run(dep))


def test_a_run_of_them_as_used(dep):
    """A prompt, decode tokens and a drafted tree through append and attention, against attention over what the
    definition of the norm and rotation gives in 64 bits."""
    hq, hk, d, page, n_seq = 12, 4, 128, 16, 3
    freqs, amplitude = dep.rotary_freqs(d, 1e4, factor=2, original=128)
    qw, kw = (1 + 0.2 * rnd(1, d)).bfloat16(), (1 + 0.2 * rnd(2, d)).bfloat16()
    kc, vc = (torch.full((40, page, hk, d), NAN, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(40)[:36].view(3, 12).int().cuda()
    lens = [0] * n_seq
    keys, values = [[] for _ in range(n_seq)], [[] for _ in range(n_seq)]
    from test_gpu_heads import definition
    for step, new in enumerate(([50, 1, 130], [1, 1, 1], [1, 1, 1], [7, 3, 10])):
        T = sum(new)
        packed = rnd(10 + step, T, (hq + 2 * hk) * d).bfloat16()
        q, k, v = (x.unflatten(1, (-1, d)) for x in packed.split([hq * d, hk * d, hk * d], 1))
        where = [(s, lens[s] + i) for s in range(n_seq) for i in range(new[s])]
        pos = torch.tensor([j for _, j in where], dtype=torch.int32, device="cuda")
        slots = torch.tensor([int(table[s, j // page]) * page + j % page for s, j in where], dtype=torch.int32, device="cuda")
        lens = [a + b for a, b in zip(lens, new)]
        cu = torch.tensor([0] + new).cumsum(0).int().cuda()
        tree = None
        if step == 3:  # chains with a gap: node i descends from i - 2
            tree = torch.tensor([sum(1 << j for j in range(i % 2, i + 1, 2)) for n in new for i in range(n)], device="cuda")
        rot = dep.append_kv(k, v, kc, vc, slots, pos, freqs, amplitude=amplitude, norm=True, k_weight=kw, q=q, q_weight=qw)
        o = dep.paged_attention(rot, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_seqlens=cu, tree=tree)
        yq = definition(q, pos, freqs, False, amplitude, True, qw, 1e-6, 0)[0]
        yk = definition(k, pos, freqs, False, amplitude, True, kw, 1e-6, 0)[0]
        t = 0
        for s, n in enumerate(new):
            keys[s].append(yk[t: t + n])
            values[s].append(v[t: t + n].double())
            K, V = torch.cat(keys[s]), torch.cat(values[s])
            own = torch.arange(len(K), device="cuda") - (len(K) - n)
            i = torch.arange(n, device="cuda")[:, None]
            see = (own <= i) & ((own < 0) | (tree is None) | ((i - own) % 2 == 0))
            for h in range(hq):
                x = (yq[t: t + n, h] @ K[:, h // 3].T * d ** -0.5).masked_fill(~see, -INF)
                p = x.softmax(-1)
                want, size = p @ V[:, h // 3], p @ V[:, h // 3].abs()
                # q and k as stored are off by 2^-8 each: a score by 2^-7 of the sum of its products' sizes at most, and
                # like a random walk over its d products in truth: eight times 2^-7 / sqrt(3 d) of that sum.
                off = 8 * 2.0 ** -7 / math.sqrt(3 * d) * d ** -0.5 * float((yq[t: t + n, h].abs() @ K[:, h // 3].abs().T).max())
                assert ((o[t: t + n, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * off) * size).all()
            t += n


@pytest.mark.parametrize("shift", [-300.0, -60.0, -30.0, 30.0, 200.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_from_zero(dep, shift, d):
    """All scores of a row near one value, low or high; and contexts where they change sides half way."""
    c = Case([(2, 900), (70, 300), (1, 20)], 12, 2, d, 16)
    c.q[...] = (c.q.float() * 0.1 + 1).bfloat16()
    for s in range(3):
        move = torch.full((c.lens[s], 1, 1), shift / d ** 0.5, device="cuda")
        if s < 2:
            move[c.lens[s] // 2:] *= 0.25 if shift < 0 else -0.5
        c.keys[s] = (c.keys[s].float() * 0.2 + move).bfloat16()
    c.fill()
    c.check(c.run(dep))


def test_runs_of_sequences_of_a_tile(dep):
    """Many items of one or two tiles for each block, with and without a second tile of rows."""
    g = torch.Generator().manual_seed(1)
    seqs = [(1 if i % 4 else 30, int(torch.randint(0, 200, (1,), generator=g))) for i in range(300)]
    go(dep, seqs, 12, 2, 128, 16)
    go(dep, seqs, 12, 2, 64, 8, tree=True)


def test_first_tiles_that_a_row_does_not_see(dep):
    """Whole tiles outside the pool before scores far below zero."""
    c = Case([(1, 700), (3, 500)], 8, 2, 128, 16)
    seen = [c.seen(0), c.seen(1)]
    for s in range(2):
        c.keys[s] = (c.keys[s].float() * 0.1 - 25).bfloat16()
        c.table[s, :20] = -1
        seen[s][:, :320] = False
    c.q[...] = (c.q.float() * 0.1 + 1).bfloat16()
    for s in range(2):
        at = torch.arange(320, c.lens[s], device="cuda")
        pg = c.table[s].long()[at // 16]
        c.k[pg, at % 16], c.v[pg, at % 16] = c.keys[s][320:], c.values[s][320:]
    c.check(c.run(dep), seen)


@pytest.mark.parametrize("n,hq,hk", [(64, 96, 8), (43, 14, 1), (30, 40, 1), (64, 32, 1), (25, 21, 1)])
def test_many_rows_of_equal_trees(dep, n, hq, hk):
    """Two to eight blocks of rows of every sequence, and over eight, enough of them to fill the GPU."""
    for seqs in ([(n, 3000), (n, 900), (0, 70), (n, 2500)], [(n, 500 + 13 * i) for i in range(24 // hk + 1)]):
        go(dep, seqs, hq, hk, 128, 16, tree=True, seed=n)
        go(dep, seqs, hq, hk, 64, 16, seed=n)


def test_no_wait_gives_up(dep):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(3):
        c = Case([(1, 3000), (40, 100), (7, 0)], 24, 2, 64 * (1 + i % 2), 16, seed=i, tree=i == 2)
        c.check(c.run(dep, status=status))
    assert status.item() == 0


def test_the_workspace_is_given_back(dep):
    """After a call and after a refusal; on a stream of the caller's it is that stream's."""
    c = Case([(1, 300), (3, 50)], 8, 2, 64, 16)
    out, other = torch.empty_like(c.q), torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for stream in (None, other, other.cuda_stream, 0):
        dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, out=out, stream=stream)
        assert torch.cuda.memory_allocated() == before
    torch.cuda.synchronize()
    with pytest.raises(dep.DepError):
        dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, out=c.q)
    with pytest.raises(dep.DepError):
        dep.paged_attention(c.q, c.k, c.v, c.table, c.kv, cu_seqlens=c.cu, out=out, scale=1e300)
    assert torch.cuda.memory_allocated() == before
