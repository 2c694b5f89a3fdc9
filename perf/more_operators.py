"""The operators of a softmax-attention layer between its two projections, as they are measured.

A layer whose packed input projection has 14560 rows and whose output projection is 7168 x 12288 has
96 query heads of 128 channels; with 8 key and value heads the projection's first 112 x 128 columns
are q, k and v, read in place.  Between the projections it runs

  rotate  q and k, head by head: y = x / rms(x) * weight, then the rotation by the position: for pair
          i of the rotated channels (their two halves, or neighbours) (a, b) becomes
          amplitude * (a cos t - b sin t, b cos t + a sin t) with t = position * freqs[i];
  append  the same on k; k and v are stored to a cache of pages at each token's slot (negative:
          padding), q may be rotated in the same call;
  attend  o = softmax(scale * q K^T) V over the pages of each sequence, whose last n positions are
          those of its n new tokens.  A token sees all positions before these, and of them the ones
          that its mask names (a tree of drafted tokens), or those up to its own.

`own` is set by whoever measures: False computes plain torch operations, True calls the framework.
"""
import math

import torch

own = False

EPS = 1e-6
PACKED = 14560  # columns of the packed projection's output where q, k and v fit into them


# ---- the cases -------------------------------------------------------------------------------

def _rotate(tokens, hq, hk, d, rot, interleaved, norm, far):
    """far: positions up to a million, frequencies scaled for a context 16 times the trained one."""
    return {"op": "rotate", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot, "interleaved": interleaved,
            "norm": norm, "far": far}


def _append(tokens, hq, hk, d, page, by_head, with_q):
    """by_head: a page holds the tokens of each head together, else the heads of each token."""
    return {"op": "append", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "page": page, "by_head": by_head, "with_q": with_q}


def _attend(seqs, tokens, tree, context, ragged, hq, hk, d, page, by_head):
    """`context` positions in the cache before the new tokens and `tokens` new ones, both in equal
    parts or (context always, tokens where there is no tree) ragged over `seqs` sequences."""
    return {"op": "attend", "seqs": seqs, "tokens": tokens, "tree": tree, "context": context, "ragged": ragged,
            "hq": hq, "hk": hk, "d": d, "page": page, "by_head": by_head}


def listed():
    return [
        # one decode token of one user: pure latency
        {"name": "rotate_1", **_rotate(1, 96, 8, 128, 128, False, True, False)},
        # a prompt
        {"name": "rotate_8192", **_rotate(8192, 96, 8, 128, 128, False, True, False)},
        # odd heads, neighbours of a part of each rotated, far positions in a scaled context, no norm
        {"name": "rotate_1037_part", **_rotate(1037, 20, 4, 80, 32, True, False, True)},
        # a decode batch: k and v into their pages, q rotated on the way
        {"name": "append_16", **_append(16, 96, 8, 128, 64, False, True)},
        # a prompt's keys and values
        {"name": "append_8192", **_append(8192, 96, 8, 128, 64, False, False)},
        # smaller heads, pages laid out by head that are no power of two
        {"name": "append_777_by_head", **_append(777, 20, 4, 64, 24, True, True)},
        # one decode token of one user with a short context: pure latency
        {"name": "attend_1x512", **_attend(1, 1, False, 511, False, 96, 8, 128, 64, False)},
        # one decode token of one user with a long context: the axis is split over the GPU
        {"name": "attend_1x131072", **_attend(1, 1, False, 131071, False, 96, 8, 128, 64, False)},
        # a decode batch with contexts of all lengths
        {"name": "attend_64_ragged", **_attend(64, 64, False, 262144, True, 96, 8, 128, 64, False)},
        # trees of 16 drafted tokens for each of 16 users
        {"name": "tree_16x16", **_attend(16, 256, True, 65536, True, 96, 8, 128, 64, False)},
        # wide trees over long contexts, where the tensor cores bound the call
        {"name": "tree_8x64", **_attend(8, 512, True, 131072, False, 96, 8, 128, 64, False)},
        # pieces of prompts of several users, causal; smaller heads, other pages
        {"name": "attend_1501_causal", **_attend(3, 1501, False, 5000, True, 20, 4, 64, 24, True)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(96, 8), (96, 8), (64, 8), (20, 4), (14, 14), (8, 1)]


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend"])
    hq, hk = rng.choice(HEADS)
    if op == "rotate":
        d, rot = rng.choice([(128, 128), (128, 64), (64, 64), (80, 32), (96, 96), (256, 64), (256, 256)])
        tokens = min(_log(rng, 1, 8192), 8192 * 104 * 128 // ((hq + hk) * d))
        return _rotate(tokens, hq, hk, d, rot, rng.random() < 0.4, rng.random() < 0.7, rng.random() < 0.4)
    page, by_head = rng.choice([16, 24, 64, 64, 128, 256, 5]), rng.random() < 0.3
    if op == "append":
        return _append(_log(rng, 1, 8192), hq, hk, rng.choice([128, 128, 64]), page, by_head, rng.random() < 0.5)
    d = rng.choice([128, 128, 64])
    seqs = _log(rng, 1, 64)
    kind = rng.choice(["one", "tree", "causal"])
    tokens = seqs * (1 if kind == "one" else _log(rng, 2, 64)) if kind != "causal" else _log(rng, seqs + 1, 2048)
    most = min(262144, 12288 * 8 * 128 * 64 // (tokens * hq * d // seqs), 262144 * 1024 // (hk * d))
    return _attend(seqs, tokens, kind == "tree", _log(rng, 16, max(17, most)), rng.random() < 0.6, hq, hk, d, page, by_head)


# ---- inputs ----------------------------------------------------------------------------------

def _cut(total, parts, g, least):
    """`total` in `parts` whole numbers of at least `least`, cut at random places."""
    free = total - least * parts
    cuts = sorted(torch.randint(0, free + 1, (parts - 1,), generator=g).tolist())
    return [b - a + least for a, b in zip([0] + cuts, cuts + [free])]


def _equal(total, parts):
    return [total * (i + 1) // parts - total * i // parts for i in range(parts)]


def _frequencies(d, base, factor, trained):
    """radians a position for d / 2 pairs; factor 1: base ** (-2i/d).  Else slow ones are divided by
    the factor, fast ones (32 turns and more in the trained context) kept, a ramp between."""
    f = base ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    if factor == 1:
        return f, 1.0
    turns = lambda n: d * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(turns(32)), 0), min(math.ceil(turns(1)), d - 1)
    ramp = ((torch.arange(d // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1


def _cache(pages, page, heads, d, by_head, normal):
    if by_head:
        return normal(pages, heads, page, d).bfloat16().transpose(1, 2)
    return normal(pages, page, heads, d).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed + 77)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op, T, hq, hk, d = (case[i] for i in ("op", "tokens", "hq", "hk", "d"))
    s = {"case": case}
    # q, k and v are columns of the packed projection's output
    width = (hq + 2 * hk) * d
    packed = normal(T, max(width, PACKED) if width <= PACKED else width).bfloat16()
    q, k, v = packed[:, :width].split([hq * d, hk * d, hk * d], 1)
    s["q"], s["k"], s["v"] = q.view(T, hq, d), k.view(T, hk, d), v.view(T, hk, d)
    if op != "attend":
        far = case.get("far", False)
        rot = case.get("rot", d)
        freqs, s["amplitude"] = _frequencies(rot, 5e5, 16 if far else 1, 65536)
        s["freqs"] = freqs.cuda()
        top = 2 ** 20 if far else 2 ** 17
        start = int(torch.randint(0, top - T, (1,), generator=host))
        s["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int32)
        if op == "append" and T <= 256:  # decode: every token is of another sequence
            s["positions"] = torch.randint(0, top, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["norm"] = case.get("norm", True)
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * normal(d)).bfloat16() if s["norm"] else None for _ in range(2))
        s["q_out"] = torch.empty(T, hq, d, device="cuda", dtype=torch.bfloat16)
    if op == "rotate":
        s["k_out"] = torch.empty(T, hk, d, device="cuda", dtype=torch.bfloat16)
        return s
    page = case["page"]
    if op == "append":
        pages = -(-T // page) + 3
        # tokens fill pages that lie anywhere in the pool, from a place inside the first on; a few are padding
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda") + int(torch.randint(0, page, (1,), generator=host))
        slots = order[at // page] * page + at % page
        pad = torch.rand(T, generator=g, device="cuda") < (0.05 if T > 64 else 0)
        s["slots"] = torch.where(pad, -1, slots).to(torch.int32)
        s["k_cache"], s["v_cache"] = (_cache(pages, page, hk, d, case["by_head"], normal) for _ in range(2))
        return s
    n, C = case["seqs"], case["context"]
    before = _cut(C, n, host, 0) if case["ragged"] else _equal(C, n)
    equal = case["tree"] or T == n or not case["ragged"]
    s["new"] = _equal(T, n) if equal else _cut(T, n, host, 0)
    s["lens"] = [a + b for a, b in zip(before, s["new"])]
    s["cu"] = torch.tensor([0] + s["new"]).cumsum(0).to("cuda", torch.int32)
    s["kv_lens"] = torch.tensor(s["lens"]).to("cuda", torch.int32)
    need = [-(-i // page) for i in s["lens"]]
    pages = sum(need) + 2
    wide = max(need)
    # which pages a sequence has: anywhere in the pool, the table filled up with -1
    order = torch.randperm(pages, generator=g, device="cuda")
    count = torch.tensor(need, device="cuda")
    first = count.cumsum(0) - count
    at = torch.arange(wide, device="cuda")
    s["table"] = torch.where(at < count[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)
    s["k_cache"], s["v_cache"] = (_cache(pages, page, hk, d, case["by_head"], normal) for _ in range(2))
    s["tree"] = _trees(s["new"], host).cuda() if case["tree"] else None
    s["out"] = torch.empty(T, hq, d, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty(T, hq, device="cuda")
    return s


def _trees(new, host):
    """For each drafted token the set of itself and its ancestors, bit j for the sequence's j-th."""
    rows = []
    for n in new:
        seen = []
        parents = torch.randint(-1, 1 << 20, (n,), generator=host).tolist()
        for j in range(n):
            up = max(0, j - 1 - parents[j] % 5)  # one of the five drafted last
            seen.append((seen[up] if j and parents[j] >= 0 else 0) | 1 << j)
        rows += [x - (1 << 64) if x >> 63 else x for x in seen]
    return torch.tensor(rows, dtype=torch.int64)


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return {"rotate": _run_rotate, "append": _run_append, "attend": _run_attend}[s["case"]["op"]](s)


def _turned(s, x, weight):
    """Norm and rotation of [T, heads, d] in 32 bits, angles in 64."""
    x = x.float()
    if s["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    t = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((s["amplitude"] * f(t)).float()[:, None] for f in (torch.cos, torch.sin))
    rot = 2 * s["freqs"].numel()
    part, rest = x[..., :rot], x[..., rot:]
    if s["case"].get("interleaved", False):
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((part, rest), -1).bfloat16()


def _run_rotate(s):
    if own:
        import skinny_bf16_split_gb300 as dep
        dep.norm_rotate(s["q"], s["k"], s["positions"], s["freqs"], interleaved=s["case"]["interleaved"],
                        amplitude=s["amplitude"], norm=s["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                        eps=EPS, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    return {"q": _turned(s, s["q"], s["q_weight"]), "k": _turned(s, s["k"], s["k_weight"])}


def _run_append(s):
    c = s["case"]
    if own:
        import skinny_bf16_split_gb300 as dep
        dep.append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["freqs"],
                      amplitude=s["amplitude"], norm=s["norm"], k_weight=s["k_weight"], eps=EPS,
                      q=s["q"] if c["with_q"] else None, q_weight=s["q_weight"] if c["with_q"] else None,
                      q_out=s["q_out"] if c["with_q"] else None)
        out = {"k": s["k_cache"], "v": s["v_cache"]}
        return {**out, "q": s["q_out"]} if c["with_q"] else out
    live = s["slots"] >= 0
    page, place = s["slots"][live].long() // c["page"], s["slots"][live].long() % c["page"]
    s["k_cache"][page, place] = _turned(s, s["k"], s["k_weight"])[live]
    s["v_cache"][page, place] = s["v"][live]
    out = {"k": s["k_cache"], "v": s["v_cache"]}
    return {**out, "q": _turned(s, s["q"], s["q_weight"])} if c["with_q"] else out


def _run_attend(s):
    c = s["case"]
    if own:
        import skinny_bf16_split_gb300 as dep
        dep.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], cu_seqlens=s["cu"],
                            tree=s["tree"], out=s["out"], lse=s["lse"])
        return {"o": s["out"], "lse": s["lse"]}
    n, T, hq, hk, d = (c[i] for i in ("seqs", "tokens", "hq", "hk", "d"))
    dev, L, N, G = s["q"].device, max(s["lens"]), max(s["new"]), hq // hk
    at = torch.arange(L, device=dev)
    page = s["table"].long()[:, at // c["page"]].clamp(min=0)
    keys, values = (x[page, at % c["page"]].float().transpose(1, 2) for x in (s["k_cache"], s["v_cache"]))  # [n, hk, L, d]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    row = torch.arange(N, device=dev)
    token = (s["cu"][:-1].long()[:, None] + row).clamp(max=T - 1)
    q = s["q"][token].float().view(n, N, hk, G, d).permute(0, 2, 1, 3, 4).reshape(n, hk, N * G, d)
    x = (q * d ** -0.5) @ keys.transpose(-1, -2)
    # which of the sequence's new tokens a position is; negative: a position before them
    j = at - (s["kv_lens"].long() - new)[:, None]
    if s["tree"] is not None:
        seen = (s["tree"][token][:, :, None] >> j.clamp(0, 63)[:, None]) & 1 == 1
        seen = (seen & (j < 64)[:, None]) | (j < 0)[:, None]
    else:
        seen = j[:, None] <= row[:, None]
    seen = (seen & (j < new[:, None])[:, None])[:, None, :, None].expand(n, 1, N, G, L).reshape(n, 1, N * G, L)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ values / torch.where(total > 0, total, 1)
    lse = (top + total.log())[..., 0]
    live = row < new[:, None]
    o = o.view(n, hk, N, G, d).permute(0, 2, 1, 3, 4).reshape(n, N, hq, d)[live]
    lse = lse.view(n, hk, N, G).permute(0, 2, 1, 3).reshape(n, N, hq)[live]
    return {"o": o.bfloat16(), "lse": lse}


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    op, T, hq, hk, d = (case[i] for i in ("op", "tokens", "hq", "hk", "d"))
    if op == "rotate":
        return {"bytes": 4 * T * (hq + hk) * d + 4 * T + 8 * d, "flops": 8 * T * (hq + hk) * d}
    if op == "append":
        heads = 2 * hk + (hq if case["with_q"] else 0)
        return {"bytes": 4 * T * heads * d + 8 * T + 8 * d, "flops": 8 * T * (heads - hk) * d}
    n, C = case["seqs"], case["context"]
    pairs = T * C / n + T * (T / n + 1) / 2  # by the mean where lengths are ragged
    return {"bytes": 4 * (C + T) * hk * d + 4 * T * hq * d + 4 * T * hq + 4 * (C + T) / case["page"],
            "flops": 4 * pairs * hq * d}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _turned_exactly(s, x, weight, interleaved):
    x = x.double()
    if s["norm"]:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    out = x.clone()
    for i, f in enumerate(s["freqs"].tolist()):
        t = s["positions"].double()[:, None] * f
        z = torch.polar(torch.full_like(t, s["amplitude"]), t)
        at = (2 * i, 2 * i + 1) if interleaved else (i, i + s["freqs"].numel())
        turned = torch.complex(x[..., at[0]], x[..., at[1]]) * z
        out[..., at[0]], out[..., at[1]] = turned.real, turned.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    interleaved = case.get("interleaved", False)
    if case["op"] == "rotate":
        return {i: _turned_exactly(s, s[i], s[i + "_weight"], interleaved) for i in ("q", "k")}
    if case["op"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        slots = s["slots"].long()
        t = (slots >= 0).nonzero()[:, 0]
        k[slots[t] // case["page"], slots[t] % case["page"]] = _turned_exactly(s, s["k"], s["k_weight"], interleaved)[t]
        v[slots[t] // case["page"], slots[t] % case["page"]] = s["v"][t].double()
        out = {"k": k, "v": v}
        return {**out, "q": _turned_exactly(s, s["q"], s["q_weight"], interleaved)} if case["with_q"] else out
    T, hq, hk, d, page = (case[i] for i in ("tokens", "hq", "hk", "d", "page"))
    o = torch.zeros(T, hq, d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(T, hq, device="cuda", dtype=torch.float64)
    first = 0
    for i, (new, length) in enumerate(zip(s["new"], s["lens"])):
        pages = s["table"][i, : -(-length // page)].long()
        keys, values = (c[pages].flatten(0, 1)[:length].double() for c in (s["k_cache"], s["v_cache"]))  # [length, hk, d]
        hidden = torch.zeros(new, length, device="cuda", dtype=torch.bool)
        if s["tree"] is None:
            hidden[:, length - new:] = torch.ones(new, new, device="cuda", dtype=torch.bool).triu(1)
        else:
            for j in range(new):
                hidden[:, length - new + j] = (s["tree"][first: first + new] & ((1 << j) - ((1 << 64) if j == 63 else 0))) == 0
        for h in range(hq):
            x = s["q"][first: first + new, h].double() @ keys[:, h // (hq // hk)].T / math.sqrt(d)
            x[hidden] = -math.inf
            lse[first: first + new, h] = x.logsumexp(-1)
            o[first: first + new, h] = x.softmax(-1) @ values[:, h // (hq // hk)]
        first += new
    return {"o": o, "lse": lse}
