"""The operators around the decode projections of a delta-attention layer, as they are measured.

A layer whose packed input projection is 49376 x 7168 and whose output projection is
7168 x 12288 has 96 heads of 128 channels.  Around those projections it runs

  norm   h = bf16(x + residual), y = h / rms(h) * weight, stored as BF16 or in 8 bits with scales
         (int8: one scale a token; e4m3: one scale a group of 128 columns);
  int8   y[b, n] = bf16(x_scale[b] * w_scale[n] * sum_k xq[b, k] * wq[n, k]): the projection with
         8-bit integers on both sides, half the weight bytes of the BF16 one;
  delta  the gated delta rule over ragged sequences, from one token each to long ones:
         S <- S diag(exp(g_t)),  S <- S + beta_t (v_t - S k_t) k_t^T,  o_t = scale S q_t
         with a state S [Dv, Dk] in 32 bits for each sequence and head.

`own` is set by whoever measures: False computes plain torch operations, True calls the framework.
"""
import math

import torch

own = False

CHUNK = 32      # tokens handled at once by the plain form of the delta rule
GROUP = 128     # columns that share an e4m3 scale
EPS = 1e-6      # of both norms


# ---- the cases -------------------------------------------------------------------------------

def _norm(rows, cols, fmt, residual=True):
    return {"op": "norm", "rows": rows, "cols": cols, "fmt": fmt, "residual": residual}


def _int8(rows, n, k):
    return {"op": "int8", "rows": rows, "n": n, "k": k}


def _delta(seqs, total, ragged, hq, hv, dk, dv, channel, zero):
    """`total` tokens in `seqs` sequences, in equal parts or ragged; channel: a decay for every
    channel, else one a head; zero: sequences start from an empty state."""
    return {"op": "delta", "seqs": seqs, "total": total, "ragged": ragged, "hq": hq, "hv": hv,
            "dk": dk, "dv": dv, "channel": channel, "zero": zero}


def listed():
    return [
        # one decode token enters the layer, for an 8-bit projection: pure latency
        {"name": "norm_int8_1x7168", **_norm(1, 7168, "int8")},
        # a full decode batch
        {"name": "norm_int8_256x7168", **_norm(256, 7168, "int8")},
        # a prompt enters the layer
        {"name": "norm_e4m3_8192x7168", **_norm(8192, 7168, "e4m3")},
        # rows that are neither aligned nor a whole number of vectors, BF16 out
        {"name": "norm_bf16_1037x5001", **_norm(1037, 5001, "bf16")},
        # the output projection of one decode token: the weight's bytes are all that matters
        {"name": "int8_1_7168x12288", **_int8(1, 7168, 12288)},
        # the packed input projection of a decode batch
        {"name": "int8_16_49376x7168", **_int8(16, 49376, 7168)},
        # a wide batch, where the tensor cores bound the call
        {"name": "int8_256_14560x7168", **_int8(256, 14560, 7168)},
        # an odd shape: a ragged last tile, and columns that end inside a stage
        {"name": "int8_37_2311x3056", **_int8(37, 2311, 3056)},
        # one decode token of one user: 96 heads' states read and written once
        {"name": "delta_decode_1", **_delta(1, 1, False, 96, 96, 128, 128, True, False)},
        # a decode batch
        {"name": "delta_decode_64", **_delta(64, 64, False, 96, 96, 128, 128, True, False)},
        # prompts of several users in one call, every state empty at the start
        {"name": "delta_prefill_8192", **_delta(4, 8192, True, 96, 96, 128, 128, True, True)},
        # a continued prompt with one decay a head, shared query and key heads, smaller heads
        {"name": "delta_extend_3001", **_delta(5, 3001, True, 8, 32, 64, 128, False, False)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "int8", "delta", "delta"])
    if op == "norm":
        rows = _log(rng, 1, 8192)
        cols = rng.choice([7168, 12288, 8 * _log(rng, 8, 1536), _log(rng, 64, 12288)])
        if rows * cols > 8192 * 7168:
            rows = 8192 * 7168 // cols
        return _norm(rows, cols, rng.choice(["bf16", "int8", "e4m3"]), rng.random() < 0.75)
    if op == "int8":
        n, k = rng.choice([(7168, 12288), (14560, 7168), (49376, 7168), (_log(rng, 64, 16384), 16 * _log(rng, 8, 768))])
        return _int8(_log(rng, 1, 256 if n <= 16384 else 64), n, k)
    hq, hv = rng.choice([(96, 96), (12, 12), (16, 32), (8, 32)])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    channel = rng.random() < 0.6
    if rng.random() < 0.5:  # decode: one token, or the few of a verified draft, for every sequence
        seqs = _log(rng, 1, 128)
        return _delta(seqs, seqs * rng.choice([1, 1, 2, 4]), False, hq, hv, dk, dv, channel, False)
    total = _log(rng, 65, 8192)
    return _delta(_log(rng, 1, max(1, min(16, total // 32))), total, True, hq, hv, dk, dv, channel, rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------------

def _lengths(case, seed):
    """Host-side lengths of the sequences: equal, or cut at random places (one may be empty)."""
    n, total = case["seqs"], case["total"]
    if not case["ragged"]:
        return [total // n] * n
    g = torch.Generator().manual_seed(seed + 77)
    cuts = sorted(torch.randint(0, total + 1, (n - 1,), generator=g).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        T, D = case["rows"], case["cols"]
        s["x"] = normal(T, D).bfloat16()
        s["residual"] = (4 * normal(T, D)).bfloat16() if case["residual"] else None
        s["weight"] = (1 + 0.2 * normal(D)).bfloat16()
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty((T, D), device="cuda", dtype={"bf16": torch.bfloat16, "int8": torch.int8,
                                                             "e4m3": torch.float8_e4m3fn}[case["fmt"]])
        s["scale"] = {"bf16": None, "int8": torch.empty(T, device="cuda"),
                      "e4m3": torch.empty((T, -(-D // GROUP)), device="cuda")}[case["fmt"]]
    elif case["op"] == "int8":
        B, N, K = case["rows"], case["n"], case["k"]
        for name, rows, sigma in (("x", B, 1.0), ("w", N, 0.02)):
            a = normal(rows, K) * sigma
            top = a.abs().amax(1) / 127
            s[name] = torch.round(a / top[:, None]).to(torch.int8)
            s[name + "_scale"] = top
            del a
        s["out"] = torch.empty((B, N), device="cuda", dtype=torch.bfloat16)
        s["handle"] = []  # the program's plan for this weight, made on its first call and kept
    else:
        n, T, hq, hv, dk, dv = (case[i] for i in ("seqs", "total", "hq", "hv", "dk", "dv"))
        # q, k and v are columns of one packed projection's output, as in the layer
        packed = normal(T, hq * dk * 2 + hv * dv).bfloat16()
        q, k, v = packed.split([hq * dk, hq * dk, hv * dv], 1)
        s["q"], s["k"], s["v"] = q.view(T, hq, dk), k.view(T, hq, dk), v.view(T, hv, dv)
        rate = torch.exp(torch.empty(hv, device="cuda").uniform_(math.log(1 / 16), math.log(4), generator=g))
        if case["channel"]:
            s["g"] = -torch.nn.functional.softplus(normal(T, hv, dk) - 2) * rate[:, None]
        else:
            s["g"] = -torch.nn.functional.softplus(normal(T, hv) - 2) * rate
        s["beta"] = torch.sigmoid(normal(T, hv))
        s["lengths"] = _lengths(case, seed)
        cu = torch.tensor([0] + s["lengths"]).cumsum(0)
        s["cu"] = cu.to("cuda", torch.int32) if case["ragged"] else None
        s["state"] = None if case["zero"] else 0.3 * normal(n, hv, dv, dk)
        s["state_out"] = torch.empty(n, hv, dv, dk, device="cuda")
        s["out"] = torch.empty(T, hv, dv, device="cuda", dtype=torch.bfloat16)
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    return {"norm": _run_norm, "int8": _run_int8, "delta": _run_delta}[s["case"]["op"]](s)


def _groups(p, fill=0.0):
    """[T, D] -> [T, groups, 128], the last group filled up."""
    T, D = p.shape
    return torch.nn.functional.pad(p, (0, -D % GROUP), value=fill).view(T, -1, GROUP)


def _run_norm(s):
    fmt = s["case"]["fmt"]
    if own:
        import skinny_bf16_split_gb300 as dep
        dep.add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, quant=None if fmt == "bf16" else fmt,
                         out=s["out"], out_scale=s["scale"], residual_out=s["residual_out"])
        out = {"y": s["out"]} if fmt == "bf16" else _stands_for(s["out"], s["scale"])
        if s["residual"] is not None:
            out["h"] = s["residual_out"]
        return out
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).bfloat16()
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    p = hf * s["weight"].float()  # exact: 8 significant bits on both sides
    if fmt == "bf16":
        out = {"y": (p * rstd).bfloat16()}
    elif fmt == "int8":
        # 1/rms cancels out of the quotient, which is taken in 64 bits for values next to a border
        top = p.abs().amax(1, keepdim=True)
        q = torch.round(127 * p.double() / top.double()).to(torch.int8)
        out = _stands_for(q, (top * rstd / 127)[:, 0])
    else:
        pg = _groups(p)
        top = pg.abs().amax(2, keepdim=True)
        q = (448 * pg.double() / top.double()).float().to(torch.float8_e4m3fn)
        scale = top[..., 0] * rstd / 448
        out = _stands_for(q.view(h.shape[0], -1)[:, : h.shape[1]], scale)
    if s["residual"] is not None:
        out["h"] = h
    return out


def _stands_for(q, scale):
    """8-bit values with their scales: the scales, and the whole numbers (int8) or 8-bit floats
    (e4m3) that they multiply, each as the value it stands for."""
    return {"q": q.float(), "scale": scale} if q.dtype != torch.int8 else {"q": q, "scale": scale}


def _run_int8(s):
    if own:
        import skinny_bf16_split_gb300 as dep
        if not s["handle"]:
            s["handle"].append(dep.Int8Projection(s["w"], s["w_scale"], max_rows=s["case"]["rows"]))
        return s["handle"][0].run(s["x"], s["x_scale"], out=s["out"])
    acc = s["x"].float() @ s["w"].float().t()
    return (acc * s["x_scale"][:, None] * s["w_scale"]).bfloat16()


def _run_delta(s):
    c = s["case"]
    if own:
        import skinny_bf16_split_gb300 as dep
        dep.gated_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["state_out"],
                             cu_seqlens=s["cu"], n_seq=c["seqs"], l2norm=True, out=s["out"])
        return {"o": s["out"], "state": s["state_out"]}
    n, T, hv, dk, dv = c["seqs"], c["total"], c["hv"], c["dk"], c["dv"]
    dev = s["q"].device
    C = min(CHUNK, max(1, max(s["lengths"])))
    # cut the ragged sequences into a flat list of chunks [Z, C], the last of each filled up with
    # zeros (no decay, no write), and one more that is empty, for sequences that have ended
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=dev) * (T // n)
    parts = (cu[1:] - cu[:-1] + C - 1) // C
    first = torch.nn.functional.pad(parts.cumsum(0), (1, 0))
    Z, steps = sum(-(-i // C) for i in s["lengths"]), max(-(-i // C) for i in s["lengths"])
    seq = torch.repeat_interleave(torch.arange(n, device=dev), parts, output_size=Z)
    place = cu[seq, None] + (torch.arange(Z, device=dev) - first[seq])[:, None] * C + torch.arange(C, device=dev)
    live = torch.nn.functional.pad(place < cu[seq + 1, None], (0, 0, 0, 1))
    place = torch.nn.functional.pad(place.clamp(max=T - 1), (0, 0, 0, 1))

    def laid(a):  # [T, heads, ...] -> [Z + 1, hv, C, ...] in 32 bits
        a = a.float()[place] * live.view(Z + 1, C, *[1] * (a.dim() - 1))
        if a.shape[2] != hv:
            a = a.repeat_interleave(hv // a.shape[2], 2)
        return a.movedim(2, 1)

    def unit(a):
        return a * torch.rsqrt(a.square().sum(-1, keepdim=True) + EPS)

    q, k, v = unit(laid(s["q"])) * dk ** -0.5, unit(laid(s["k"])), laid(s["v"])
    beta = laid(s["beta"])[..., None]
    g = laid(s["g"])
    G = (g if c["channel"] else g[..., None].expand(*g.shape, dk)).cumsum(2)
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    if c["channel"]:
        fall = torch.exp((G[..., :, None, :] - G[..., None, :, :]).masked_fill(~low[..., None], -math.inf))
        kk = (k[..., :, None, :] * k[..., None, :, :]).mul_(fall).sum(-1)
        qk = (q[..., :, None, :] * k[..., None, :, :]).mul_(fall).sum(-1)
        del fall
    else:
        fall = torch.exp((G[..., :, None, 0] - G[..., None, :, 0]).masked_fill(~low, -math.inf))
        kk = k @ k.transpose(-1, -2) * fall
        qk = q @ k.transpose(-1, -2) * fall
    # (I + strictly lower part of beta kk)^-1 by forward substitution, all chunks at once
    A = (beta * kk).tril(-1)
    inv = torch.eye(C, device=dev).expand_as(A).contiguous()
    for i in range(1, C):
        inv[..., i, :i] = -(A[..., i : i + 1, :i] @ inv[..., :i, :i]).squeeze(-2)
    eG = torch.exp(G)
    new_v, new_k = inv @ (beta * v), inv @ (beta * k * eG)
    q_in = q * eG
    k_out = k * torch.exp(G[..., -1:, :] - G)
    last = eG[..., -1, :]
    S = torch.zeros(n, hv, dv, dk, device=dev) if s["state"] is None else s["state"]
    o = torch.empty_like(v)
    for z in range(steps):  # the state goes from chunk to chunk
        at = torch.where(z < parts, first[:-1] + z, Z)
        u = new_v[at] - new_k[at] @ S.transpose(-1, -2)
        o[at] = q_in[at] @ S.transpose(-1, -2) + qk[at] @ u
        S = S * last[at, :, None, :] + u.transpose(-1, -2) @ k_out[at]
    o = o.movedim(1, 2)[live].bfloat16()
    return {"o": o, "state": S}


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        T, D = case["rows"], case["cols"]
        out = {"bf16": 2 * T * D, "int8": T * D + 4 * T, "e4m3": T * D + 4 * T * -(-D // GROUP)}[case["fmt"]]
        return {"bytes": T * D * (6 if case["residual"] else 2) + 2 * D + out, "flops": 6 * T * D}
    if case["op"] == "int8":
        B, N, K = case["rows"], case["n"], case["k"]
        return {"bytes": N * K + B * K + 2 * B * N + 4 * (B + N), "flops": 2 * B * N * K}
    n, T, hq, hv, dk, dv = (case[i] for i in ("seqs", "total", "hq", "hv", "dk", "dv"))
    token = 4 * hq * dk + 4 * hv * dv + 4 * hv * (dk if case["channel"] else 1) + 4 * hv
    return {"bytes": T * token + n * hv * dv * dk * 4 * (1 if case["zero"] else 2), "flops": 7 * T * hv * dk * dv}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        D = case["cols"]
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).bfloat16().double()  # the sum is stored in BF16 and read back
        rms = (h.pow(2).sum(1) / D + EPS).sqrt()
        y = h * s["weight"].double() / rms[:, None]
        if case["fmt"] == "bf16":
            out = {"y": y}
        elif case["fmt"] == "int8":
            out = {"q": None, "scale": y.abs().amax(1) / 127}
        else:
            out = {"q": None, "scale": _groups(y).abs().amax(2) / 448}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if case["op"] == "int8":
        a, b = s["x"].double() * s["x_scale"].double()[:, None], s["w"].double() * s["w_scale"].double()[:, None]
        return a @ b.t()
    # token by token, from the definition
    n, T, hq, hv, dk, dv = (case[i] for i in ("seqs", "total", "hq", "hv", "dk", "dv"))
    S = torch.zeros(n, hv, dv, dk, device="cuda", dtype=torch.float64)
    if s["state"] is not None:
        S += s["state"]
    first = torch.tensor([0] + s["lengths"], device="cuda").cumsum(0)[:-1]
    lengths = torch.tensor(s["lengths"], device="cuda")
    share = torch.arange(hv, device="cuda") // (hv // hq)
    qn, kn = (a.double() / (a.double().pow(2).sum(-1, keepdim=True) + EPS).sqrt() for a in (s["q"], s["k"]))
    v, beta = s["v"].double(), s["beta"].double()
    fall = s["g"].double().exp()
    if not case["channel"]:
        fall = fall[..., None]
    o = torch.zeros(T, hv, dv, device="cuda", dtype=torch.float64)
    order = sorted(range(n), key=lambda i: -s["lengths"][i])
    by_length = torch.tensor(order, device="cuda")
    for t in range(max(s["lengths"])):
        at = by_length[: sum(1 for i in s["lengths"] if i > t)]
        tok = first[at] + t
        kt, qt = kn[tok][:, share], qn[tok][:, share]
        St = S[at] * fall[tok][:, :, None, :]
        err = (v[tok] - torch.einsum("nhvk,nhk->nhv", St, kt)) * beta[tok][..., None]
        St = St + err[..., None] * kt[:, :, None, :]
        S[at] = St
        o[tok] = torch.einsum("nhvk,nhk->nhv", St, qt) * dk ** -0.5
    return {"o": o, "state": S}
