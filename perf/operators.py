"""Measured cases of the attention operators that follow the short convolution.

The layer's output row of a token is [Q | K | V] (query heads, key heads, value
heads, each of ``hd`` channels).  Four things a program does with it:

``fwd``     causal attention over whole prompts, grouped heads, packed sequences:
            o and the log-sum-exp of every row (dsc_attn_fwd);
``train``   the same and its gradients for a given dL/do (dsc_attn_fwd, dsc_attn_bwd);
``append``  the new tokens' keys and values written into a paged cache, keys (and
            queries) turned by the rotary embedding on the way (dsc_kv_append);
``decode``  attention of one new token per sequence over the paged cache
            (dsc_attn_decode).

Where ``own`` is true, ``run`` makes the library's calls; otherwise it computes
the same values with elementary torch operations in fp32, rounded once.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt in front of the ~150M block (QKV width 2304 = 3 * 12 * 64): latency
        {"name": "fwd-one-prompt", "op": "fwd", "dtype": "bf16", "B": 1, "T": 37, "Hq": 12, "Hkv": 12, "hd": 64,
         "lo": 0, "hi": 0},
        # a full batch of the ~150M block
        {"name": "fwd-150m", "op": "fwd", "dtype": "bf16", "B": 8, "T": 2048, "Hq": 12, "Hkv": 12, "hd": 64,
         "lo": 0, "hi": 0},
        # packed prompts of the ~2B block (QKV width 6144 = (32 + 8 + 8) * 128), grouped heads
        {"name": "fwd-2b-packed", "op": "fwd", "dtype": "bf16", "B": 4, "T": 4096, "Hq": 32, "Hkv": 8, "hd": 128,
         "lo": 256, "hi": 4096},
        # short ragged prompts in full precision, a head that fills no power of two
        {"name": "fwd-fp32-ragged", "op": "fwd", "dtype": "fp32", "B": 1, "T": 5003, "Hq": 9, "Hkv": 3, "hd": 80,
         "lo": 1, "hi": 700},
        # training steps: the ~150M block, the ~2B block on packed sequences, a short fp32 check run
        {"name": "train-150m", "op": "train", "dtype": "bf16", "B": 8, "T": 2048, "Hq": 12, "Hkv": 12, "hd": 64,
         "lo": 0, "hi": 0},
        {"name": "train-2b-packed", "op": "train", "dtype": "bf16", "B": 4, "T": 4096, "Hq": 32, "Hkv": 8, "hd": 128,
         "lo": 256, "hi": 4096},
        {"name": "train-fp32-ragged", "op": "train", "dtype": "fp32", "B": 1, "T": 1501, "Hq": 6, "Hkv": 2, "hd": 64,
         "lo": 1, "hi": 400},
        # one decoding step's new tokens of 64 sequences, and a packed prefill of the ~2B block
        {"name": "append-step", "op": "append", "dtype": "bf16", "S": 64, "lo": 1, "hi": 1, "past": 2000, "Hq": 12,
         "Hkv": 12, "hd": 64, "page": 16, "rotate": True},
        {"name": "append-prefill", "op": "append", "dtype": "bf16", "S": 12, "lo": 256, "hi": 2400, "past": 300,
         "Hq": 32, "Hkv": 8, "hd": 128, "page": 64, "rotate": True},
        # one sequence (latency), a serving batch of ragged lengths, few sequences over a long fp32 cache
        {"name": "decode-one", "op": "decode", "dtype": "bf16", "S": 1, "lo": 777, "hi": 777, "Hq": 12, "Hkv": 12,
         "hd": 64, "page": 16},
        {"name": "decode-batch", "op": "decode", "dtype": "bf16", "S": 64, "lo": 1, "hi": 16384, "Hq": 32, "Hkv": 8,
         "hd": 128, "page": 64},
        {"name": "decode-long-fp32", "op": "decode", "dtype": "fp32", "S": 2, "lo": 60001, "hi": 131073, "Hq": 16,
         "Hkv": 2, "hd": 128, "page": 48},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(case, seed=0):
    """Lengths of the case's sequences (host integers): a mix that belongs to the case, for the cached
    sequences in an order that belongs to the seed."""
    g = torch.Generator().manual_seed(17)
    if case["op"] in ("append", "decode"):
        n = torch.randint(case["lo"], case["hi"] + 1, (case["S"],), generator=g)
        return n[torch.randperm(case["S"], generator=g.manual_seed(int(seed)))].tolist()
    if case["lo"] == 0:
        return [case["T"]] * case["B"]
    out = []
    for _ in range(case["B"]):  # rows are filled one after the other, the last sequence is cut
        left = case["T"]
        while left:
            n = min(left, int(torch.randint(case["lo"], case["hi"] + 1, (1,), generator=g)))
            out.append(n)
            left -= n
    return out


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "append", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    hd = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7])
    c = {"op": op, "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "hd": hd}
    if op in ("fwd", "train"):
        # a token alone in its sequence has zero gradients of q and k, so training draws start above that
        T = _log_int(rng, 1 if op == "fwd" else 16, 4096 if dtype == "bf16" else 1500)
        B = rng.randint(1, 4)
        lo, hi = rng.choice([(0, 0), (1, 40), (1, max(2, T // 3)), (max(1, T // 4), T)])
        c.update(B=B, T=T, lo=lo, hi=hi)
    elif op == "append":
        n = _log_int(rng, 1, 1500)
        c.update(S=_log_int(rng, 1, 64) if n < 100 else rng.randint(1, 8), lo=rng.choice([1, n]), hi=n,
                 past=rng.choice([0, rng.randint(1, 4000)]), page=rng.choice([16, 24, 64, 128]),
                 rotate=rng.choice([True, True, False]))
    else:
        n = _log_int(rng, 1, 60000)
        c.update(S=_log_int(rng, 1, max(1, min(128, 200000 // n))), lo=rng.choice([1, n]), hi=n,
                 page=rng.choice([1, 16, 24, 64, 256]))
    return c


# ------------------------------------------------------------------- inputs

def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _views(row, case):
    """q, k, v views of rows [Q | K | V] (last dimension (Hq + 2 Hkv) hd)."""
    Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    q, k, v = row.split([Hq * hd, Hkv * hd, Hkv * hd], dim=-1)
    return q.unflatten(-1, (Hq, hd)), k.unflatten(-1, (Hkv, hd)), v.unflatten(-1, (Hkv, hd))


def _rows(g, lead, case):
    """[Q | K | V] rows as the layer leaves them: scores of a few units, values of one."""
    Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    dt = DTYPES[case["dtype"]]
    row = _normal(g, (*lead, (Hq + 2 * Hkv) * hd), 1.0, dt)
    row[..., :(Hq + Hkv) * hd] *= 1.4
    return row


def _pages(g, lens, page, width, pool):
    """A page table (len(lens), width) of the given lengths over a shuffled pool of pages; -1 past each length."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pool, generator=g, device="cuda")[:sum(need)].to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda") < torch.tensor(need, device="cuda")[:, None]] = order
    return table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    lens = _lengths(case, seed)
    s = {"op": case["op"], "scale": 1.0 / math.sqrt(hd), "lens_host": lens, "longest": max(lens)}
    if case["op"] in ("fwd", "train"):
        B, T = case["B"], case["T"]
        s["qkv"] = _rows(g, (B, T), case)
        s["q"], s["k"], s["v"] = _views(s["qkv"], case)
        if case["lo"]:
            s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        else:
            s["cu"] = None
        s["o"] = torch.empty((B, T, Hq, hd), dtype=dt, device="cuda")
        s["lse"] = torch.empty((Hq, B * T), dtype=torch.float32, device="cuda")
        if case["op"] == "train":
            s["do"] = _normal(g, (B, T, Hq, hd), 1.0, dt)
            s["dqkv"] = torch.empty_like(s["qkv"])
            s["dq"], s["dk"], s["dv"] = _views(s["dqkv"], case)
    elif case["op"] == "append":
        N = sum(lens)
        past = torch.randint(0, case["past"] + 1, (len(lens),), generator=g, device="cuda", dtype=torch.int32)
        total = [n + p for n, p in zip(lens, past.tolist())]
        s["qkv"] = _rows(g, (N,), case)
        s["q"], s["k"], s["v"] = _views(s["qkv"], case)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32) if case["hi"] > 1 else None
        s["start"] = past
        width = -(-(case["hi"] + case["past"]) // case["page"])
        pool = len(lens) * width + 3
        s["pages"] = _pages(g, total, case["page"], width, pool)
        s["k_cache"] = _normal(g, (pool, Hkv, case["page"], hd), 1.0, dt)
        s["v_cache"] = _normal(g, (pool, Hkv, case["page"], hd), 1.0, dt)
        s["q_out"] = torch.empty((N, Hq, hd), dtype=dt, device="cuda")
        s["table"] = None
        if case["rotate"]:
            m = torch.arange(case["hi"] + case["past"], device="cuda", dtype=torch.float64)
            theta = 10000.0 ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
            ang = m[:, None] * theta
            s["table"] = torch.stack([ang.cos(), ang.sin()], dim=-1).to(torch.float32).contiguous()
    else:
        S = case["S"]
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        pool = sum(-(-n // case["page"]) for n in lens) + 3
        s["pages"] = _pages(g, lens, case["page"], -(-max(lens) // case["page"]), pool)
        s["q"] = _normal(g, (S, Hq, hd), 1.4, dt)
        s["k_cache"] = _normal(g, (pool, Hkv, case["page"], hd), 1.4, dt)
        s["v_cache"] = _normal(g, (pool, Hkv, case["page"], hd), 1.0, dt)
        s["o"] = torch.empty((S, Hq, hd), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    from input_dependent_short_amd import binding as b
    op = s["op"]
    if op == "append":
        b.dsc_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["start"], cu_seqlens=s["cu"],
                        table=s["table"], q=s["q"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "decode":
        if "ws" not in s:  # kept by the program from step to step
            n = b.dsc_attn_decode_workspace_size(s["q"].dtype, *s["q"].shape[:2], *s["k_cache"].shape[1:2],
                                                 s["q"].shape[2], s["k_cache"].shape[2], s["pages"].shape[1])
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        b.dsc_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lens"], s["o"], s["ws"],
                          scale=s["scale"])
        return {"o": s["o"]}
    b.dsc_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["lse"], cu_seqlens=s["cu"], scale=s["scale"])
    if op == "fwd":
        return {"o": s["o"], "lse": s["lse"]}
    if "ws" not in s:
        B, T, Hq, hd = s["q"].shape
        n = b.dsc_attn_bwd_workspace_size(s["q"].dtype, B, T, Hq, s["k"].shape[2], hd)
        s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    b.dsc_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"], s["ws"],
                   cu_seqlens=s["cu"], scale=s["scale"])
    return {"o": s["o"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _padded(s):
    """Token index (S, L) of every place of the sequences padded to the longest, and which places hold a token."""
    B, T = s["q"].shape[:2]
    N, dev = B * T, s["q"].device
    if s["cu"] is None:
        at = torch.arange(N, device=dev).view(B, T)
        return at, torch.ones_like(at, dtype=torch.bool)
    at = s["cu"][:-1, None].long() + torch.arange(s["longest"], device=dev)
    there = at < s["cu"][1:, None]
    return at.clamp(max=N - 1), there


def _heads(x, at, there, H):
    """(N, h, hd) -> fp32 (S, H, L, hd), heads repeated to H, zero outside the sequences."""
    x = x.flatten(0, 1)[at].float() * there[..., None, None]
    return x.repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2).contiguous()


def _attend(s):
    """Padded q, k, v, the probabilities, the rows' log-sum-exp and the output, all fp32."""
    H = s["q"].shape[2]
    at, there = _padded(s)
    q, k, v = (_heads(s[n], at, there, H) for n in "qkv")
    L = q.shape[2]
    sc = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    sc.masked_fill_(torch.ones(L, L, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = sc.sub_(top).exp_()
    tot = p.sum(-1, keepdim=True)
    p.div_(tot)
    return at, there, q, k, v, p, (tot.log() + top).squeeze(-1), torch.matmul(p, v)


def _tokens(x, s, at, there, dtype):
    """(S, h, L, hd) -> (B, T, h, hd): each token's row, rounded once."""
    B, T = s["q"].shape[:2]
    out = torch.empty((B * T, x.shape[1], x.shape[3]), dtype=dtype, device=x.device)
    out[at[there]] = x.transpose(1, 2)[there].to(dtype)
    return out.unflatten(0, (B, T))


def _plain_fwd(s):
    at, there, _, _, _, _, lse, o = _attend(s)
    flat = torch.empty((lse.shape[1], s["lse"].shape[1]), dtype=torch.float32, device=lse.device)
    flat[:, at[there]] = lse.transpose(0, 1)[:, there]
    return {"o": _tokens(o, s, at, there, s["q"].dtype), "lse": flat}


def _plain_train(s):
    at, there, q, k, v, p, _, o = _attend(s)
    H, Hkv, dt = s["q"].shape[2], s["k"].shape[2], s["q"].dtype
    g = _heads(s["do"], at, there, H)
    delta = (g * o).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), g)
    ds = torch.matmul(g, v.transpose(-1, -2).contiguous()).sub_(delta).mul_(p).mul_(s["scale"])
    del p
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
    del ds
    dk, dv = (x.unflatten(1, (Hkv, H // Hkv)).sum(2) for x in (dk, dv))
    return {"o": _tokens(o, s, at, there, dt), "dq": _tokens(dq, s, at, there, dt),
            "dk": _tokens(dk, s, at, there, dt), "dv": _tokens(dv, s, at, there, dt)}


def _turn(x, cs):
    """Pairs (2i, 2i+1) of the last dimension turned by the angle with cos, sin = cs[..., i, :], in fp32."""
    x = x.float().unflatten(-1, (-1, 2))
    a, b, c, sn = x[..., 0], x[..., 1], cs[..., 0], cs[..., 1]
    return torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)


def _plain_append(s):
    N, page, dt = s["k"].shape[0], s["k_cache"].shape[2], s["k"].dtype
    n = torch.arange(N, device=s["k"].device)
    if s["cu"] is None:
        seq, index = n, torch.zeros_like(n)
    else:
        seq = torch.searchsorted(s["cu"].long(), n, right=True) - 1
        index = n - s["cu"].long()[seq]
    pos = s["start"].long()[seq] + index
    q, k = s["q"], s["k"]
    if s["table"] is not None:
        cs = s["table"][pos][:, None]
        q, k = _turn(q, cs).to(dt), _turn(k, cs).to(dt)
    at = s["pages"][seq, pos // page].long()
    s["k_cache"][at, :, pos % page] = k
    s["v_cache"][at, :, pos % page] = s["v"]
    return {"q": q.contiguous(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_decode(s):
    S, H, hd = s["q"].shape
    pool, Hkv, page, _ = s["k_cache"].shape
    at = s["pages"].clamp(min=0).long()
    W = at.shape[1]
    k, v = (s[n][at].transpose(1, 2).reshape(S, Hkv, W * page, hd).float() for n in ("k_cache", "v_cache"))
    there = (torch.arange(W * page, device=at.device) < s["lens"][:, None])[:, None, None]
    q = s["q"].float().view(S, Hkv, H // Hkv, hd)
    sc = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"]).masked_fill_(~there, -math.inf)
    p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    return {"o": torch.matmul(p, v).view(S, H, hd).to(s["q"].dtype)}


_PLAIN = {"fwd": _plain_fwd, "train": _plain_train, "append": _plain_append, "decode": _plain_decode}


# ------------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    lens = _lengths(case)
    N = sum(lens)
    if case["op"] in ("fwd", "train"):
        pairs = sum(n * (n + 1) // 2 for n in lens)
        qo, kv = N * Hq * hd * es, N * Hkv * hd * es
        if case["op"] == "fwd":
            return {"bytes": 2 * qo + 2 * kv + 4 * N * Hq, "flops": 4 * pairs * Hq * hd}
        return {"bytes": 4 * qo + 4 * kv, "flops": 14 * pairs * Hq * hd}
    if case["op"] == "append":
        return {"bytes": 2 * N * (Hq + 2 * Hkv) * hd * es + (4 * N * hd if case["rotate"] else 0),
                "flops": 6 * N * (Hq + Hkv) * hd // 2 if case["rotate"] else 0}
    return {"bytes": 2 * N * Hkv * hd * es + 2 * case["S"] * Hq * hd * es, "flops": 4 * N * Hq * hd}


# ------------------------------------------------------------------- 64 bits

def _exact_sequence(q, k, v, scale, g=None):
    """One sequence's (n, h, hd) tensors in fp64: o, lse and, with g = dL/do, the gradients, a query head at a time."""
    n, Hq, _ = q.shape
    Hkv = k.shape[1]
    future = torch.arange(n, device=q.device)[None, :] > torch.arange(n, device=q.device)[:, None]
    o, lse = torch.empty_like(q), torch.empty((Hq, n), dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for h in range(Hq):
        j = h // (Hq // Hkv)
        qh, kh, vh = q[:, h].contiguous(), k[:, j].contiguous(), v[:, j].contiguous()
        sc = (qh @ kh.T * scale).masked_fill(future, -math.inf)
        lse[h] = torch.logsumexp(sc, dim=1)
        p = torch.exp(sc - lse[h][:, None])
        o[:, h] = p @ vh
        if g is not None:
            gh = g[:, h].contiguous()
            dv[:, j] += p.T @ gh
            dp = gh @ vh.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
            dq[:, h] = ds @ kh
            dk[:, j] += ds.T @ qh
    return o, lse, dq, dk, dv


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "train"):
        q, k, v = (s[n].flatten(0, 1).double() for n in "qkv")
        g = s["do"].flatten(0, 1).double() if case["op"] == "train" else None
        parts, at = [], 0
        for n in s["lens_host"]:
            parts.append(_exact_sequence(q[at:at + n], k[at:at + n], v[at:at + n], s["scale"],
                                         None if g is None else g[at:at + n]))
            at += n
        B, T = case["B"], case["T"]
        cat = [torch.cat([p[i] for p in parts], dim=1 if i == 1 else 0) for i in range(5)]
        tok = [x if i == 1 else x.unflatten(0, (B, T)) for i, x in enumerate(cat)]
        if case["op"] == "fwd":
            return {"o": tok[0], "lse": tok[1]}
        return {"o": tok[0], "dq": tok[2], "dk": tok[3], "dv": tok[4]}
    if case["op"] == "append":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        page, hd = case["page"], case["hd"]
        theta = torch.tensor([10000.0 ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
        at, turned = 0, []
        for i, n in enumerate(s["lens_host"]):
            m = int(s["start"][i]) + torch.arange(n, device="cuda")
            rows = [q[at:at + n], k[at:at + n]]
            if case["rotate"]:
                z = torch.exp(1j * (m[:, None].double() * theta))[:, None]
                rows = [torch.view_as_real(torch.view_as_complex(x.reshape(n, -1, hd // 2, 2).contiguous()) * z)
                        .flatten(-2) for x in rows]
            turned.append(rows[0])
            pg = s["pages"][i][m // page].long()
            kc[pg, :, m % page] = rows[1]
            vc[pg, :, m % page] = v[at:at + n]
            at += n
        return {"q": torch.cat(turned), "k_cache": kc, "v_cache": vc}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    page, G = case["page"], case["Hq"] // case["Hkv"]
    for i, n in enumerate(s["lens_host"]):
        pg = s["pages"][i][: -(-n // page)].long()
        for j in range(case["Hkv"]):
            k = s["k_cache"][pg, j].double().reshape(-1, case["hd"])[:n]
            v = s["v_cache"][pg, j].double().reshape(-1, case["hd"])[:n]
            qh = s["q"][i, j * G:(j + 1) * G].double()
            out[i, j * G:(j + 1) * G] = torch.softmax(qh @ k.T.contiguous() * s["scale"], dim=1) @ v
    return {"o": out}
