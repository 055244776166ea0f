"""Plain fp64 attention, its gradients and the bounds on what a correct kernel may be off.

Everything is written out per sequence and query head with dense score
matrices in numpy.  Bounds per output element, from the roundings a kernel may
make (u = 2^-8, half a unit in the last of the 8 significant bits of bf16; e = 1e-5, fp32 sums of a few hundred products
and the exponential's argument): with bf16 the probabilities and score
gradients are rounded once as operands (u each, relative), o once before delta
is formed from it, and every output once.
"""
from __future__ import annotations

import numpy as np

U = {"bf16": 2.0 ** -8, "fp32": 0.0}
E = 1e-5


def segments(B, T, cu):
    edges = [b * T for b in range(B + 1)] if cu is None else [int(c) for c in cu]
    return [(a, b) for a, b in zip(edges[:-1], edges[1:]) if b > a]


def forward(q, k, v, scale, segs):
    """(N,Hq,d), (N,Hkv,d) fp64 -> o (N,Hq,d), lse (Hq,N)."""
    N, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, lse = np.zeros((N, Hq, d)), np.zeros((Hq, N))
    for a, b in segs:
        keep = np.tril(np.ones((b - a, b - a), bool))
        for h in range(Hq):
            p, l = _probs(q[a:b, h], k[a:b, h // G], scale, keep)
            lse[h, a:b] = l
            o[a:b, h] = p @ v[a:b, h // G]
    return o, lse


def _probs(q, k, scale, keep):
    s = np.where(keep, q @ k.T * scale, -np.inf)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    tot = w.sum(1, keepdims=True)
    return w / tot, (np.log(tot) + top)[:, 0]


def full(q, k, v, g, scale, segs, dtype):
    """o, lse, dq, dk, dv and a bound per element of each (dict of (value, bound))."""
    N, Hq, d = q.shape
    Hkv = k.shape[1]
    G, u = Hq // Hkv, U[dtype]
    z = lambda x: (np.zeros_like(x), np.zeros_like(x))
    (o, bo), (dq, bq), (dk, bk), (dv, bv) = z(q), z(q), z(k), z(v)
    lse = np.zeros((Hq, N))
    bl = np.zeros((Hq, N))
    for a, b in segs:
        keep = np.tril(np.ones((b - a, b - a), bool))
        for h in range(Hq):
            j = h // G
            qh, kh, vh, gh = q[a:b, h], k[a:b, j], v[a:b, j], g[a:b, h]
            p, l = _probs(qh, kh, scale, keep)
            lse[h, a:b] = l
            bl[h, a:b] = E * (1 + np.abs(l) + (np.abs(qh) @ np.abs(kh).T * scale * keep).max(1))
            o[a:b, h] = p @ vh
            bo[a:b, h] = (2 * u + E) * (p @ np.abs(vh))
            dp = gh @ vh.T
            delta = (gh * o[a:b, h]).sum(1, keepdims=True)
            dabs = (np.abs(gh) * np.abs(o[a:b, h])).sum(1, keepdims=True)
            pabs = np.abs(gh) @ np.abs(vh).T
            ds = scale * p * (dp - delta)
            # operand rounding of ds, delta from the rounded o, fp32 noise of the two sums that are subtracted
            eds = u * np.abs(ds) + scale * p * (u * dabs + E * (pabs + dabs))
            dq[a:b, h] = ds @ kh
            bq[a:b, h] = eds @ np.abs(kh)
            dk[a:b, j] += ds.T @ qh
            bk[a:b, j] += eds.T @ np.abs(qh)
            dv[a:b, j] += p.T @ gh
            bv[a:b, j] += (u + E) * (p.T @ np.abs(gh))
    tiny = 1e-7
    out = {"o": (o, bo + tiny), "lse": (lse, bl)}
    for n, x, bx in (("dq", dq, bq), ("dk", dk, bk), ("dv", dv, bv)):
        out[n] = (x, bx + (u + 2.0 ** -24) * np.abs(x) + tiny)
    return out


def rope(x, pos, base):
    """(N,h,d) rows turned pair by pair by pos * base^(-2i/d)."""
    d = x.shape[-1]
    ang = pos[:, None] * base ** (-np.arange(0, d, 2) / d)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = np.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 1::2] * c + x[..., 0::2] * s
    return y


def decode(q, ks, vs, scale, dtype):
    """One query row per sequence (S,Hq,d) over lists of (n,Hkv,d) -> o and its bound."""
    o, bo = np.zeros_like(q), np.zeros_like(q)
    u = U[dtype]
    for i, (k, v) in enumerate(zip(ks, vs)):
        if len(k) == 0:
            continue
        G = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            p, _ = _probs(q[i:i + 1, h], k[:, h // G], scale, np.ones((1, len(k)), bool))
            o[i, h] = (p @ v[:, h // G])[0]
            bo[i, h] = ((2 * u + E) * (p @ np.abs(v[:, h // G])))[0]
    return o, bo + 1e-7
