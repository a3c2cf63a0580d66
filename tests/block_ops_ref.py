"""Plain float64 forms, with derived error bounds, of the operators that train and
adapt a block of packed layers: the residual stream's norms, adapters, attention
over whole prompts.  Written from the formulas, no library call."""
from __future__ import annotations

import math

import torch
from packed_ops_ref import EPS, U32

# the smallest step of a type's values near zero, halved: what rounding may add to a tiny value
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def within(got, ref, err, msg=""):
    """|got - ref| <= half a step of got's type at ref, and err (before the rounding, so that step is taken behind it)."""
    e = EPS[got.dtype]
    tol = err * (1 + e) + e * ref.abs() + TINY[got.dtype]
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), f"{msg}: {int(bad.sum())} of {bad.numel()}, worst {float((off / tol.clamp(min=1e-300)).max()):.3g} of the bound"


# ---------------------------------------------------------------- norms

# A sum of squares is added in a tree: 16 values a thread at most, 6 steps over a wave's lanes, 16 waves; a
# product's and a root's rounding and a few more operations on each side: 64 units cover the relative error of
# every factor below.
K = 64 * U32


def unit64(x, eps):
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    return x * r, r


def norm64(R, B, gamma, post, gate, alpha, eps):
    """{h, y} as (value, bound)"""
    one = torch.ones(R.shape[1], dtype=torch.float64, device=R.device)
    h, e = R, torch.zeros_like(R)
    if B is not None:
        b = B if post is None else unit64(B, eps)[0] * post
        add = alpha * (one if gate is None else gate) * b
        h = R + add
        e = K * (R.abs() + add.abs())
    g = one if gamma is None else gamma
    y, r = unit64(h, eps)
    # the root's argument: each h off by e
    shift = (e * h.abs()).mean(1, keepdim=True) * r * r
    return {"h": (h, e), "y": (y * g, (K + shift) * (y * g).abs() + r * g.abs() * e)}


def norm_backward64(dY, H, dH, B, gamma, post, gate, alpha, eps):
    """{dr, db, dgamma, dpost, dgate} as (value, bound)"""
    one = torch.ones(H.shape[1], dtype=torch.float64, device=H.device)
    gm, pw, gw = (one if t is None else t for t in (gamma, post, gate))
    m = H.shape[0]
    n, r = unit64(H, eps)
    g = dY * gm
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    x = torch.zeros_like(H) if dH is None else dH
    dh = x + r * (g - n * mean(g * n))
    e = K * (x.abs() + r * (g.abs() + 2 * n.abs() * mean((g * n).abs())))
    rows = (m + 300) * U32                               # a column's sum: rows one after the other, groups, parts
    out = {"dr": (dh, e), "dgamma": ((dY * n).sum(0), (rows + K) * (dY * n).abs().sum(0))}
    db, edb = alpha * gw * dh, (alpha * gw).abs() * (e + K * dh.abs())
    if B is not None:
        u, q = unit64(B, eps) if post is not None else (B, one)
        b = u * pw
        out["dgate"] = (alpha * (dh * b).sum(0), abs(alpha) * ((rows + 2 * K) * (dh * b).abs() + e * b.abs()).sum(0))
        if post is not None:
            out["dpost"] = ((db * u).sum(0), ((rows + 2 * K) * (db * u).abs() + edb * u.abs()).sum(0))
            gb, eg = db * pw, pw.abs() * edb
            v = q * (gb - u * mean(gb * u))
            edb = q * (eg + u.abs() * mean(eg * u.abs())) + K * q * (gb.abs() + 2 * u.abs() * mean((gb * u).abs()))
            db = v
    out["db"] = (db, edb)
    return out


# ---------------------------------------------------------------- adapters

def token_adapters(q_start, adapter, n_adapters, m):
    """Per token: its adapter, -1 without one, -2 outside the batch."""
    out = torch.full((m,), -2, dtype=torch.long)
    for b in range(len(adapter)):
        t0, t1 = max(int(q_start[b]), 0), min(int(q_start[b + 1]), m)
        if t1 > t0:
            a = int(adapter[b])
            out[t0:t1] = a if 0 <= a < n_adapters else -1
    return out


def piece_error(s, dtype):
    """Of a row of fp32 values in two 16-bit pieces: half a step of half a step; fp16's second piece may be below its
    normal range, 2^-25 of the row's power of two."""
    e = EPS[dtype] ** 2 * s.abs()
    return e if dtype == torch.bfloat16 else e + 2.0 ** -24 * s.abs().amax(-1, keepdim=True)


def lora64(X, A, B, scale, ids, R, dtype):
    """{s, y} as (value, bound); rows outside the batch are 0 here."""
    m, r, d_out = X.shape[0], A.shape[1], B.shape[1]
    s = torch.zeros((m, r), dtype=torch.float64, device=X.device)
    es, y = torch.zeros_like(s), torch.zeros((m, d_out), dtype=torch.float64, device=X.device)
    ey = torch.zeros_like(y)
    for a in sorted(set(ids.tolist()) - {-1, -2}):
        t = (ids == a).to(X.device)
        s[t] = X[t] @ A[a].t()
        es[t] = (X.shape[1] + 64) * U32 * (X[t].abs() @ A[a].abs().t())
        y[t] = scale[a] * (s[t] @ B[a].t())
        mag = (s[t].abs() + es[t]) @ B[a].abs().t()
        ey[t] = scale[a].abs() * ((es[t] + piece_error(s[t], dtype)) @ B[a].abs().t() + (2 * r + 32) * U32 * mag)
    if R is not None:
        y = y + R
        ey = ey + 2 * U32 * y.abs()
    return {"s": (s, es), "y": (y, ey)}


def lora_backward64(dY, X, S, A, B, scale, ids, R, dtype):
    """{dx, da, db} as (value, bound)"""
    m = dY.shape[0]
    dx = torch.zeros((m, A.shape[2]), dtype=torch.float64, device=dY.device)
    edx, da, db = torch.zeros_like(dx), torch.zeros_like(A), torch.zeros_like(B)
    eda, edb = torch.zeros_like(A), torch.zeros_like(B)
    cut = 2.0 ** -24                                     # S and dS enter dA's and dB's products in three bf16 pieces
    for a in sorted(set(ids.tolist()) - {-1, -2}):
        t = (ids == a).to(dY.device)
        ds = dY[t] @ B[a]
        e = (B.shape[1] + 64) * U32 * (dY[t].abs() @ B[a].abs())
        dx[t] = scale[a] * (ds @ A[a])
        mag = (ds.abs() + e) @ A[a].abs()
        edx[t] = scale[a].abs() * ((e + piece_error(ds, dtype)) @ A[a].abs() + (2 * A.shape[1] + 32) * U32 * mag)
        sums = (3 * int(t.sum()) + 64) * U32
        da[a] = scale[a] * (ds.t() @ X[t])
        eda[a] = scale[a].abs() * ((e + (cut + sums) * (ds.abs() + e)).t() @ X[t].abs())
        db[a] = scale[a] * (dY[t].t() @ S[t])
        edb[a] = scale[a].abs() * (cut + sums) * (dY[t].abs().t() @ S[t].abs())
    if R is not None:
        dx = dx + R
        edx = edx + 2 * U32 * dx.abs()
    return {"dx": (dx, edx), "da": (da, eda), "db": (db, edb)}


# ---------------------------------------------------------------- whole prompts

def spans(q_start, T, max_len):
    for b in range(len(q_start) - 1):
        t0, t1 = max(int(q_start[b]), 0), min(int(q_start[b + 1]), T)
        if t1 > t0:
            yield t0, min(t1 - t0, max_len)


def _heads(x, rep=1):
    return x.double().transpose(0, 1).repeat_interleave(rep, 0)


def prompt64(Q, K_, V, q_start, scale, max_len=1 << 30):
    """(out, lse, bound of out, bound of lse, touched)"""
    T, H, hd = Q.shape
    rep, dt = H // K_.shape[1], Q.dtype
    out = torch.zeros((T, H, hd), dtype=torch.float64, device=Q.device)
    lse, eo, el = torch.zeros((T, H), dtype=torch.float64, device=Q.device), torch.zeros_like(out), None
    el = torch.zeros_like(lse)
    touched = torch.zeros(T, dtype=torch.bool, device=Q.device)
    for t0, n in spans(q_start, T, max_len):
        at = slice(t0, t0 + n)
        touched[at] = True
        q, k, v = _heads(Q[at]), _heads(K_[at], rep), _heads(V[at], rep)
        later = torch.ones((n, n), dtype=torch.bool, device=Q.device).triu(1)
        s = (q @ k.transpose(1, 2) * scale).masked_fill(later, -math.inf)
        # a score's error: hd products, the scale, the subtraction of the maximum and the exponential's argument
        es = abs(scale) * (hd + 8) * U32 * (q.abs() @ k.abs().transpose(1, 2)).masked_fill(later, 0).amax(-1)
        es = es + 8 * U32 * s.masked_fill(later, 0).abs().amax(-1)
        p = torch.softmax(s, -1)
        out[at] = (p @ v).transpose(0, 1)
        lse[at] = torch.logsumexp(s, -1).transpose(0, 1)
        # fp16 probabilities below 2^-24 of 2^10 are in steps of that
        low = 2.0 ** -34 * n if dt == torch.float16 else 0.0
        mag = (p @ v.abs()) + low * v.abs().amax(1, keepdim=True)
        eo[at] = ((EPS[dt] + 2 * es + (n + 64) * U32)[..., None] * mag + low * v.abs().amax(1, keepdim=True)).transpose(0, 1)
        el[at] = (es + (n + 64) * U32 + 4 * U32 * lse[at].transpose(0, 1).abs()).transpose(0, 1)
    return out, lse, eo, el, touched


def prompt_backward64(dO, Q, K_, V, out, lse, q_start, scale, max_len=1 << 30):
    """{dq, dk, dv} as (value, bound), from the given out and lse"""
    T, H, hd = Q.shape
    n_kv, dt = K_.shape[1], Q.dtype
    rep = H // n_kv
    f = dict(dtype=torch.float64, device=Q.device)
    dq, dk, dv = torch.zeros((T, H, hd), **f), torch.zeros((T, n_kv, hd), **f), torch.zeros((T, n_kv, hd), **f)
    eq, ek, ev = torch.zeros_like(dq), torch.zeros_like(dk), torch.zeros_like(dv)
    for t0, n in spans(q_start, T, max_len):
        at = slice(t0, t0 + n)
        q, k, v, do, o = _heads(Q[at]), _heads(K_[at], rep), _heads(V[at], rep), _heads(dO[at]), _heads(out[at])
        L = lse[at].double().transpose(0, 1)[..., None]
        later = torch.ones((n, n), dtype=torch.bool, device=Q.device).triu(1)
        s = q @ k.transpose(1, 2) * scale
        p = torch.exp(s - L).masked_fill(later, 0)
        es = abs(scale) * (hd + 8) * U32 * (q.abs() @ k.abs().transpose(1, 2)) + 8 * U32 * (s.abs() + L.abs())
        dp, D = do @ v.transpose(1, 2), (do * o).sum(-1, keepdim=True)
        edp = (hd + 8) * U32 * (do.abs() @ v.abs().transpose(1, 2)) + (hd + 8) * U32 * (do * o).abs().sum(-1, keepdim=True)
        ds = p * (dp - D)
        # p off by 2 es relatively, rounded: half a step (fp16: held times 2^14, so 2^-39 at least)
        low = 2.0 ** -38 if dt == torch.float16 else 0.0
        ep = (EPS[dt] + 2 * es) * p + low * (~later)
        eds = p * edp + 2 * es * ds.abs()
        eds = eds + EPS[dt] * (ds.abs() + eds)
        if dt == torch.float16:
            # held below a power of two that a column's (for dK: a key's, for dQ: a token's) values may be 2^8 under at least
            eds = eds + 2.0 ** -32 * torch.maximum(ds.abs().amax(1, keepdim=True), ds.abs().amax(2, keepdim=True)) * (~later)
        sums = (rep * n + 64) * U32
        kv = lambda x: x.view(n_kv, rep, n, hd).sum(1).transpose(0, 1)  # noqa: E731
        T_ = lambda x: x.transpose(1, 2)  # noqa: E731
        dq[at] = (scale * (ds @ k)).transpose(0, 1)
        eq[at] = (abs(scale) * ((eds + sums * ds.abs()) @ k.abs())).transpose(0, 1)
        dk[at], ek[at] = kv(scale * (T_(ds) @ q)), kv(abs(scale) * (T_(eds + sums * ds.abs()) @ q.abs()))
        dv[at], ev[at] = kv(T_(p) @ do), kv(T_(ep + sums * p) @ do.abs())
    return {"dq": (dq, eq), "dk": (dk, ek), "dv": (dv, ev)}
