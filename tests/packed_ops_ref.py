"""Plain float64 forms of the operators on the packed 4-bit layer and of the
4-bit cache, for their tests: written from the formulas, no library call."""
from __future__ import annotations

import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step
U32 = 2.0 ** -24


def layer(d_out, d_in, G, seed, device="cpu", zeros=None, perm=False):
    """Random packed layer: codes [d_out, d_in], packed words, scales, zero points, perm (or None)."""
    g = torch.Generator().manual_seed(seed)
    Ge = d_in if G == -1 else G
    ng = -(-d_in // Ge)
    codes = torch.randint(0, 16, (d_out, d_in), generator=g)
    scales = torch.rand((d_out, ng), generator=g) * 0.019 + 0.001
    z = torch.randint(0, 16, (d_out, ng), generator=g) if zeros is None else torch.tensor(zeros)[
        torch.randint(0, len(zeros), (d_out, ng), generator=g)]
    p = torch.randperm(d_in, generator=g).to(torch.int32) if perm else None
    w = codes.view(d_out, d_in // 8, 8) << (4 * torch.arange(8))
    words = w.sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    dev = lambda t: None if t is None else t.to(device)  # noqa: E731
    return dict(codes=dev(codes), packed=dev(words), scales=dev(scales), zeros=dev(z.to(torch.int32)), perm=dev(p), G=G)


def dense64(L, dtype):
    """The weight in channel order, [d_out, d_in] float64: round16(scale * (code - zero))."""
    d_in = L["codes"].shape[1]
    G = d_in if L["G"] == -1 else L["G"]
    of = torch.arange(d_in, device=L["codes"].device) // G
    w = (L["scales"][:, of] * (L["codes"] - L["zeros"][:, of]).float()).to(dtype).double()
    if L["perm"] is None:
        return w
    out = torch.empty_like(w)
    out[:, L["perm"].long()] = w
    return out


def act64(x, name):
    """(value, slope)"""
    if name == "relu":
        return x.clamp(min=0), (x > 0).double()
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(x / math.sqrt(2)))
        return x * c, c + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x ** 3))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)
    return x, torch.ones_like(x)


def sum_error(x, W, K):
    """Bound on the rounding of K fp32 additions of exact products: every partial sum is at most sum |x||w|."""
    return (K + 16) * U32 * (x.abs() @ W.abs().t())


# the activations' slopes are at most 1.13, and their fp32 evaluation is off by
# a few units of the value and of the argument (exp of an argument y off by
# |y| 2^-24): 32 |y| 2^-24 covers all four
SLOPE = 1.13
ACT_ERR = 32 * U32


def grid_rows(x):
    """(step, lo, codes) of rows [..., hd], fp32 arithmetic, as the cache defines them."""
    x = x.float()
    nan = torch.isnan(x)
    y = x.clamp(-65504.0, 65504.0)
    lo = torch.where(nan, torch.full_like(y, math.inf), y).amin(-1, keepdim=True)
    hi = torch.where(nan, torch.full_like(y, -math.inf), y).amax(-1, keepdim=True)
    none = lo > hi
    lo, hi = torch.where(none, torch.zeros_like(lo), lo), torch.where(none, torch.zeros_like(hi), hi)
    lo = lo.half().float()
    step = ((hi - lo).clamp(min=0) / 15).half().float()
    c = torch.where(step > 0, torch.round((y - lo) / step), torch.zeros_like(y))
    c = torch.where(nan, torch.zeros_like(c), c).clamp(0, 15)
    return step, lo, c


def cache_values(codes, grid):
    """[pages, kv, page, hd] float64, and the grids' step and lo."""
    sh = 4 * torch.arange(8, device=codes.device)
    c = ((codes.long()[..., None] >> sh) & 15).flatten(-2).double()
    step, lo = grid[..., :1].double(), grid[..., 1:].double()
    return lo + step * c, step, lo


def attention64(q, kc, kg, vc, vg, table, q_start, kv_len, scale, max_q=None, max_kv=None):
    """(out, bound, touched) for q [T, heads, hd] float64; loops over sequences and heads.  bound: a
    derived bound on the error of the kernels before the output's rounding, per 2^-24, and the sum
    that the rounding of the probabilities to 16 bits is relative to."""
    T, H, hd = q.shape
    n_pages, n_kv, page = kc.shape[:3]
    rep = H // n_kv
    kx, ks, kl = cache_values(kc, kg)
    vx, vs, vl = cache_values(vc, vg)
    out = torch.zeros_like(q)
    err = torch.zeros_like(q)
    touched = torch.zeros(T, dtype=torch.bool)
    cap = table.shape[1] * page if max_kv is None else min(max_kv, table.shape[1] * page)
    for b in range(len(kv_len)):
        t0, t1 = min(int(q_start[b]), T), min(int(q_start[b + 1]), T)
        n_q = t1 - t0
        n_k = min(int(kv_len[b]), cap)
        if n_q <= 0:
            continue
        pos = torch.arange(max(n_k, 0))
        pg = table[b, pos // page].long() if n_k > 0 else torch.zeros(0, dtype=torch.long)
        there = (pg >= 0) & (pg < n_pages)
        pos, pg = pos[there], pg[there]
        first = int(kv_len[b]) - n_q
        for i in range(n_q if max_q is None else min(n_q, max_q)):
            touched[t0 + i] = True
            sel = pos <= first + i
            p_, g_ = pos[sel], pg[sel]
            if not len(p_):
                continue
            for h in range(H):
                at = (g_, h // rep, p_ % page)
                qi = q[t0 + i, h]
                s = kx[at] @ qi * scale
                p = torch.softmax(s, 0)
                v = vx[at]
                out[t0 + i, h] = p @ v
                # scores: hd products of q with 16 + code in fp32, then two fp32 steps
                qa = qi.abs().sum()
                ds = (abs(scale) * (hd + 8) * U32 * qa * (31 * ks[at] + (kl[at] - 16 * ks[at]).abs())).max()
                ds = ds + 4 * U32 * s.abs().max()
                mag = p @ (31 * vs[at] + (vl[at] - 16 * vs[at]).abs())
                err[t0 + i, h] = (2 * ds + (len(p_) + 64) * U32) * mag
    return out, err, touched
