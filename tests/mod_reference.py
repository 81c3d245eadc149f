"""Plain float64 definitions of the attention KL over modified scores, one
head at a time, with the error bounds that the GPU tests hold the kernels to.

A problem is a dict: q1 [B, H, NQ, d1], k1 [B, HK1, NK, d1], q2, k2 (float64
copies of the bf16 values), scale1, cap1, slopes1 ([H] or None), table1
([H, nb] or None), maxd1, both1 (the same with 2), causal, prefix ([B] or
None), doc_q [B, NQ], doc_k [B, NK] (or None).
"""

import numpy as np

BF16 = 2.0 ** -8    # one rounding to bf16, relative
F32 = 2.0 ** -24    # one rounding to fp32, relative


def bucket(r, nb, maxd, both):
    """Bucket of each relative position in the integer array r, from the
    distances at which the next bucket begins (compared as whole powers, so no
    logarithm is rounded): bucket e + i covers d >= e (maxd / e)^(i / (n - e))."""
    r = np.asarray(r)
    n = nb // 2 if both else nb
    d = np.abs(r) if both else np.maximum(-r, 0)
    e = n // 2
    out = np.minimum(d, e)
    for i in range(1, n - e):
        # d^(n-e) e^i >= maxd^i e^(n-e), in Python's integers
        first = next(x for x in range(e, maxd + 1) if x ** (n - e) * e ** i >= maxd ** i * e ** (n - e))
        out = np.where(d >= first, e + i, out)
    return out + np.where(both & (r > 0), n, 0)


def visible(p, b):
    nq, nk = p["q1"].shape[2], p["k1"].shape[2]
    j = np.arange(nk)[None, :]
    vis = np.ones((nq, nk), dtype=bool)
    if p["causal"]:
        vis = j <= np.arange(nq)[:, None] + nk - nq
        if p["prefix"] is not None:
            vis |= j < p["prefix"][b]
    if p["doc_q"] is not None:
        a, c = p["doc_q"][b][:, None], p["doc_k"][b][None, :]
        vis &= (a == c) & (a >= 0)
    return vis


def score(p, t, b, h):
    """(S, derivative of S by s q.k, bound on the error of S) of side t."""
    q, k = p["q" + t][b, h], p["k" + t][b, h // (p["q1"].shape[1] // p["k" + t].shape[1])]
    nq, nk = q.shape[0], k.shape[0]
    s, d = p["scale" + t], q.shape[1]
    x = s * (q @ k.T)
    # fp32 accumulation of d products, the scale (two roundings) and the bias added last
    err = (d + 4) * F32 * s * (np.abs(q) @ np.abs(k).T)
    grad = np.ones_like(x)
    cap = p["cap" + t]
    if cap:
        th = np.tanh(x / cap)
        x, grad = cap * th, 1 - th * th
        # the polynomial (1.1e-7 = 1.9 roundings, with the folded coefficients' own two) or the quotient
        # (ex2 and rcp at 2 units each, a cancellation of at most two bits)
        err = err * grad + 16 * F32 * np.abs(x)
    r = np.arange(nk)[None, :] - np.arange(nq)[:, None] - (nk - nq)
    bias = np.zeros_like(x)
    if p["slopes" + t] is not None:
        bias = -p["slopes" + t][h] * np.abs(r)
    if p["table" + t] is not None:
        tab = np.clip(p["table" + t][h], -1e30 / np.log2(np.e), 1e30 / np.log2(np.e))
        bias = tab[bucket(r, tab.shape[0], p["maxd" + t], p["both" + t])]
    x = x + bias
    # bias, reference and their sums: each at most the size of the largest term
    err = err + 6 * F32 * (np.abs(x) + np.abs(bias)) + 4 * F32
    return x, grad, err


def lse(x, vis):
    m = np.where(vis, x, -np.inf).max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        return np.where(np.isfinite(m[:, 0]), m[:, 0] + np.log(np.where(vis, np.exp(x - m), 0.0).sum(1)), -np.inf)


def forward_head(p, b, h):
    """kl, lse1, lse2 [NQ] and their bounds."""
    vis = visible(p, b)
    (x1, _, e1), (x2, _, e2) = score(p, "1", b, h), score(p, "2", b, h)
    l1, l2 = lse(x1, vis), lse(x2, vis)
    # a row whose every score is a mask's (below -6.9e5) on one side sees nothing
    seen = np.minimum(np.where(vis, x1, -np.inf).max(1), np.where(vis, x2, -np.inf).max(1)) > -6.9e5
    l1, l2 = np.where(seen, l1, -np.inf), np.where(seen, l2, -np.inf)
    with np.errstate(invalid="ignore", over="ignore"):
        p1 = np.where(vis, np.exp(x1 - l1[:, None]), 0.0)
        p2 = np.where(vis, np.exp(x2 - l2[:, None]), 0.0)
        r = np.where(vis, (x1 - l1[:, None]) - (x2 - l2[:, None]), 0.0)
        kl = (p1 * r).sum(1)
        dev = p1 * np.abs(r - kl[:, None])
        n = vis.sum(1)
        # relative error of a sum of n exponentials (ex2: 2 units), taken in blocks
        su = (np.minimum(n, 64) + 16) * F32
        g1, g2 = (p1 * e1).sum(1) + su, (p2 * e2).sum(1) + su
        bl1, bl2 = g1 + 4 * F32 * np.abs(l1), g2 + 4 * F32 * np.abs(l2)
        # dKL = sum p1 (r - KL) dS1 + sum (p2 - p1) dS2, and the roundings of the sum of p1 (e1 - e2)
        bk = (dev * (e1 + e2 + su[:, None])).sum(1) + ((p1 + p2) * e2).sum(1) + 2 * su
        bk = bk + su * (p1 * np.abs(r)).sum(1) + 8 * F32 * np.abs(l1 - l2)
    fix = lambda v, z: np.where(seen, v, z)  # noqa: E731
    return fix(kl, 0.0), l1, l2, fix(bk, 0.0), fix(bl1, 0.0), fix(bl2, 0.0)


def forward(p):
    B, H = p["q1"].shape[:2]
    return [np.stack(x).reshape(B, H, -1) for x in zip(*(forward_head(p, b, h) for b in range(B) for h in range(H)))]


def grid_error(p, kl, dkl, mode):
    """What the deterministic mode's rounding may add to each row of dq: every
    key tile's contribution to row i is rounded to a multiple of 2^-e with
    2^e (bound_i) > 2^21, so by at most 2^-(e + 1) < 2^-22 bound_i, where
    bound_i = 1.0078125 s |dKL_i| max|K| C_i, C = 2 TV (mode P2) or
    2 (k + TV) (mode P1), k = KL + 1e-4, TV = min(1, sqrt(k / 2)) + 1e-4."""
    k_ = p["k" + mode]
    tiles = -(-k_.shape[2] // 128)
    g = p["q1"].shape[1] // k_.shape[1]
    kmax = np.abs(k_).max((2, 3)).repeat(g, 1)[:, :, None]
    k = np.maximum(kl, 0.0) + 1e-4
    tv = np.minimum(1.0, np.sqrt(k / 2)) + 1e-4
    c = 2 * tv if mode == "2" else 2 * (k + tv)
    return (tiles * 2.0 ** -22 * 1.01 * p["scale" + mode] * np.abs(dkl) * kmax * c)[..., None]


def backward(p, kl, l1, l2, dkl, mode):
    """Gradients of sum(dkl KL) for side `mode` ("1" or "2") from the given kl
    and lse (float64 copies of what the kernel is given), and their bounds:
    dq, dk, dtable, and the same again."""
    B, H, NQ, _ = p["q1"].shape
    t = mode
    q, k = p["q" + t], p["k" + t]
    hk, g = k.shape[1], H // k.shape[1]
    dq, dk = np.zeros(q.shape), np.zeros(k.shape)
    bq, bk, ak = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    tab = p["table" + t]
    dt = np.zeros(tab.shape) if tab is not None else None
    bt = np.zeros(tab.shape) if tab is not None else None
    s = p["scale" + t]
    NK = k.shape[2]
    for b in range(B):
        for h in range(H):
            seen = np.isfinite(l1[b, h])
            vis = visible(p, b) & seen[:, None]
            (x1, g1, e1), (x2, g2, e2) = score(p, "1", b, h), score(p, "2", b, h)
            w = np.where(seen, dkl[b, h], 0.0)[:, None]
            with np.errstate(invalid="ignore", over="ignore"):
                a1, a2 = x1 - l1[b, h][:, None], x2 - l2[b, h][:, None]
                p1, p2 = np.where(vis, np.exp(a1), 0.0), np.where(vis, np.exp(a2), 0.0)
                # exponent: the score, -LSE log2 e and their sum; ex2 two units
                u1 = e1 + F32 * (4 * np.abs(l1[b, h][:, None]) + 2 * np.abs(a1) + 8)
                u2 = e2 + F32 * (4 * np.abs(l2[b, h][:, None]) + 2 * np.abs(a2) + 8)
                if t == "2":
                    ds = np.where(vis, w * (p2 - p1), 0.0)
                    es = np.where(vis, np.abs(w) * (p2 * u2 + p1 * u1), 0.0)
                else:
                    dev = a1 - a2 - kl[b, h][:, None]
                    ds = np.where(vis, w * p1 * dev, 0.0)
                    es = np.where(vis, np.abs(w) * p1 * (np.abs(dev) * u1 + u1 + u2 + 4 * F32 * np.abs(kl[b, h][:, None])), 0.0)
            gr = g2 if t == "2" else g1
            dx = s * ds * gr
            # the derivative 1 - T^2 errs by at most 64 roundings of 1
            ex = s * (es + 64 * F32 * np.abs(ds)) + BF16 * np.abs(dx)
            kk = k[b, h // g]
            # padded keys and queries (ids below 0) may hold anything
            kz = kk if p["doc_k"] is None else np.where((p["doc_k"][b] >= 0)[:, None], kk, 0.0)
            qz = q[b, h] if p["doc_q"] is None else np.where((p["doc_q"][b] >= 0)[:, None], q[b, h], 0.0)
            dq[b, h] = dx @ kz
            bq[b, h] = ex @ np.abs(kz) + (NK + 8) * F32 * (np.abs(dx) @ np.abs(kz))
            dk[b, h // g] += dx.T @ qz
            ak = np.abs(dx).T @ np.abs(qz)
            bk[b, h // g] += ex.T @ np.abs(qz) + (NQ + 8 + 2 * g) * F32 * ak
            if tab is not None:
                r = np.arange(NK)[None, :] - np.arange(NQ)[:, None] - (NK - NQ)
                idx = bucket(r, tab.shape[1], p["maxd" + t], p["both" + t])
                for i in range(tab.shape[1]):
                    dt[h, i] += ds[idx == i].sum()
                    # sums over columns, tiles, warps, key tiles: each a short chain
                    bt[h, i] += es[idx == i].sum() + 256 * F32 * np.abs(ds[idx == i]).sum()
    # the output's own rounding
    bq, bk = bq + BF16 * (np.abs(dq) + bq), bk + BF16 * (np.abs(dk) + bk)
    return dq, dk, dt, bq, bk, bt
