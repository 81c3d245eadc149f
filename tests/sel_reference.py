"""The float64 definitions of mod_reference.py over selected blocks of keys:
a problem as there, with blocks [B, HS, NQ, T] (any integers) and bs."""

from unittest import mock

import numpy as np

import mod_reference as ref


def chosen(p, b, h):
    """[NQ, NK]: whether key j lies in a block that query i selected for head h."""
    H, NK = p["q1"].shape[1], p["k1"].shape[2]
    idx = p["blocks"][b, h // (H // p["blocks"].shape[1])]
    nb = -(-NK // p["bs"])
    on = np.zeros((idx.shape[0], nb), dtype=bool)
    for t in range(idx.shape[1]):
        ok = (idx[:, t] >= 0) & (idx[:, t] < nb)
        on[np.nonzero(ok)[0], idx[ok, t]] = True
    return on.repeat(p["bs"], 1)[:, :NK]


def _one(p, b, h):
    """The problem of a single head."""
    H = p["q1"].shape[1]
    one = dict(p)
    for t in "12":
        hk = h // (H // p["k" + t].shape[1])
        one["q" + t], one["k" + t] = p["q" + t][b:b + 1, h:h + 1], p["k" + t][b:b + 1, hk:hk + 1]
    for name in ("doc_q", "doc_k", "prefix"):
        one[name] = None if p[name] is None else p[name][b:b + 1]
    dense = ref.visible
    return one, mock.patch.object(ref, "visible", lambda q, _: dense(q, 0) & chosen(p, b, h))


def forward(p):
    """kl, lse1, lse2 and their bounds, [B, H, NQ]."""
    B, H, NQ, _ = p["q1"].shape
    out = [np.zeros((B, H, NQ)) for _ in range(6)]
    for b in range(B):
        for h in range(H):
            one, patch = _one(p, b, h)
            with patch:
                for o, x in zip(out, ref.forward_head(one, 0, 0)):
                    o[b, h] = x
    return out


def backward(p, kl, l1, l2, dkl, mode):
    """dq, dk and their bounds, for side `mode`, from the given rows."""
    B, H, NQ, _ = p["q1"].shape
    q, k = p["q" + mode], p["k" + mode]
    g = H // k.shape[1]
    dq, bq = np.zeros(q.shape), np.zeros(q.shape)
    dk, bk = np.zeros(k.shape), np.zeros(k.shape)
    for b in range(B):
        for h in range(H):
            one, patch = _one(p, b, h)
            at = (slice(b, b + 1), slice(h, h + 1))
            with patch:
                x = ref.backward(one, kl[at], l1[at], l2[at], dkl[at], mode)
            dq[at], bq[at] = x[0], x[3]
            dk[b, h // g] += x[1][0, 0]
            bk[b, h // g] += x[4][0, 0]
    # (the bounds of shared heads: one rounding to bf16 of the sum instead of one each)
    return dq, dk, bq, bk + ref.BF16 * np.abs(dk)
