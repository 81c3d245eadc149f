"""Selected blocks in calls of the sizes that they are made for: plans made by
three launches, in several chunks of queries and several steps of a chunk, and
selection heads taken a few at a time (groups).  Against float64 on the GPU,
element by element, and against the same heads called one at a time."""

import math

import pytest
import torch

import attention_distillation_kl_gb300 as skl

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24  # one rounding, relative


def problem(B=1, H=4, HK1=2, HK2=2, HS=2, N=2500, d1=64, d2=64, bs=32, T=20, docs=False, seed=0, gone=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = {n: torch.randn((B, h, N, d), generator=g, device="cuda").to(torch.bfloat16)
         for n, h, d in (("q1", H, d1), ("k1", HK1, d1), ("q2", H, d2), ("k2", HK2, d2))}
    nb = -(-N // bs)
    idx = torch.randint(-1, nb, (B, HS, N, T), generator=g, device="cuda", dtype=torch.int32)
    idx[..., 1] = torch.where(torch.rand((B, HS, N), generator=g, device="cuda") < 0.1, idx[..., 0], idx[..., 1])
    idx[:, :, 3::7, 0] = 0  # a block that many share: a list of many tiles
    idx[:, :, ::19] = -1
    for b, h in gone:
        idx[b, h] = -1
    ids = None
    if docs:
        ids = torch.sort(torch.randint(0, 3, (B, N), generator=g, device="cuda"), dim=1)[0].int()
        ids[:, N - N // 9:] = -1
    return x, idx, dict(causal=True, doc_q=ids, doc_k=ids)


def groups(x, idx, backward, mode="2"):
    """Selection heads at a time, and how many times: their queries' rows, and dQ's, in a third of L2 (40 MB)."""
    H, N, d1 = x["q1"].shape[1:]
    d2 = x["q2"].shape[3]
    heads = idx.shape[0] * idx.shape[1]
    row = 2 * (d1 + d2) + (4 * -(-(d2 if mode == "2" else d1) // 32) * 32 if backward else 0)
    at_once = int(max(1, min(heads, 40.0e6 / (row * (H // idx.shape[1]) * N))))
    return at_once, -(-heads // at_once)


def sides(x):
    return [skl.AttnSide(x["q" + t], x["k" + t], 1 / math.sqrt(x["q" + t].shape[3])) for t in "12"]


def head64(x, idx, bs, ids, b, h):
    """(scores and their error, visible) of a head, in float64: fp32 sums of d products, the scale twice."""
    B, H, N, _ = x["q1"].shape
    nb = -(-N // bs)
    i = torch.arange(N, device="cuda")
    on = torch.zeros((N, nb + 1), dtype=torch.bool, device="cuda")
    at = idx[b, h // (H // idx.shape[1])].long()
    on.scatter_(1, torch.where(at >= 0, at, nb), True)
    vis = on[:, :nb].repeat_interleave(bs, 1)[:, :N] & (i[None, :] <= i[:, None])
    if ids is not None:
        vis &= (ids[b][:, None] == ids[b][None, :]) & (ids[b] >= 0)[:, None]
    out = []
    for t in "12":
        q, k = x["q" + t][b, h].double(), x["k" + t][b, h // (H // x["k" + t].shape[1])].double()
        s = 1 / math.sqrt(q.shape[1])
        out += [s * (q @ k.T), (q.shape[1] + 4) * F32 * s * (q.abs() @ k.abs().T)]
        out[-1] = out[-1] + 6 * F32 * out[-2].abs() + 4 * F32
    return *out, vis


def within(got, want, bound, what):
    err = torch.where(want == got, 0.0, (got.double() - want).abs())
    assert torch.isfinite(err).all(), f"{what}: not finite where the definition is"
    over = (err - bound - 1e-30).flatten()
    at = over.argmax()
    assert over[at] <= 0, f"{what} at {at}: error {err.flatten()[at]:.3g}, bound {bound.flatten()[at]:.3g}"


def check(x, idx, bs, where, heads=None):
    """Both directions and modes against float64 (the rows of `heads`, or all, and every dk)."""
    p1, p2 = sides(x)
    B, H, N, _ = x["q1"].shape
    rows = skl.streamkl_fwd_sel(p1, p2, idx, bs, **where)
    dkl = torch.rand(rows[0].shape, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") * 2 - 0.5
    grads = {m: skl.streamkl_bwd_sel(p1, p2, idx, bs, *rows, dkl, f, **where)
             for m, f in (("1", skl.STREAMKL_GRAD_P1), ("2", skl.STREAMKL_GRAD_P2))}
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    T = idx.shape[3]
    ids = where["doc_q"]
    dk, bk = ({m: torch.zeros(x["k" + m].shape, dtype=torch.float64, device="cuda") for m in "12"} for _ in range(2))
    for b in range(B):
        for h in range(H):
            x1, e1, x2, e2, vis = head64(x, idx, bs, ids, b, h)
            hide = lambda v: v.masked_fill(~vis, -math.inf)  # noqa: E731
            seen = vis.any(1)
            l1, l2 = (torch.logsumexp(hide(v), 1) for v in (x1, x2))
            z1, z2 = (torch.where(seen, v, 0.0)[:, None] for v in (l1, l2))
            w1, w2 = torch.exp(hide(x1 - z1)), torch.exp(hide(x2 - z2))
            r = ((x1 - z1) - (x2 - z2)).masked_fill(~vis, 0.0)
            kl = (w1 * r).sum(1)
            # relative error of a sum of exponentials (ex2: 2 units), in blocks, merged slot by slot
            su = (torch.minimum(vis.sum(1), torch.tensor(64, device="cuda")) + 16 + T) * F32
            b1, b2 = (w1 * e1).sum(1) + su + 4 * F32 * z1[:, 0].abs(), (w2 * e2).sum(1) + su + 4 * F32 * z2[:, 0].abs()
            bkl = (w1 * (r - kl[:, None]).abs() * (e1 + e2 + su[:, None])).sum(1) + ((w1 + w2) * e2).sum(1) + 2 * su + \
                su * (w1 * r.abs()).sum(1) + 8 * F32 * (z1 - z2)[:, 0].abs()
            for g, v, e, what in zip(rows, (kl, l1, l2), (bkl, b1, b2), ("KL", "LSE1", "LSE2")):
                within(g[b, h], torch.where(seen, v, 0.0 if what == "KL" else -math.inf), torch.where(seen, e, 0.0), what)
            # the gradients from the rows that they are given
            kl, l1, l2 = (v[b, h].double() for v in rows)
            z1, z2 = (torch.where(seen, v, 0.0)[:, None] for v in (l1, l2))
            a1, a2 = x1 - z1, x2 - z2
            w1, w2 = torch.exp(hide(a1)), torch.exp(hide(a2))
            u1, u2 = (e + F32 * (4 * z.abs() + 2 * a.abs() + 8) for e, z, a in ((e1, z1, a1), (e2, z2, a2)))
            w = dkl[b, h].double()[:, None]
            for m in "12":
                q, k = x["q" + m][b, h].double(), x["k" + m][b, h // (H // x["k" + m].shape[1])].double()
                s = 1 / math.sqrt(q.shape[1])
                if m == "2":
                    ds, es = w * (w2 - w1), w.abs() * (w2 * u2 + w1 * u1)
                else:
                    dev = a1 - a2 - kl[:, None]
                    ds = w * w1 * dev
                    es = w.abs() * w1 * (dev.abs() * u1 + u1 + u2 + 4 * F32 * kl.abs()[:, None])
                dx, ex = s * ds, s * (es + 64 * F32 * ds.abs()) + BF16 * s * ds.abs()
                dq, bq = dx @ k, ex @ k.abs() + (N + 8) * F32 * (dx.abs() @ k.abs())
                # a block's share is rounded to the row's grid: by 2^-22 of its bound at most (streamkl_bwd's mode)
                at = torch.clamp(kl, min=0.0) + 1e-4
                tv = torch.clamp(torch.sqrt(at / 2), max=1.0) + 1e-4
                grid = T * 2.0 ** -22 * 1.01 * s * w[:, 0].abs() * k.abs().max() * (2 * tv if m == "2" else 2 * (at + tv))
                bq = bq + 1.01 * grid[:, None]
                if heads is None or h in heads:
                    within(grads[m][0][b, h], dq, bq + BF16 * (dq.abs() + bq), f"dq, mode P{m}, head {b} {h}")
                hk = h // (H // x["k" + m].shape[1])
                dk[m][b, hk] += dx.T @ q
                # (a chain of MMAs over the rows of all shared heads, then a share for each CTA)
                n = N * (H // x["k" + m].shape[1]) + 320
                bk[m][b, hk] += ex.T @ q.abs() + n * F32 * (dx.abs().T @ q.abs())
    for m in "12":
        within(grads[m][1], dk[m], bk[m] + BF16 * (dk[m].abs() + bk[m]), f"dk, mode P{m}")
    return rows, dkl, grads


PLANS = {  # more than 512 queries x lanes a warp
    "five slots, one step a chunk": dict(N=5000, T=5, H=2, HK1=1, HK2=2),
    "seven slots, several steps a chunk": dict(N=9000, T=7, H=2, HK1=2, HK2=2, bs=64),
    "twenty slots, several steps a chunk": dict(N=2500, T=20),
    "32 slots": dict(N=2100, T=32, bs=128, d1=128, d2=80),
    "documents": dict(B=2, N=2600, T=12, docs=True),
}


@pytest.mark.parametrize("name", PLANS)
def test_plans_of_three_launches(name):
    kw = PLANS[name]
    T, span = kw["T"], 1
    while span < T:
        span *= 2
    assert -(-kw["N"] // 32) * span > 512
    x, idx, where = problem(**kw)
    check(x, idx, kw.get("bs", 32), where)


GROUPS = {
    "one kernel for the plan": dict(H=40, HK1=5, HK2=5, HS=5, N=2000, T=4, bs=64, d1=128, d2=128),
    "three launches": dict(H=40, HK1=5, HK2=5, HS=5, N=2000, T=12, bs=64, d1=128, d2=128),
    "units of a selection": dict(B=2, H=24, HK1=6, HK2=3, HS=3, N=2400, T=8, bs=64, d1=128, d2=128),
    "documents, a narrower student": dict(B=2, H=24, HK1=3, HK2=6, HS=3, N=2600, T=6, bs=128, d1=128, d2=96, docs=True),
    "groups with nothing": dict(H=40, HK1=5, HK2=5, HS=5, N=2000, T=4, bs=64, d1=128, d2=128, gone=[(0, 0), (0, 1), (0, 4)]),
    "nothing in between": dict(H=40, HK1=5, HK2=5, HS=5, N=2000, T=4, bs=32, d1=128, d2=128, gone=[(0, 1), (0, 2), (0, 3)]),
}


@pytest.mark.parametrize("name", GROUPS)
def test_groups_of_selection_heads(name):
    kw = GROUPS[name]
    x, idx, where = problem(**kw)
    at_once, n = groups(x, idx, True)
    assert n >= 3 and at_once >= 2 and groups(x, idx, False)[1] >= 2
    heads = idx.shape[0] * idx.shape[1]
    assert heads % at_once != 0 or idx.shape[0] > 1
    bs = kw["bs"]
    rows, dkl, grads = check(x, idx, bs, where, heads=range(0, kw["H"], 5))
    # a selection head at a time (one group): the same sums of every row, whatever CTA made them
    B, H, HS = idx.shape[0], kw["H"], kw["HS"]
    for b in range(B):
        for s in range(HS):
            one = {}
            for name_, t in x.items():
                n = t.shape[1] // HS
                one[name_] = t[b:b + 1, s * n:(s + 1) * n]
            sel = idx[b:b + 1, s:s + 1].contiguous()
            here = dict(where)
            for i in ("doc_q", "doc_k"):
                here[i] = None if where[i] is None else where[i][b:b + 1].contiguous()
            at = (slice(b, b + 1), slice(s * (H // HS), (s + 1) * (H // HS)))
            alone = skl.streamkl_fwd_sel(*sides(one), sel, bs, **here)
            assert all(torch.equal(u, v[at]) for u, v in zip(alone, rows))
            for m, f in (("1", skl.STREAMKL_GRAD_P1), ("2", skl.STREAMKL_GRAD_P2)):
                dq, _ = skl.streamkl_bwd_sel(*sides(one), sel, bs, *alone, dkl[at].contiguous(), f, **here)
                assert torch.equal(dq, grads[m][0][at])


def test_long_calls_are_repeatable_with_their_own_workspace():
    """Also with a workspace of just the bytes asked for, whatever it holds; one byte less is refused."""
    x, idx, where = problem(**GROUPS["three launches"])
    p1, p2 = sides(x)
    rows = skl.streamkl_fwd_sel(p1, p2, idx, 64, **where)
    dkl = torch.ones_like(rows[0])
    for mode in (skl.STREAMKL_GRAD_P1, skl.STREAMKL_GRAD_P2):
        want = skl.streamkl_bwd_sel(p1, p2, idx, 64, *rows, dkl, mode, **where)
        need = skl.streamkl_bwd_sel_workspace_bytes(p1, p2, idx, 64, mode, **where)
        for fill in (0, 0x5a, 255):
            ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
            got = skl.streamkl_bwd_sel(p1, p2, idx, 64, *rows, dkl, mode, **where, workspace=ws[:need])
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert (ws[need:] == fill).all()
        with pytest.raises(skl.StreamKLError):
            skl.streamkl_bwd_sel(p1, p2, idx, 64, *rows, dkl, mode, **where, workspace=ws[:need - 1])
    need = skl.streamkl_fwd_sel_workspace_bytes(p1, p2, idx, 64, **where)
    for fill in (0, 0x5a, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        got = skl.streamkl_fwd_sel(p1, p2, idx, 64, **where, workspace=ws[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, rows)) and (ws[need:] == fill).all()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
