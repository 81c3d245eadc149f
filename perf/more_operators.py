"""Cases for distilling attention that reads only selected blocks of keys, and
for models whose positions have several axes:

  rotate   rotary positions with several axes, and their inverse (the gradient)
  pool     one key for each block of keys: the mean
  select   the blocks whose keys score best for each query
  fwd      KL and both log-sum-exps over the keys of the selected blocks
  bwd      gradient into either side's q and k of the same

rotate: pair p of a row's values, (x[p], x[p + R]) or (x[2p], x[2p + 1]), turns
by the angle position[axis of p] * inv_freq[p]; values beyond 2R are copied.
select: block j scores sum_h q_h . kb_j for a query, over the query heads that
share the key head; candidates are the blocks that hold a key the query may
see; its first `sink` and last `local` candidates are always taken.  Selected
blocks are listed in ascending order, -1 behind them.
fwd, bwd: as the dense ones, key j counts only where block j // bs is selected.
"""

import math
import random

import torch

own = False


def _rot(name, B, H, N, d, sections, **kw):
    c = dict(name=name, op="rotate", B=B, H=H, N=N, d=d, sections=sections, interleaved=False, inverse=False, bshd=True)
    c.update(kw)
    return c


def _sel(name, op, B, H, HK1, HK2, NQ, NK, d1, d2, bs, T, **kw):
    c = dict(name=name, op=op, B=B, H=H, HK1=HK1, HK2=HK2, NQ=NQ, NK=NK, d1=d1, d2=d2, bs=bs, T=T, causal=True, docs=0,
             mode="", sink=1, local=1, bshd=True)
    c.update(kw)
    return c


def listed():
    return [
        # queries of a video model: time, height and width, the largest rotation
        _rot("rotate video", 1, 32, 32760, 128, "16,24,24"),
        # gradient of a batch of images' keys: two axes, pairs side by side, part of the row, odd length
        _rot("rotate images back", 3, 5, 1531, 96, "18,18", interleaved=True, inverse=True, bshd=False),
        # keys of a long context, one for each 64
        dict(name="pool long", op="pool", B=1, HK=8, NK=65536, d=128, bs=64, docs=0, bshd=True),
        # a padded batch of odd length
        dict(name="pool padded", op="pool", B=3, HK=5, NK=1531, d=96, bs=32, docs=1, bshd=False),
        # a long sequence with grouped key heads: the largest selection
        _sel("select long", "select", 1, 32, 8, 8, 16384, 16384, 128, 128, 64, 16),
        # the last tokens of a long context, as in serving
        _sel("select few rows", "select", 1, 32, 8, 8, 16, 65536, 128, 128, 64, 32),
        # the smallest call, where latency counts
        _sel("fwd short", "fwd", 1, 8, 2, 2, 256, 256, 64, 64, 32, 4),
        # a long sequence with grouped key heads: the largest forward
        _sel("fwd long", "fwd", 1, 32, 8, 8, 16384, 16384, 128, 128, 64, 16),
        # the last tokens of a long context: few rows, a long key axis
        _sel("fwd few rows", "fwd", 1, 32, 8, 8, 16, 65536, 128, 128, 64, 32),
        # the smallest training call
        _sel("bwd short", "bwd", 1, 8, 2, 2, 256, 256, 64, 64, 32, 4, mode="P2"),
        # a training step of a long sequence with grouped key heads: the largest backward
        _sel("bwd long", "bwd", 1, 32, 8, 8, 8192, 8192, 128, 128, 64, 16, mode="P2"),
        # gradient into the first side over packed documents of odd length, a student of half the width, large blocks
        _sel("bwd packed P1", "bwd", 2, 16, 4, 8, 2111, 2111, 128, 64, 128, 8, mode="P1", docs=5, bshd=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "pool", "select", "fwd", "fwd", "bwd", "bwd"])
    bshd = rng.random() < 0.6
    if op == "rotate":
        while True:
            B, H, N, d = rng.choice([1, 2, 3]), rng.randint(1, 32), _log_int(rng, 1, 32760), 16 * rng.randint(2, 8)
            if B * H * N * d <= 32 * 32760 * 128:
                break
        axes, left, parts = rng.randint(1, 4), d // 2 if rng.random() < 0.6 else max(4, d // 3), []
        for a in range(axes - 1):
            parts.append(rng.randint(1, max(1, left // 2)))
            left -= parts[-1]
        parts.append(max(1, left))
        return dict(op=op, B=B, H=H, N=N, d=d, sections=",".join(str(p) for p in parts), interleaved=rng.random() < 0.4,
                    inverse=rng.random() < 0.5, bshd=bshd)
    if op == "pool":
        while True:
            B, HK, NK, d = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 5, 8]), _log_int(rng, 1, 65536), 16 * rng.randint(2, 8)
            if B * HK * NK * d <= 8 * 65536 * 128:
                break
        return dict(op=op, B=B, HK=HK, NK=NK, d=d, bs=rng.choice([32, 64, 128]), docs=rng.choice([0, 1]), bshd=bshd)
    n = {"select": 16384, "fwd": 16384, "bwd": 8192}[op]
    while True:
        nk = _log_int(rng, 64, 65536 if op != "bwd" else 16384)
        nq = nk if rng.random() < 0.6 else max(1, int(round(nk * math.exp(-rng.uniform(0.0, 7.0)))))
        bs, hk = rng.choice([32, 64, 64, 128]), rng.choice([1, 2, 3, 4, 8])
        nb = -(-nk // bs)
        T = min(rng.choice([2, 4, 7, 8, 16, 24, 32]), nb + 1)
        h = hk * rng.choice([1, 2, 3, 4, 8])
        b = rng.choice([1, 1, 2, 3])
        if op == "select" and (T < 4 or nb < 3 * T):  # something is left to choose
            continue
        if h <= 32 and T >= 2 and b * h * nq * nk <= 32 * n * n and b * h * nq * T * bs <= 32 * n * 1024:
            break
    d2 = 16 * rng.randint(2, 8)
    d1 = rng.choice([d2, d2, 128])
    return dict(op=op, B=b, H=h, HK1=rng.choice([hk, h]), HK2=hk, NQ=nq, NK=nk, d1=d1, d2=d2, bs=bs, T=T,
                causal=rng.random() < 0.8, docs=rng.choice([0, 0, 1, 4] if op != "select" else [0, 1]) if nq == nk else 0,
                mode=rng.choice(["P1", "P2"]) if op == "bwd" else "", sink=1, local=1, bshd=bshd)


def _ids(c):
    """Document ids [B, N] of packed sequences: `docs` documents of uneven
    lengths and a padded tail (id -1), the same for every seed."""
    rng = random.Random(1000 * c["NK"] + c["docs"])
    rows = []
    for _ in range(c["B"]):
        n = c["NK"]
        pad = rng.randint(0, n // 8)
        cuts = sorted(rng.randint(0, n - pad) for _ in range(c["docs"] - 1))
        row = []
        for i, (lo, hi) in enumerate(zip([0] + cuts, cuts + [n - pad])):
            row += [i] * (hi - lo)
        rows.append(row + [-1] * pad)
    return rows


def _positions(c, axes):
    """A grid of positions for each batch entry: the last axis runs fastest,
    the first (time) goes on from a far offset."""
    sides = [23, 29, 7][: max(0, axes - 1)]
    out = []
    for a in range(axes):
        step = math.prod(sides[a:]) if a < len(sides) else 1
        per = [(n // step) % sides[a - 1] if a else n // step for n in range(c["N"])]
        out.append([[p + (1000 * b if a == 0 else 0) for p in per] for b in range(c["B"])])
    return out


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(h, n, d):  # [B, h, n, d] in fp32
        return torch.randn((c["B"], h, n, d), generator=g, device=dev)

    def lay(x):  # as bf16; a view of [B, N, H, d] where that is how the projection left it
        x = x.to(torch.bfloat16)
        return x.transpose(1, 2).contiguous().transpose(1, 2) if c["bshd"] else x

    s = dict(case=c, doc=None)
    if c.get("docs"):
        s["doc"] = torch.tensor(_ids(c), dtype=torch.int32, device=dev)
    if c["op"] == "rotate":
        sections = [int(x) for x in c["sections"].split(",")]
        s["x"] = lay(rand(c["H"], c["N"], c["d"]))
        s["pos"] = torch.tensor(_positions(c, len(sections)), dtype=torch.int32, device=dev)
        R = sum(sections)
        s["inv_freq"] = torch.tensor([10000.0 ** (-p / R) for p in range(R)], dtype=torch.float32, device=dev)
        s["sections"] = sections
        return s
    if c["op"] == "pool":
        s["k"] = lay(rand(c["HK"], c["NK"], c["d"]) + rand(c["HK"], 1, c["d"]))
        return s
    # stretches of 128 keys share a topic, and a query looks for the topic of some stretch
    seg = (c["NK"] + 127) // 128

    def topical(h, hk, n, d, topic):
        where = torch.arange(n, device=dev) // 128 if h == 0 else \
            torch.randint(0, seg, ((n + 15) // 16,), generator=g, device=dev).repeat_interleave(16)[:n]
        t = topic[:, :, where]
        return (t if h == 0 else t.repeat_interleave(h // hk, 1)) + rand(hk if h == 0 else h, n, d)

    for t in "12":
        hk, d = c["HK" + t], c["d" + t]
        topic = rand(hk, seg, d)
        s["q" + t], s["k" + t] = lay(topical(c["H"], hk, c["NQ"], d, topic)), lay(topical(0, hk, c["NK"], d, topic))
        s["scale" + t] = 1.0 / math.sqrt(d)
    s["kb"] = _plain_pool(s["k2"], c["bs"], s["doc"])
    if c["op"] == "select":
        return s
    s["blocks"] = _plain_select(s, torch.float32)
    if c["op"] == "bwd":  # what the forward left, and the loss's gradient per row
        s["kl"], s["lse1"], s["lse2"] = _plain_fwd(s)
        s["dkl"] = torch.rand((c["B"], c["H"], c["NQ"]), generator=g, device=dev) + 0.5
    return s


def _plain_rotate(s):
    c, x = s["case"], s["x"]
    R = s["inv_freq"].shape[0]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=x.device),
                                   torch.tensor(s["sections"], device=x.device))
    angle = s["pos"].double()[axis].permute(1, 2, 0) * s["inv_freq"].double()  # far positions: 64 bits
    if c["inverse"]:
        angle = -angle
    co, si = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    f = x.float()
    out = f.clone()
    a, b = (slice(0, 2 * R, 2), slice(1, 2 * R, 2)) if c["interleaved"] else (slice(0, R), slice(R, 2 * R))
    out[..., a] = f[..., a] * co - f[..., b] * si
    out[..., b] = f[..., a] * si + f[..., b] * co
    return out.to(torch.bfloat16)


def _plain_pool(k, bs, doc):
    B, H, N, d = k.shape
    pad = -N % bs
    keep = torch.ones((B, N), device=k.device) if doc is None else (doc >= 0).float()
    f = torch.where(keep[:, None, :, None] > 0, k.float(), 0.0)
    f = torch.nn.functional.pad(f, (0, 0, 0, pad)).reshape(B, H, -1, bs, d).sum(3)
    n = torch.nn.functional.pad(keep, (0, pad)).reshape(B, 1, -1, bs).sum(3, keepdim=True)
    return (f / n.clamp(min=1)).to(torch.bfloat16)


def _candidates(s):
    """[B, NQ, NB]: blocks that hold a key the query may see (documents lie in one piece)."""
    c, dev = s["case"], s["q2"].device
    nb = (c["NK"] + c["bs"] - 1) // c["bs"]
    i = torch.arange(c["NQ"], device=dev)[:, None] + c["NK"] - c["NQ"]
    first = torch.arange(nb, device=dev)[None, :] * c["bs"]
    see = (first <= i) if c["causal"] else torch.ones_like(first <= i)
    see = see[None].expand(c["B"], -1, -1)
    if s["doc"] is not None:
        k = torch.nn.functional.pad(s["doc"], (0, -c["NK"] % c["bs"]), value=-1).reshape(c["B"], nb, c["bs"])
        lo, hi = torch.where(k >= 0, k, 2 ** 30).amin(2), k.amax(2)
        q = s["doc"][:, :, None]
        see = see & (q >= 0) & (lo[:, None] <= q) & (q <= hi[:, None])
    return see


def _plain_select(s, dtype=torch.float64):
    c = s["case"]
    hk, T = c["HK2"], c["T"]
    cand = _candidates(s)[:, None]
    forced = cand & ((cand.cumsum(3) <= c["sink"]) | (cand.flip(3).cumsum(3).flip(3) <= c["local"]))
    q = s["q2"].to(dtype).reshape(c["B"], hk, -1, c["NQ"], c["d2"]).sum(2)
    score = torch.matmul(q, s["kb"].to(dtype).transpose(2, 3))  # 64 bits: values next to the border
    score = torch.where(forced, math.inf, torch.where(cand, score, -math.inf))
    top, idx = torch.sort(score, dim=3, descending=True, stable=True)
    nb = idx.shape[3]
    idx = torch.where(top[..., :T] > -math.inf, idx[..., :T], nb)
    idx = torch.nn.functional.pad(idx, (0, max(0, T - nb)), value=nb)
    idx = torch.sort(idx, dim=3)[0]
    return torch.where(idx < nb, idx, -1).to(torch.int32)


def _plain_parts(s):
    """(b, heads, S1, S2, visible) of as many heads at a time as 2^28 scores hold."""
    c, dev = s["case"], s["q1"].device
    nq, nk, H = c["NQ"], c["NK"], c["H"]
    nb = (nk + c["bs"] - 1) // c["bs"]
    step = max(1, min(H, 2 ** 28 // (nq * nk)))
    i = torch.arange(nq, device=dev)[:, None] + nk - nq
    base = torch.arange(nk, device=dev)[None, :] <= (i if c["causal"] else nk)
    hs = s["blocks"].shape[1]
    for b in range(c["B"]):
        see = base
        if s["doc"] is not None:
            see = see & (s["doc"][b][:, None] == s["doc"][b][None, :]) & (s["doc"][b] >= 0)[:, None]
        for h0 in range(0, H, step):
            h = torch.arange(h0, min(H, h0 + step), device=dev)
            idx = s["blocks"][b].long()
            on = torch.zeros((hs, nq, nb + 1), dtype=torch.bool, device=dev)
            on.scatter_(2, torch.where(idx >= 0, idx, nb), True)
            vis = on[..., :nb].repeat_interleave(c["bs"], 2)[..., :nk][h // (H // hs)] & see
            x = []
            for t in "12":
                k = s["k" + t][b].float()[h // (H // c["HK" + t])]
                x.append(torch.matmul(s["q" + t][b, h].float(), k.transpose(1, 2)) * s["scale" + t])
            yield b, h, x[0], x[1], vis


def _plain_lse(x):
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    return torch.log(torch.exp(x - m).sum(-1)) + m[..., 0]


def _plain_fwd(s):
    c = s["case"]
    kl, lse1, lse2 = (torch.empty((c["B"], c["H"], c["NQ"]), device=s["q1"].device) for _ in range(3))
    for b, h, x1, x2, vis in _plain_parts(s):
        x1, x2 = x1.masked_fill_(~vis, -math.inf), x2.masked_fill_(~vis, -math.inf)
        l1, l2 = _plain_lse(x1), _plain_lse(x2)
        lp1, lp2 = x1 - l1[..., None], x2 - l2[..., None]
        kl[b, h] = torch.where(vis, torch.exp(lp1) * (lp1 - lp2), 0.0).sum(-1)
        lse1[b, h], lse2[b, h] = l1, l2
    return kl, lse1, lse2


def _plain_bwd(s):
    c, t = s["case"], s["case"]["mode"][1]
    q, k, hk = s["q" + t], s["k" + t], c["HK" + t]
    dq = torch.empty(q.shape, device=q.device)
    dk = torch.zeros(k.shape, device=q.device)
    for b, h, x1, x2, vis in _plain_parts(s):
        lp1, lp2 = x1 - s["lse1"][b, h][..., None], x2 - s["lse2"][b, h][..., None]
        if t == "2":
            ds = torch.exp(lp2) - torch.exp(lp1)
        else:
            ds = torch.exp(lp1) * (lp1 - lp2 - s["kl"][b, h][..., None])
        dx = s["scale" + t] * torch.where(vis, s["dkl"][b, h][..., None] * ds, 0.0)
        at = h // (c["H"] // hk)
        dq[b, h] = torch.matmul(dx, k[b].float()[at])
        dk[b].index_add_(0, at, torch.matmul(dx.transpose(1, 2), q[b, h].float()))
    return dict(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16))


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "rotate":
            return _plain_rotate(s)
        if op == "pool":
            return _plain_pool(s["k"], c["bs"], s["doc"])
        return {"select": _plain_select, "fwd": _plain_fwd, "bwd": _plain_bwd}[op](s)
    import attention_distillation_kl_gb300 as skl
    if op == "rotate":
        rotary = skl.Rotary(s["inv_freq"], s["pos"], s["sections"], interleaved=c["interleaved"])
        return skl.streamkl_rotate(s["x"], rotary, inverse=c["inverse"])
    if op == "pool":
        return skl.streamkl_pool_blocks(s["k"], c["bs"], doc_k=s["doc"])
    where = dict(causal=c["causal"], doc_q=s["doc"], doc_k=s["doc"])
    if op == "select":
        return skl.streamkl_select_blocks(s["q2"], s["kb"], c["T"], c["bs"], c["NK"], sink=c["sink"], local=c["local"],
                                          **where)
    p1, p2 = (skl.AttnSide(s["q" + t], s["k" + t], s["scale" + t]) for t in "12")
    if op == "fwd":
        return skl.streamkl_fwd_sel(p1, p2, s["blocks"], c["bs"], **where)
    mode = skl.STREAMKL_GRAD_P1 if c["mode"] == "P1" else skl.STREAMKL_GRAD_P2
    dq, dk = skl.streamkl_bwd_sel(p1, p2, s["blocks"], c["bs"], s["kl"], s["lse1"], s["lse2"], s["dkl"], mode, **where)
    return dict(dq=dq, dk=dk)


def _counts(c):
    """(candidate blocks, keys seen in the selected ones) over all queries of the batch."""
    i = torch.arange(c["NQ"]) + c["NK"] - c["NQ"]
    nb = (c["NK"] + c["bs"] - 1) // c["bs"]
    hi = torch.clamp(i + 1, min=0) if c["causal"] else torch.full_like(i, c["NK"])
    blocks = keys = 0
    ids = _ids(c) if c["docs"] else [None] * c["B"]
    for row in ids:
        lo, top, ok = torch.zeros_like(i), hi, torch.ones_like(i, dtype=torch.bool)
        if row is not None:
            row = torch.tensor(row)
            ok = row >= 0
            lo = torch.searchsorted(torch.where(ok, row, 2 ** 30), row)
            top = torch.minimum(hi, torch.searchsorted(torch.where(ok, row, 2 ** 30), row, right=True))
        n = torch.where(ok & (top > lo), (top - 1) // c["bs"] - lo // c["bs"] + 1, 0)
        # all visible keys where every candidate is taken, else whole blocks but for the last one
        part = c["T"] * c["bs"] - (c["bs"] - 1 - (top - 1) % c["bs"])
        blocks += int(n.clamp(max=nb).sum())
        keys += int(torch.where(n <= c["T"], torch.where(ok, (top - lo).clamp(min=0), 0), part).sum())
    return blocks, keys


def work(case):
    c = case
    if c["op"] == "rotate":
        n = c["B"] * c["H"] * c["N"] * c["d"]
        return {"bytes": 4 * n + 4 * c["B"] * c["N"] * len(c["sections"].split(",")), "flops": 3 * n}
    if c["op"] == "pool":
        n = c["B"] * c["HK"] * c["d"]
        return {"bytes": 2 * n * (c["NK"] + -(-c["NK"] // c["bs"])), "flops": n * c["NK"]}
    blocks, keys = _counts(c)
    nb = -(-c["NK"] // c["bs"])
    rows = c["B"] * c["H"] * c["NQ"]
    idx = 4 * c["B"] * c["HK2"] * c["NQ"] * c["T"]
    if c["op"] == "select":
        return {"bytes": 2 * rows * c["d2"] + 2 * c["B"] * c["HK2"] * nb * c["d2"] + idx,
                "flops": 2 * c["HK2"] * blocks * c["d2"] + rows * c["d2"]}
    read = min(c["NK"], c["NQ"] * c["T"] * c["bs"])  # keys that some query can have selected
    pairs = c["H"] * keys
    q = rows * (c["d1"] + c["d2"]) * 2
    k = c["B"] * read * (c["HK1"] * c["d1"] + c["HK2"] * c["d2"]) * 2
    if c["op"] == "fwd":
        return {"bytes": q + k + idx + rows * 12, "flops": 2 * pairs * (c["d1"] + c["d2"])}
    dg, hkg = (c["d1"], c["HK1"]) if c["mode"] == "P1" else (c["d2"], c["HK2"])
    out = (rows + c["B"] * c["NK"] * hkg) * dg * 2
    return {"bytes": q + k + idx + rows * 16 + out, "flops": 2 * pairs * (c["d1"] + c["d2"]) + 4 * pairs * dg}


def exact(case, seed):
    """The definitions in 64 bits: rotations as complex numbers, selected keys
    gathered for each query."""
    c = case
    if c["op"] in ("fwd", "bwd") and c["B"] * c["H"] * c["NQ"] * c["T"] * c["bs"] * (c["d1"] + c["d2"]) > 1.6e11:
        return None
    s = prepare(case, seed)
    if c["op"] == "rotate":
        R = s["inv_freq"].shape[0]
        parts = [p.double() for p in s["x"][..., : 2 * R].unfold(3, 2, 2).unbind(4)] if c["interleaved"] else \
            [p.double() for p in s["x"][..., : 2 * R].split(R, 3)]
        turn, at = [], 0
        for a, n in enumerate(s["sections"]):
            turn.append(s["pos"][a].double()[..., None] * s["inv_freq"][at: at + n].double())
            at += n
        turn = torch.cat(turn, 2)[:, None]
        z = torch.complex(*parts) * torch.polar(torch.ones_like(turn), -turn if c["inverse"] else turn)
        pair = torch.stack((z.real, z.imag), 4).flatten(3) if c["interleaved"] else torch.cat((z.real, z.imag), 3)
        return torch.cat((pair, s["x"][..., 2 * R:].double()), 3)
    if c["op"] == "pool":
        k, out = s["k"].double(), []
        for j in range(0, c["NK"], c["bs"]):
            part = k[:, :, j: j + c["bs"]]
            keep = torch.ones(part.shape[0], part.shape[2], dtype=torch.bool, device=k.device) if s["doc"] is None \
                else s["doc"][:, j: j + c["bs"]] >= 0
            total = part.masked_fill(~keep[:, None, :, None], 0.0).sum(2)
            out.append(total / keep.sum(1).clamp(min=1)[:, None, None])
        return torch.stack(out, 2)
    dev, nq, nk, H, bs, T = s["q1"].device, c["NQ"], c["NK"], c["H"], c["bs"], c["T"]
    if c["op"] == "select":
        cand, hk = _candidates(s), c["HK2"]
        out = torch.full((c["B"], hk, nq, T), -1, dtype=torch.int32, device=dev)
        nb = cand.shape[2]
        place = torch.arange(nb, device=dev)
        for b in range(c["B"]):
            first = torch.where(cand[b], place, nb).sort(1)[0][:, : c["sink"]]
            last = torch.where(cand[b], place, -1).sort(1, descending=True)[0][:, : c["local"]]
            for h in range(hk):
                score = torch.zeros((nq, nb), dtype=torch.float64, device=dev)
                for m in range(h * (H // hk), (h + 1) * (H // hk)):
                    score += s["q2"][b, m].double() @ s["kb"][b, h].double().T
                key = torch.cat((score.masked_fill(~cand[b], -math.inf), torch.full((nq, 1), -math.inf, dtype=torch.float64,
                                                                                    device=dev)), 1)
                key.scatter_(1, first, math.inf)
                key.scatter_(1, torch.where(last >= 0, last, nb), math.inf)
                key[:, nb] = -math.inf
                taken = torch.zeros((nq, nb + 1), dtype=torch.bool, device=dev)
                for _ in range(min(T, nb)):
                    best = key.amax(1, keepdim=True)
                    j = torch.where(key == best, torch.arange(nb + 1, device=dev), nb + 1).amin(1, keepdim=True)
                    j = torch.where(best > -math.inf, j, nb)
                    taken.scatter_(1, j, True)
                    key.scatter_(1, j, -math.inf)
                taken = taken[:, :nb]
                at = taken.cumsum(1) - 1
                row, col = taken.nonzero(as_tuple=True)
                out[b, h, row, at[row, col]] = col.int()
        return out
    hs = s["blocks"].shape[1]
    t = c["mode"][1] if c["op"] == "bwd" else "2"
    kl = torch.zeros((c["B"], H, nq), dtype=torch.float64, device=dev)
    lse = {x: torch.empty_like(kl) for x in "12"}
    dq = torch.zeros(s["q" + t].shape, dtype=torch.float64, device=dev)
    dk = torch.zeros(s["k" + t].shape, dtype=torch.float64, device=dev)
    some = max(1, min(nq, 2 ** 25 // (T * bs * max(c["d1"], c["d2"]))))
    for b in range(c["B"]):
        for h in range(H):
            k = {x: s["k" + x][b, h // (H // c["HK" + x])].double() for x in "12"}
            q = {x: s["q" + x][b, h].double() for x in "12"}
            for i0 in range(0, nq, some):
                i = torch.arange(i0, min(nq, i0 + some), device=dev)
                idx = s["blocks"][b, h // (H // hs), i].long()
                j = (idx[:, :, None] * bs + torch.arange(bs, device=dev)).reshape(len(i), -1)
                see = (idx >= 0).repeat_interleave(bs, 1) & (j < nk)
                if c["causal"]:
                    see &= j <= i[:, None] + nk - nq
                j = j.clamp(0, nk - 1)
                if s["doc"] is not None:
                    see &= (s["doc"][b][j] == s["doc"][b][i][:, None]) & (s["doc"][b][i] >= 0)[:, None]
                y = {x: (k[x][j] @ q[x][i][:, :, None])[..., 0] * s["scale" + x] for x in "12"}
                if c["op"] == "fwd":
                    l1, l2 = (torch.logsumexp(y[x].masked_fill(~see, -math.inf), 1) for x in "12")
                    lse["1"][b, h, i], lse["2"][b, h, i] = l1, l2
                    p = torch.exp(y["1"] - l1[:, None])
                    kl[b, h, i] = (p * (y["1"] - y["2"] - (l1 - l2)[:, None])).masked_fill(~see, 0.0).sum(1)
                    continue
                l1, l2 = s["lse1"][b, h, i].double()[:, None], s["lse2"][b, h, i].double()[:, None]
                w, a = s["dkl"][b, h, i].double()[:, None], torch.exp(y["1"] - l1)
                ds = w * (torch.exp(y["2"] - l2) - a) if t == "2" else \
                    w * a * (y["1"] - l1 - y["2"] + l2 - s["kl"][b, h, i].double()[:, None])
                dx = s["scale" + t] * ds.masked_fill(~see, 0.0)
                dq[b, h, i] = (dx[:, None] @ k[t][j])[:, 0]
                dk[b, h // (H // c["HK" + t])].index_add_(0, j.flatten(), (dx[:, :, None] * q[t][i][:, None]).flatten(0, 1))
    return (kl, lse["1"], lse["2"]) if c["op"] == "fwd" else dict(dq=dq, dk=dk)
