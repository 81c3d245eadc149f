"""Cases for the attention KL over modified scores: capped by a tanh, biased by
distance (fixed slopes or a learned table of buckets), restricted to documents
or opened to a prefix; forward, backward into either side, and the gradient of
the learned table.

With r = j - i - (NK - NQ), per side: X = s q.k, Y = cap tanh(X / cap) (or X),
S = Y + bias_h(r), bias = -slope_h |r| or table[h, bucket(r)].  KL and the two
log-sum-exps per query row; rows that see no key have KL 0 and LSE -inf.
"""

import math
import random

import torch

own = False

NB, MAXD = 32, 128  # buckets of a learned table and the distance where they end


def _case(name, op, B, H, HK1, HK2, NQ, NK, d1, d2, **kw):
    c = dict(name=name, op=op, B=B, H=H, HK1=HK1, HK2=HK2, NQ=NQ, NK=NK, d1=d1, d2=d2, causal=True, prefix=False,
             docs=0, cap1=0.0, cap2=0.0, bias1="none", bias2="none", mode="", bshd=True)
    c.update(kw)
    return c


def listed():
    return [
        # one short prompt, both models capped: the smallest call, where latency counts
        _case("fwd short", "fwd", 1, 8, 8, 8, 256, 256, 64, 64, cap1=50.0, cap2=50.0),
        # a long sequence with grouped key heads, both models capped: the largest call
        _case("fwd long capped", "fwd", 1, 32, 8, 8, 8192, 8192, 128, 128, cap1=50.0, cap2=50.0),
        # sequences packed from documents with a padded tail; slopes on both sides, the student's head is half as wide
        _case("fwd packed slopes", "fwd", 2, 16, 16, 16, 4096, 4096, 128, 64, docs=12, bias1="slopes", bias2="slopes"),
        # an encoder pair with learned bidirectional buckets, odd length, padded batch
        _case("fwd encoder buckets", "fwd", 3, 12, 12, 12, 1531, 1531, 64, 64, causal=False, docs=1, bias1="both ways",
              bias2="both ways", bshd=False),
        # the last tokens of a long context: few rows, a long key axis
        _case("fwd few rows", "fwd", 1, 32, 8, 8, 16, 32768, 128, 128, cap1=50.0, cap2=30.0),
        # the smallest training call
        _case("bwd short", "bwd", 1, 8, 8, 8, 256, 256, 64, 64, cap1=50.0, cap2=50.0, mode="P2"),
        # a training step of a capped pair with grouped key heads: the largest backward
        _case("bwd long capped", "bwd", 1, 32, 8, 8, 4096, 4096, 128, 128, cap1=50.0, cap2=50.0, mode="P2"),
        # gradient into the first side over packed documents with slopes, odd length
        _case("bwd packed slopes P1", "bwd", 2, 16, 16, 16, 2111, 2111, 128, 64, docs=7, bias1="slopes",
              bias2="slopes", mode="P1"),
        # a prefix seen by all rows, a plain teacher and a capped student, head dim between tile widths
        _case("bwd prefix", "bwd", 2, 16, 4, 4, 2000, 2000, 96, 96, prefix=True, cap2=30.0, mode="P2", bshd=False),
        # a decoder's learned buckets: gradients of q, k and the table
        _case("bwd buckets", "bwd", 1, 16, 16, 16, 4096, 4096, 64, 64, bias1="one way", bias2="one way", mode="P2"),
        # an encoder's learned buckets in a padded batch of odd length
        _case("bwd encoder buckets", "bwd", 4, 12, 12, 12, 777, 777, 64, 64, causal=False, docs=1, bias1="both ways",
              bias2="both ways", mode="P2", bshd=False),
        # learned buckets and a cap on one side, gradient into the first side
        _case("bwd buckets capped P1", "bwd", 2, 8, 8, 4, 1000, 1300, 128, 128, cap1=50.0, bias1="one way",
              bias2="slopes", mode="P1"),
    ]


def draw(rng):
    op = rng.choice(["fwd", "bwd"])
    most = 32 * 8192 * 8192 if op == "fwd" else 32 * 4096 * 4096
    while True:
        nk = int(round(math.exp(rng.uniform(math.log(16), math.log(32768 if op == "fwd" else 8192)))))
        nq = nk if rng.random() < 0.6 else max(1, int(round(nk * math.exp(-rng.uniform(0.0, 6.0)))))
        hk = rng.choice([1, 2, 3, 4, 8])
        h = hk * rng.choice([1, 1, 2, 4])
        b = rng.choice([1, 1, 2, 3, 5])
        if b * h * nq * nk <= most:
            break
    d1 = 16 * rng.randint(2, 8)
    causal = rng.random() < 0.7
    docs = rng.choice([0, 0, 1, 5]) if nq == nk else 0
    bias = ["none", "none", "slopes", "one way" if causal else "both ways"]
    return dict(op=op, B=b, H=h, HK1=hk, HK2=rng.choice([hk, h]), NQ=nq, NK=nk, d1=d1,
                d2=rng.choice([d1, d1, 64, 128]), causal=causal, prefix=causal and rng.random() < 0.25, docs=docs,
                cap1=rng.choice([0.0, 30.0, 50.0]), cap2=rng.choice([0.0, 30.0, 50.0]), bias1=rng.choice(bias),
                bias2=rng.choice(bias), mode=rng.choice(["P1", "P2"]) if op == "bwd" else "", bshd=rng.random() < 0.5)


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


def _prefixes(c):
    rng = random.Random(77 * c["NK"] + c["B"])
    return [rng.randint(0, c["NK"] // 2) for _ in range(c["B"])]


def _slopes(h):
    return [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(n, h, d, sd):
        x = sd * torch.randn((c["B"], n, h, d), generator=g, device=dev) if c["bshd"] else \
            sd * torch.randn((c["B"], h, n, d), generator=g, device=dev)
        return x

    def lay(x):  # [B, H, N, d]; a view of [B, N, H, d] where that is how the projection left it
        x = x.to(torch.bfloat16)
        return x.transpose(1, 2) if c["bshd"] else x

    q1, k1 = rand(c["NQ"], c["H"], c["d1"], 1.6), rand(c["NK"], c["HK1"], c["d1"], 1.6)
    if (c["d1"], c["HK1"]) == (c["d2"], c["HK2"]):  # a student that has come near its teacher
        q2 = q1 + 0.3 * rand(c["NQ"], c["H"], c["d2"], 1.0)
        k2 = k1 + 0.3 * rand(c["NK"], c["HK2"], c["d2"], 1.0)
    else:
        q2, k2 = rand(c["NQ"], c["H"], c["d2"], 1.3), rand(c["NK"], c["HK2"], c["d2"], 1.3)
    s = dict(case=c, q1=lay(q1), k1=lay(k1), q2=lay(q2), k2=lay(k2), doc=None, prefix=None)
    if c["docs"]:
        s["doc"] = torch.tensor(_ids(c), dtype=torch.int32, device=dev)
    if c["prefix"]:
        s["prefix"] = torch.tensor(_prefixes(c), dtype=torch.int32, device=dev)
    for t in "12":
        kind = c["bias" + t]
        s["slopes" + t] = torch.tensor(_slopes(c["H"]), dtype=torch.float32, device=dev) if kind == "slopes" else None
        s["table" + t] = torch.randn((c["H"], NB), generator=g, device=dev) if "way" in kind else None
        s["scale" + t] = 1.0 / math.sqrt(c["d" + t])
    if c["op"] == "bwd":  # what the forward left, and the loss's gradient per row
        s["kl"], s["lse1"], s["lse2"] = _plain_fwd(s)
        s["dkl"] = torch.rand((c["B"], c["H"], c["NQ"]), generator=g, device=dev) + 0.5
    return s


def _bucket(r, both):
    """Bucket of the relative position r: half of the buckets for each
    direction where both count, the near half one distance each, the rest in
    steps of the logarithm up to MAXD.  In 64 bits: borders are whole distances."""
    n = NB // 2 if both else NB
    base = torch.where(r > 0, n, 0) if both else torch.zeros_like(r)
    d = r.abs() if both else (-r).clamp(min=0)
    e = n // 2
    far = e + torch.floor((n - e) * torch.log(d.clamp(min=1).double() / e) / math.log(MAXD / e) + 1e-9).long()
    return base + torch.where(d < e, d, far.clamp(max=n - 1))


def _relative(c, dev):
    i = torch.arange(c["NQ"], device=dev)[:, None] + (c["NK"] - c["NQ"])
    return torch.arange(c["NK"], device=dev)[None, :] - i


def _plain_visible(s):
    c, dev = s["case"], s["q1"].device
    r = _relative(c, dev)
    vis = (r <= 0) if c["causal"] else torch.ones_like(r, dtype=torch.bool)
    vis = vis[None]
    if s["prefix"] is not None:
        vis = vis | (torch.arange(c["NK"], device=dev)[None, None, :] < s["prefix"][:, None, None])
    if s["doc"] is not None:
        q, k = s["doc"][:, :, None], s["doc"][:, None, :]
        vis = vis & (q == k) & (q >= 0)
    return vis[:, None]


def _plain_scores(s, t):
    """(S, tanh(X / cap) or None) of side t, [B, H, NQ, NK], 32 bits."""
    c = s["case"]
    q, k = s["q" + t].float(), s["k" + t].float()
    hk = k.shape[1]
    x = torch.matmul(q.reshape(c["B"], hk, -1, c["NQ"], q.shape[3]), k[:, :, None].transpose(3, 4))
    x = x.reshape(c["B"], c["H"], c["NQ"], c["NK"]) * s["scale" + t]
    cap, th = c["cap" + t], None
    if cap:
        th = torch.tanh(x / cap)
        x = cap * th
    r = _relative(c, q.device)
    if s["slopes" + t] is not None:
        x = x - s["slopes" + t][:, None, None] * r.abs()
    if s["table" + t] is not None:
        x = x + s["table" + t][:, _bucket(r, c["bias" + t] == "both ways")]
    return x, th


def _plain_lse(x):
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    return torch.log(torch.exp(x - m).sum(-1)) + m[..., 0]


def _plain_fwd(s):
    vis = _plain_visible(s)
    x1 = _plain_scores(s, "1")[0].masked_fill(~vis, -math.inf)
    lse1 = _plain_lse(x1)
    lp1 = x1 - lse1[..., None]
    x2 = _plain_scores(s, "2")[0].masked_fill(~vis, -math.inf)
    lse2 = _plain_lse(x2)
    lp2 = x2 - lse2[..., None]
    kl = torch.where(vis, torch.exp(lp1) * (lp1 - lp2), 0.0).sum(-1)
    return kl, lse1, lse2


def _plain_bwd(s):
    c = s["case"]
    vis, t = _plain_visible(s), c["mode"][1]
    (x1, th1), (x2, th2) = _plain_scores(s, "1"), _plain_scores(s, "2")
    lp1, lp2 = x1 - s["lse1"][..., None], x2 - s["lse2"][..., None]
    if t == "2":
        ds = torch.exp(lp2) - torch.exp(lp1)
    else:
        ds = torch.exp(lp1) * (lp1 - lp2 - s["kl"][..., None])
    ds = torch.where(vis, s["dkl"][..., None] * ds, 0.0)
    th = th1 if t == "1" else th2
    dx = s["scale" + t] * (ds if th is None else ds * (1 - th * th))
    q, k = s["q" + t].float(), s["k" + t].float()
    hk, d = k.shape[1], k.shape[3]
    dx = dx.reshape(c["B"], hk, -1, c["NQ"], c["NK"])
    dq = torch.matmul(dx, k[:, :, None]).reshape(c["B"], c["H"], c["NQ"], d)
    dk = torch.matmul(dx.transpose(3, 4), q.reshape(c["B"], hk, -1, c["NQ"], d)).sum(2)
    out = dict(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16))
    if s["table" + t] is not None:
        # sums along the diagonals (one per relative position): rows from the last to the first, each one place further
        # to the right than the one before
        nq, nk = c["NQ"], c["NK"]
        flat = torch.nn.functional.pad(ds.sum(0).flip(1), (0, nq)).reshape(c["H"], -1)[:, : nq * (nk + nq - 1)]
        per_r = flat.reshape(c["H"], nq, nk + nq - 1).sum(1, dtype=torch.float64)
        r = torch.arange(nk + nq - 1, device=q.device) - (nq - 1) - (nk - nq)
        table = torch.zeros((c["H"], NB), dtype=torch.float64, device=q.device)
        out["dtable"] = table.index_add_(1, _bucket(r, c["bias" + t] == "both ways"), per_r).float()
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_fwd(s) if c["op"] == "fwd" else _plain_bwd(s)
    import attention_distillation_kl_gb300 as skl
    p1, p2 = (skl.AttnSide(s["q" + t], s["k" + t], s["scale" + t], softcap=c["cap" + t], slopes=s["slopes" + t],
                           table=s["table" + t], max_distance=MAXD, bidirectional=c["bias" + t] == "both ways")
              for t in "12")
    where = dict(causal=c["causal"], prefix=s["prefix"], doc_q=s["doc"], doc_k=s["doc"])
    if c["op"] == "fwd":
        return skl.streamkl_fwd_mod(p1, p2, **where)
    mode = skl.STREAMKL_GRAD_P1 if c["mode"] == "P1" else skl.STREAMKL_GRAD_P2
    dq, dk, dtable = skl.streamkl_bwd_mod(p1, p2, s["kl"], s["lse1"], s["lse2"], s["dkl"], mode, **where)
    return dict(dq=dq, dk=dk) if dtable is None else dict(dq=dq, dk=dk, dtable=dtable)


def work(case):
    c = case
    r = torch.arange(c["NK"])[None, :] - torch.arange(c["NQ"])[:, None] - (c["NK"] - c["NQ"])
    pairs = 0
    ids = torch.tensor(_ids(c)) if c["docs"] else None
    pre = _prefixes(c) if c["prefix"] else None
    for b in range(c["B"]):
        vis = (r <= 0) if c["causal"] else torch.ones_like(r, dtype=torch.bool)
        if pre:
            vis[:, : pre[b]] = True
        if ids is not None:
            vis &= (ids[b][:, None] == ids[b][None, :]) & (ids[b] >= 0)[:, None]
        pairs += int(vis.sum()) * c["H"]
    dg, hkg = (c["d1"], c["HK1"]) if c["mode"] == "P1" else (c["d2"], c["HK2"])
    rows = c["B"] * c["H"] * c["NQ"]
    q = rows * (c["d1"] + c["d2"]) * 2
    k = c["B"] * c["NK"] * (c["HK1"] * c["d1"] + c["HK2"] * c["d2"]) * 2
    if c["op"] == "fwd":
        return {"bytes": q + k + rows * 12, "flops": 2 * pairs * (c["d1"] + c["d2"])}
    out = (rows + c["B"] * c["NK"] * hkg) * dg * 2
    return {"bytes": q + k + rows * 16 + out, "flops": 2 * pairs * (c["d1"] + c["d2"]) + 4 * pairs * dg}


def exact(case, seed):
    """The definitions in 64 bits, one head at a time."""
    c = case
    if c["B"] * c["H"] * c["NQ"] * c["NK"] > 3e9:
        return None
    s = prepare(case, seed)
    dev = s["q1"].device
    B, H, NQ, NK = c["B"], c["H"], c["NQ"], c["NK"]
    pos_q = torch.arange(NQ, device=dev) + NK - NQ
    pos_k = torch.arange(NK, device=dev)
    dist = pos_q[:, None] - pos_k[None, :]  # how far the key lies behind the query

    def edges(n):  # the first distance of each bucket but the first
        e = n // 2
        return torch.tensor([i if i <= e else e * (MAXD / e) ** ((i - e) / (n - e)) for i in range(1, n)],
                            dtype=torch.float64, device=dev)

    def find(dist, both):
        n = NB // 2 if both else NB
        d = dist.abs() if both else dist.clamp(min=0)
        idx = torch.searchsorted(edges(n) * (1 - 1e-12), d.double(), right=True)
        return torch.where(dist < 0, idx + n, idx) if both else idx

    bias_index = {t: find(dist, c["bias" + t] == "both ways") for t in "12" if s["table" + t] is not None}

    def score(t, b, h):
        q, k = s["q" + t][b, h].double(), s["k" + t][b, h // (H // c["HK" + t])].double()
        y = q @ k.T * s["scale" + t]
        grad = None
        if c["cap" + t]:
            th = torch.tanh(y / c["cap" + t])
            y, grad = c["cap" + t] * th, 1 - th.square()
        if s["slopes" + t] is not None:
            y = y - s["slopes" + t][h].double() * dist.abs()
        if t in bias_index:
            y = y + s["table" + t][h].double()[bias_index[t]]
        return y, grad

    kl = torch.zeros((B, H, NQ), dtype=torch.float64, device=dev)
    lse = {t: torch.empty_like(kl) for t in "12"}
    t = c["mode"][1] if c["op"] == "bwd" else "2"
    dq = torch.empty((B, H, NQ, c["d" + t]), dtype=torch.float64, device=dev)
    dk = torch.zeros((B, c["HK" + t], NK, c["d" + t]), dtype=torch.float64, device=dev)
    dtable = torch.zeros((H, NB), dtype=torch.float64, device=dev)
    for b in range(B):
        see = dist >= 0 if c["causal"] else torch.ones_like(dist, dtype=torch.bool)
        if s["prefix"] is not None:
            see = see | (pos_k < s["prefix"][b])[None, :]
        if s["doc"] is not None:
            see = see & (s["doc"][b][:, None] == s["doc"][b][None, :]) & (s["doc"][b] >= 0)[:, None]
        hide = ~see
        for h in range(H):
            (y1, g1), (y2, g2) = score("1", b, h), score("2", b, h)
            if c["op"] == "fwd":
                l1 = torch.logsumexp(y1.masked_fill(hide, -math.inf), 1)
                l2 = torch.logsumexp(y2.masked_fill(hide, -math.inf), 1)
                lse["1"][b, h], lse["2"][b, h] = l1, l2
                p = torch.exp(y1 - l1[:, None])
                kl[b, h] = (p * (y1 - y2 - (l1 - l2)[:, None])).masked_fill(hide, 0.0).sum(1)
                continue
            l1, l2 = s["lse1"][b, h].double()[:, None], s["lse2"][b, h].double()[:, None]
            w, a = s["dkl"][b, h].double()[:, None], torch.exp(y1 - l1)
            ds = w * (torch.exp(y2 - l2) - a) if t == "2" else w * a * (y1 - l1 - y2 + l2 - s["kl"][b, h].double()[:, None])
            ds = ds.masked_fill(hide, 0.0)
            if t in bias_index:
                dtable[h] += torch.stack([(ds * (bias_index[t] == i)).sum() for i in range(NB)])
            g = g2 if t == "2" else g1
            dx = s["scale" + t] * (ds if g is None else ds * g)
            hk = h // (H // c["HK" + t])
            dq[b, h] = dx @ s["k" + t][b, hk].double()
            dk[b, hk] += dx.T @ s["q" + t][b, h].double()
    if c["op"] == "fwd":
        return kl, lse["1"], lse["2"]
    return dict(dq=dq, dk=dk, dtable=dtable) if t in bias_index else dict(dq=dq, dk=dk)
