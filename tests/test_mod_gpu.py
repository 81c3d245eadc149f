"""The attention KL over modified scores on the GPU against the float64
definitions (mod_reference.py), element by element within bounds derived from
the roundings each path makes: bf16 products summed in fp32, the polynomial or
the quotient of the cap, ex2 at two units, dX rounded to bf16 before its two
products, one rounding of dq and dk.  Plus the forms of the call: splits,
deterministic mode, strides, another stream, graphs, padded rows."""

import math

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl
import mod_reference as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def slopes(h):
    return [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]


def problem(seed=0, B=1, H=2, HK1=None, HK2=None, NQ=150, NK=150, d1=64, d2=64, sd=1.5, causal=True, prefix=None,
            docs=None, cap1=0.0, cap2=0.0, bias1=None, bias2=None, nb=32, maxd=128, bshd=False, scale1=None,
            scale2=None, tsd=1.0):
    """(device arguments, float64 problem).  docs: None, or "packed",
    "shuffled" (ids in no order, with padding), "apart" (no query shares an id)."""
    g = torch.Generator().manual_seed(seed)
    HK1, HK2 = HK1 or H, HK2 or H

    def x(h, n, d):
        t = (sd * torch.randn((B, h, n, d), generator=g)).to(torch.bfloat16)
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if bshd else t.cuda()

    dev = dict(q1=x(H, NQ, d1), k1=x(HK1, NK, d1), q2=x(H, NQ, d2), k2=x(HK2, NK, d2))
    p = {k: f64(v) for k, v in dev.items()}
    kw = {}
    for t, d, cap, bias, sc in (("1", d1, cap1, bias1, scale1), ("2", d2, cap2, bias2, scale2)):
        sl = torch.tensor(slopes(H), dtype=torch.float32) if bias == "slopes" else None
        tab = tsd * torch.randn((H, nb), generator=g) if bias in ("one way", "both ways") else None
        sc = 1.0 / math.sqrt(d) if sc is None else sc
        kw[t] = dict(scale=sc, softcap=cap, slopes=None if sl is None else sl.cuda(),
                     table=None if tab is None else tab.cuda(), max_distance=maxd, bidirectional=bias == "both ways")
        p.update({"scale" + t: np.float64(sc), "cap" + t: cap, "slopes" + t: f64(sl), "table" + t: f64(tab),
                  "maxd" + t: maxd, "both" + t: bias == "both ways"})
    ids = None
    if docs is not None:
        if docs == "packed":
            q = torch.sort(torch.randint(0, 4, (B, NQ), generator=g), dim=1)[0]
            k = q if NQ == NK else torch.sort(torch.randint(0, 4, (B, NK), generator=g), dim=1)[0]
            q, k = q.clone(), k.clone()
            q[:, NQ - NQ // 9:] = -1
            k[:, NK - NK // 9:] = -1
        elif docs == "shuffled":
            q = torch.randint(-2, 6, (B, NQ), generator=g)
            k = torch.randint(-2, 6, (B, NK), generator=g)
        else:
            q, k = torch.zeros(B, NQ, dtype=torch.int64), torch.ones(B, NK, dtype=torch.int64)
        ids = q.int().cuda(), k.int().cuda()
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda()
    p.update(causal=causal, prefix=None if prefix is None else np.array(prefix),
             doc_q=None if ids is None else ids[0].cpu().numpy(), doc_k=None if ids is None else ids[1].cpu().numpy())
    where = dict(causal=causal, prefix=pre, doc_q=None if ids is None else ids[0], doc_k=None if ids is None else ids[1])
    return dev, kw, where, p


def sides(dev, kw):
    return (skl.AttnSide(dev["q1"], dev["k1"], **kw["1"]), skl.AttnSide(dev["q2"], dev["k2"], **kw["2"]))


def within(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    same = np.isinf(want) & (got == want)
    err = np.abs(np.where(same, 0.0, got) - np.where(same, 0.0, want))
    assert np.all(np.isfinite(err)), f"{what}: not finite where the definition is"
    over = err - bound - 1e-30
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what} at {at}: {got[at]} for {want[at]}, error {err[at]:.3g}, bound {bound[at]:.3g}"


def check_forward(p1, p2, where, p, **kw):
    got = skl.streamkl_fwd_mod(p1, p2, **where, **kw)
    torch.cuda.synchronize()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    want = ref.forward(p)
    for g, w, b, what in zip(got, want[:3], want[3:], ("KL", "LSE1", "LSE2")):
        within(g, w, b, what)
    return got


def check_backward(p1, p2, where, p, rows, mode, seed=1, **kw):
    """rows: kl, lse1, lse2 as the kernel gets them."""
    g = torch.Generator().manual_seed(seed)
    dkl = (torch.rand(rows[0].shape, generator=g) * 2 - 0.5).cuda()
    got = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2,
                               **where, **kw)
    torch.cuda.synchronize()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    want = list(ref.backward(p, *(f64(t) for t in rows), f64(dkl), mode))
    if kw.get("deterministic"):
        want[3] = want[3] + (1 + ref.BF16) * ref.grid_error(p, f64(rows[0]), f64(dkl), mode)
    for g_, w, b, what in zip(got, want[:3], want[3:], ("dq", "dk", "dtable")):
        if w is None:
            assert g_ is None, what
        else:
            within(g_, w, b, f"mode P{mode} {what}")
    return got, dkl


CASES = {
    "plain": dict(),
    "one token": dict(NQ=1, NK=1, H=1, cap1=30.0),
    "one row": dict(NQ=1, NK=300, cap1=30.0, bias2="slopes"),
    "one tile": dict(NQ=128, NK=128, cap1=50.0, cap2=30.0),
    "one past a tile": dict(NQ=129, NK=129, cap2=30.0, bias1="slopes"),
    "capped": dict(cap1=50.0, cap2=30.0, NQ=260, NK=260),
    "one side capped": dict(cap1=20.0, d1=128, NQ=200, NK=333),
    "other side capped": dict(cap2=20.0, d2=128, causal=False),
    "beyond half the cap": dict(cap1=4.0, cap2=6.0, NQ=260, NK=260, sd=2.5),
    "saturated": dict(cap1=0.5, cap2=0.25, sd=4.0, scale1=1.0, scale2=2.0),
    "a huge cap": dict(cap1=1e6, cap2=1e5, scale1=1e-4, scale2=1e-3),
    "slopes": dict(bias1="slopes", bias2="slopes", NQ=400, NK=400, H=4),
    "slopes both directions": dict(bias1="slopes", causal=False, NQ=300, NK=300),
    "steep slopes, long": dict(bias1="slopes", bias2="slopes", NQ=64, NK=1500, H=1, causal=False),
    "table one way": dict(bias1="one way", bias2="one way", NQ=500, NK=500, cap1=30.0),
    "table both ways": dict(bias1="both ways", bias2="both ways", NQ=500, NK=420, causal=False),
    "table and slopes": dict(bias1="slopes", bias2="one way", NQ=300, NK=390, cap2=30.0),
    "small table": dict(bias2="both ways", nb=4, maxd=2, NQ=150, NK=150, causal=False),
    "largest table": dict(bias2="one way", nb=64, maxd=4096, NQ=200, NK=200),
    "far table": dict(bias2="both ways", nb=64, maxd=300, NQ=700, NK=700, causal=False, H=1),
    "odd buckets": dict(bias2="one way", nb=7, maxd=11, NQ=200, NK=200, bias1="one way"),
    "grouped": dict(H=4, HK1=2, HK2=1, cap1=30.0, NQ=140, NK=260),
    "grouped table": dict(H=6, HK1=3, HK2=2, bias1="one way", bias2="one way", NQ=140, NK=140, B=2),
    "few rows of shared heads": dict(H=16, HK1=2, HK2=1, NQ=16, NK=400, cap1=30.0, bias2="one way", B=2),
    "one row of shared heads": dict(H=8, HK1=2, HK2=2, NQ=1, NK=700, bias1="slopes", bias2="slopes", d1=128),
    "33 rows of shared heads": dict(H=4, HK1=1, HK2=1, NQ=33, NK=300, causal=False, bias1="both ways", bias2="slopes"),
    "17 rows of packed shared heads": dict(H=8, HK1=2, HK2=1, NQ=17, NK=260, docs="shuffled", cap2=30.0, B=2),
    "narrow heads": dict(d1=16, d2=48, cap1=30.0, cap2=30.0),
    "padded heads": dict(d1=80, d2=112, bias2="one way"),
    "wide and narrow": dict(d1=128, d2=32, cap2=10.0),
    "128": dict(d1=128, d2=128, cap1=50.0, cap2=50.0, NQ=300, NK=300),
    "more rows than keys": dict(NQ=300, NK=170, cap1=30.0),
    "no causal row sees": dict(NQ=300, NK=1),
    "prefix": dict(B=3, prefix=[0, 70, 149], cap2=30.0),
    "prefix past the end": dict(B=3, prefix=[-5, 1000, 1], NQ=150, NK=220, bias1="slopes", bias2="one way"),
    "prefix over many tiles": dict(B=2, prefix=[300, 20], NQ=420, NK=420, H=1, bias2="one way"),
    "packed": dict(B=2, docs="packed", NQ=400, NK=400, cap1=30.0),
    "packed slopes": dict(B=2, docs="packed", NQ=400, NK=400, bias1="slopes", bias2="slopes"),
    "shuffled ids": dict(B=2, docs="shuffled", NQ=260, NK=300, causal=False, bias2="both ways"),
    "shuffled ids, causal": dict(B=2, docs="shuffled", NQ=260, NK=300, cap2=30.0),
    "ids and a prefix": dict(B=2, docs="packed", NQ=260, NK=260, prefix=[100, 10]),
    "nothing shared": dict(docs="apart", NQ=200, NK=200, causal=False, cap1=30.0, bias2="both ways"),
    "strided": dict(bshd=True, B=2, H=4, HK1=2, HK2=4, NQ=200, NK=200, cap1=30.0, bias2="one way"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    dev, kw, where, p = problem(seed=len(name), **CASES[name])
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64, 0])
@pytest.mark.parametrize("name", ["one row", "few rows of shared heads", "slopes", "shuffled ids", "prefix over many tiles", "nothing shared",
                                  "more rows than keys"])
def test_key_splits(name, splits):
    dev, kw, where, p = problem(seed=3, **CASES[name])
    check_forward(*sides(dev, kw), where, p, num_splits=splits)


@pytest.mark.parametrize("mode", "12")
@pytest.mark.parametrize("name", ["grouped table", "packed slopes", "128", "strided", "table both ways", "nothing shared"])
def test_deterministic(name, mode):
    dev, kw, where, p = problem(seed=4, **CASES[name])
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    one, dkl = check_backward(p1, p2, where, p, rows, mode, deterministic=True)
    m = skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2
    for _ in range(3):
        two = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, m, **where, deterministic=True)
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(one, two))


def test_the_tables_gradient_is_repeatable():
    dev, kw, where, p = problem(seed=5, NQ=900, NK=900, H=3, B=2, bias2="both ways", causal=False)
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    one = skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), **where)[2]
    for _ in range(3):
        assert torch.equal(one, skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), **where)[2])


def test_a_frozen_table_gets_no_gradient():
    dev, kw, where, p = problem(seed=5, bias2="one way")
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    dkl = torch.ones_like(rows[0])
    a = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True)
    b = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True, table_grad=False)
    assert b[2] is None
    # the two kernels weigh the exponentials in another order: dX may round to its neighbour
    want = ref.backward(p, *(f64(t) for t in rows), f64(dkl), "2")
    grid = (1 + ref.BF16) * ref.grid_error(p, f64(rows[0]), f64(dkl), "2")
    for x in (a, b):
        within(x[0], want[0], want[3] + grid, "dq")
        within(x[1], want[1], want[4], "dk")


def test_plain_scores_agree_with_the_plain_call():
    """No modification: the same function as streamkl_fwd and streamkl_bwd."""
    dev, kw, where, p = problem(seed=6, NQ=300, NK=340)
    p1, p2 = sides(dev, kw)
    got = check_forward(p1, p2, where, p)
    old = skl.streamkl_fwd(dev["q1"], dev["k1"], dev["q2"], dev["k2"], kw["1"]["scale"], True)
    want = ref.forward(p)
    for a, b, e in zip(got, old, want[3:]):
        assert np.all(np.abs(f64(a) - f64(b)) <= 2 * e + 1e-4 * np.abs(f64(b)))


@pytest.mark.parametrize("lowest", [-3.4028234663852886e38, -1e30, -1e9])
def test_a_table_as_a_window(lowest):
    """Far buckets at the type's lowest value: keys there count for nothing,
    and a first tile that holds only such keys must not spoil the later ones."""
    dev, kw, where, p = problem(seed=7, NQ=500, NK=500, H=1, bias1="one way", bias2="one way")
    for t in "12":
        kw[t]["table"][:, -1] = lowest
        p["table" + t][:, -1] = np.float64(np.float32(lowest))
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    check_backward(p1, p2, where, p, rows, "2")
    # the other order: only the last rows' near keys are low
    for t in "12":
        kw[t]["table"][:, -1] = 0.5
        kw[t]["table"][:, :8] = lowest
        p["table" + t][:, -1] = 0.5
        p["table" + t][:, :8] = np.float64(np.float32(lowest))
    rows = check_forward(p1, p2, where, p)
    check_backward(p1, p2, where, p, rows, "1")


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_padded_positions_may_hold_anything(junk):
    dev, kw, where, p = problem(seed=8, B=2, docs="packed", NQ=400, NK=400, cap1=30.0, bias2="one way", bshd=True)
    p1, p2 = sides(dev, kw)
    clean = check_forward(p1, p2, where, p)
    pad = where["doc_q"] < 0
    for name in ("q1", "k1", "q2", "k2"):
        dev[name].transpose(1, 2)[pad] = junk
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    for a, b in zip(rows, clean):
        assert torch.equal(a, b)
    for mode, det in (("1", False), ("2", False), ("1", True), ("2", True)):
        dkl = torch.ones_like(rows[0])
        dkl.transpose(1, 2)[pad] = junk
        got = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2,
                                   **where, deterministic=det)
        want = list(ref.backward(p, *(f64(t) for t in rows), np.ones(rows[0].shape), mode))
        if det:
            want[3] = want[3] + (1 + ref.BF16) * ref.grid_error(p, f64(rows[0]), np.ones(rows[0].shape), mode)
        for g, w, b, what in zip(got, want[:3], want[3:], ("dq", "dk", "dtable")):
            if w is not None:
                within(g, w, b, what)
        assert torch.all(got[0].transpose(1, 2)[pad] == 0) and torch.all(got[1].transpose(1, 2)[pad] == 0)


def test_nan_in_a_masked_future_key_does_not_reach_the_forward():
    dev, kw, where, p = problem(seed=9, NQ=200, NK=200, cap2=30.0)
    p1, p2 = sides(dev, kw)
    clean = skl.streamkl_fwd_mod(p1, p2, **where)
    dev["k1"][:, :, 150:] = float("nan")
    dev["k2"][:, :, 150:] = float("inf")
    got = skl.streamkl_fwd_mod(p1, p2, **where)
    for a, b in zip(got, clean):
        assert torch.equal(a[:, :, :150], b[:, :, :150])
        assert torch.all(torch.isnan(a[:, :, 150:]))


@pytest.mark.parametrize("where_nan", ["q1", "q2"])
def test_a_query_of_nans_gives_nan(where_nan):
    """Not the values of a row that sees nothing.  The other rows of its warp
    take the general path too, so they keep to the definition, not to the bits."""
    dev, kw, where, p = problem(seed=15, NQ=200, NK=200, cap1=30.0, bias2="one way")
    p1, p2 = sides(dev, kw)
    want = ref.forward(p)
    dev[where_nan][:, :, 140] = float("nan")
    got = skl.streamkl_fwd_mod(p1, p2, **where)
    keep = np.arange(200) != 140
    for i, (a, w, e) in enumerate(zip(got, want[:3], want[3:])):
        within(f64(a)[:, :, keep], w[:, :, keep], e[:, :, keep], ("KL", "LSE1", "LSE2")[i])
        if i == 0 or where_nan == f"q{i}":
            assert torch.all(torch.isnan(a[:, :, 140]))


def test_empty_rows_and_no_rows():
    dev, kw, where, p = problem(seed=10, docs="apart", causal=False, bias2="one way", H=4, HK2=2)
    p1, p2 = sides(dev, kw)
    kl, l1, l2 = skl.streamkl_fwd_mod(p1, p2, **where)
    assert torch.all(kl == 0) and torch.all(l1 == -math.inf) and torch.all(l2 == -math.inf)
    for det in (False, True):
        dq, dk, dt = skl.streamkl_bwd_mod(p1, p2, kl, l1, l2, torch.ones_like(kl), **where, deterministic=det)
        assert not dq.any() and not dk.any() and not dt.any()
    none = skl.AttnSide(dev["q2"][:, :, :0], dev["k2"], **kw["2"])
    other = skl.AttnSide(dev["q1"][:, :, :0], dev["k1"], **kw["1"])
    kl, l1, l2 = skl.streamkl_fwd_mod(other, none)
    assert kl.shape == (1, 4, 0)
    dk = torch.full_like(dev["k2"], 7.0)
    dq, dk, dt = skl.streamkl_bwd_mod(other, none, kl, l1, l2, kl, dk=dk)
    assert not dk.any() and not dt.any() and dq.shape[2] == 0


def test_outputs_given_with_strides():
    dev, kw, where, p = problem(seed=11, B=2, H=4, HK1=2, HK2=2, NQ=140, NK=170, d2=48, bias2="one way")
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    dkl = torch.ones_like(rows[0])
    want = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True)
    big_q = torch.full((2, 140, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    big_k = torch.full((2, 170, 2, 56), 3.0, dtype=torch.bfloat16, device="cuda")
    dt = torch.empty((4, 32), device="cuda")
    got = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True, dtable=dt,
                               dq=big_q.transpose(1, 2)[..., :48], dk=big_k.transpose(1, 2)[..., 8:])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[2] is dt
    assert torch.all(big_q[..., 48:] == 3) and torch.all(big_k[..., :8] == 3)


def test_refused_tensors():
    dev, kw, where, p = problem(seed=12)
    p1, p2 = sides(dev, kw)
    q = dev["q1"]
    with pytest.raises(TypeError):
        skl.AttnSide(q.float(), dev["k1"], 0.1)
    with pytest.raises(ValueError):
        skl.AttnSide(q.transpose(2, 3), dev["k1"], 0.1)
    with pytest.raises(ValueError):
        skl.AttnSide(q, dev["k1"][..., :32], 0.1)
    with pytest.raises(ValueError):
        skl.AttnSide(q, dev["k1"], 0.1, slopes=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        skl.AttnSide(q, dev["k1"], 0.1, table=torch.ones((2, 32), device="cuda", dtype=torch.bfloat16))
    ones = torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in (dict(prefix=ones), dict(causal=True, prefix=ones.long()), dict(doc_q=where["doc_q"], doc_k=ones),
                dict(causal=True, prefix=torch.ones(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, skl.StreamKLError)):
            skl.streamkl_fwd_mod(p1, p2, **bad)
    with pytest.raises(skl.StreamKLError):  # heads broadcast by a stride of 0
        one = dev["k1"][:, :1].expand(-1, 2, -1, -1)
        skl.streamkl_fwd_mod(skl.AttnSide(q, one, 0.1), p2)
    with pytest.raises(skl.StreamKLError):  # rows at odd offsets
        skl.streamkl_fwd_mod(skl.AttnSide(torch.zeros(1, 2, 150, 68, device="cuda", dtype=torch.bfloat16)[..., :64],
                                          dev["k1"], 0.1), p2)
    with pytest.raises(ValueError):
        skl.streamkl_bwd_mod(p1, p2, *[torch.zeros(1, 2, 150, device="cuda")] * 4, dtable=torch.zeros(2, 32, device="cuda"))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(skl.StreamKLError):
        skl.streamkl_bwd_mod(p1, p2, *[torch.zeros(1, 2, 150, device="cuda")] * 4, workspace=small)


def test_graphs_and_streams():
    """Two graphs with a workspace each, replayed at once with changed inputs,
    and calls on another stream."""
    calls = []
    for seed, case in ((13, CASES["packed"]), (14, CASES["table one way"])):
        dev, kw, where, p = problem(seed=seed, **case)
        p1, p2 = sides(dev, kw)
        need = skl.streamkl_fwd_mod_workspace_bytes(p1, p2, **where)
        assert need > 0
        need = max(need, skl.streamkl_bwd_mod_workspace_bytes(p1, p2, **where, deterministic=True))
        calls.append((dev, p1, p2, where, p, torch.empty(need, dtype=torch.uint8, device="cuda")))

    def step(c):
        rows = skl.streamkl_fwd_mod(c[1], c[2], **c[3], workspace=c[5])
        return rows + skl.streamkl_bwd_mod(c[1], c[2], *rows, torch.ones_like(rows[0]), **c[3], workspace=c[5],
                                           deterministic=True)

    for c in calls:
        step(c)
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    for c in calls:  # new values in place
        c[0]["q1"].mul_(0.5)
    want = [[None if t is None else t.clone() for t in step(c)] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(a is None or torch.equal(a, b) for a, b in zip(o, w))
    # eager calls handed another stream: workspace and outputs made here
    for c, s, w in zip(calls, streams, want):
        s.wait_stream(torch.cuda.current_stream())
        rows = skl.streamkl_fwd_mod(c[1], c[2], **c[3], stream=s)
        with torch.cuda.stream(s):
            one = torch.ones_like(rows[0])
        got = rows + skl.streamkl_bwd_mod(c[1], c[2], *rows, one, **c[3], stream=s, deterministic=True)
        s.synchronize()
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, w))
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK


@pytest.mark.parametrize("seed", range(12))
def test_drawn(seed):
    """Sizes, masks and modifications drawn together."""
    r = np.random.default_rng(1000 + seed)
    hk = int(r.integers(1, 4))
    causal = bool(r.integers(0, 2))
    nk = int(r.integers(1, 500))
    kinds = [None, "slopes", "one way", "both ways"]
    B = int(r.integers(1, 3))
    case = dict(B=B, H=hk * int(r.integers(1, 4)), HK1=hk, NQ=int(r.integers(1, 500)), NK=nk, causal=causal,
                d1=16 * int(r.integers(1, 9)), d2=16 * int(r.integers(1, 9)),
                prefix=[int(r.integers(0, nk + 1)) for _ in range(B)] if causal and r.integers(0, 2) else None,
                docs=[None, "packed", "shuffled"][int(r.integers(0, 3))], cap1=float(r.choice([0, 5, 30])),
                cap2=float(r.choice([0, 5, 30])), bias1=kinds[int(r.integers(0, 4))], bias2=kinds[int(r.integers(0, 4))],
                nb=2 * int(r.integers(2, 33)), maxd=int(r.integers(40, 600)), bshd=bool(r.integers(0, 2)))
    dev, kw, where, p = problem(seed=seed, **case)
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p, num_splits=int(r.integers(0, 4)))
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode, deterministic=bool(r.integers(0, 2)))


def test_a_distillation_step():
    """The calls as a training step uses them: a capped teacher with slopes, a
    student with a learned table over packed documents; the loss weighs each
    query's divergence, and its gradient reaches the student's q, k and table,
    then the teacher's q and k."""
    dev, kw, where, p = problem(seed=20, B=2, H=4, HK1=2, HK2=4, NQ=300, NK=300, d1=128, d2=64, docs="packed",
                                cap1=30.0, bias1="slopes", bias2="one way")
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    weight = (where["doc_q"] >= 0).float()[:, None].expand(-1, 4, -1) / (where["doc_q"] >= 0).sum()
    loss = (weight * rows[0]).sum()
    want = ref.forward(p)
    w64 = f64(weight)
    assert abs(float(loss) - (w64 * want[0]).sum()) <= (w64 * want[3]).sum() + 1e-6 * float(loss)
    for mode in "12":
        m = skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2
        got = skl.streamkl_bwd_mod(p1, p2, *rows, weight.contiguous(), m, **where)
        g = ref.backward(p, *(f64(t) for t in rows), w64, mode)
        for a, b, e, what in zip(got, g[:3], g[3:], ("dq", "dk", "dtable")):
            if b is not None:
                within(a, b, e, what)
    # one update in place is seen by the next call through the same sides
    got = skl.streamkl_bwd_mod(p1, p2, *rows, weight.contiguous(), **where)
    dev["q2"].sub_(got[0])
    kw["2"]["table"].sub_(got[2])
    p["q2"], p["table2"] = f64(dev["q2"]), f64(kw["2"]["table"])
    check_forward(p1, p2, where, p)


@pytest.mark.parametrize("name", ["grouped table", "shuffled ids", "one row of shared heads", "table both ways", "padded heads",
                                  "prefix over many tiles"])
def test_debug_build_checks_pass_and_match(name):
    """The build whose kernels check their indexes: no check fails, same results."""
    import os
    path = os.path.join(os.path.dirname(skl.library_path), "libstreamkl_debug.so")
    if not os.path.exists(path):
        pytest.fail("libstreamkl_debug.so was not built")
    dev, kw, where, p = problem(seed=21, **CASES[name])
    p1, p2 = sides(dev, kw)

    def calls():
        rows = tuple(skl.streamkl_fwd_mod(p1, p2, **where, num_splits=2))
        out = rows
        for mode in (skl.STREAMKL_GRAD_P1, skl.STREAMKL_GRAD_P2):
            out = out + skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), mode, **where, deterministic=True)
        torch.cuda.synchronize()
        return out

    want = calls()
    saved = skl._lib, skl.library_path
    skl._lib, skl.library_path = None, path
    try:
        assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
        got = calls()
        assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    finally:
        skl._lib, skl.library_path = saved
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_at_once():
    """Host threads that launch the same kernels with lookup rows of different
    lengths, each on its own stream."""
    import threading
    work = []
    for seed, maxd in ((22, 20), (23, 900)):
        dev, kw, where, p = problem(seed=seed, NQ=260, NK=260, bias1="one way", bias2="one way", maxd=maxd)
        p1, p2 = sides(dev, kw)
        rows = skl.streamkl_fwd_mod(p1, p2, **where)
        want = [t.clone() for t in list(rows) + list(skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), **where,
                                                                          deterministic=True))]
        work.append((p1, p2, where, want))
    torch.cuda.synchronize()
    bad = []

    def go(p1, p2, where, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    rows = skl.streamkl_fwd_mod(p1, p2, **where)
                    got = list(rows) + list(skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), **where,
                                                                 deterministic=True))
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append("results differ")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=go, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad and skl.streamkl_get_device_status() == skl.STREAMKL_OK
