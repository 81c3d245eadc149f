"""The calls over modified scores at the ends of what they accept: scores far
below anything a softmax usually meets, masks written as large negative table
entries that are still finite numbers, tiny scales, large products."""

import math

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl
import mod_reference as ref
from test_mod_gpu import check_backward, check_forward, f64, problem, sides, within

pytestmark = pytest.mark.gpu


def definition(p, b, h, low):
    """kl, lse1, lse2 [NQ] of a head in 64 bits, no score taken for a mask, and their bounds.  Scores of the sides in
    `low` have exact products q.k: what they err by is at most four roundings (scale, its product, the bias, the sum)
    of their own size."""
    vis = ref.visible(p, b)
    out = []
    for t in "12":
        x, _, e = ref.score(p, t, b, h)
        e = np.where(vis, 4 * ref.F32 * np.abs(x) if t in low else e, 0.0)
        out.append((x, ref.lse(x, vis), e))
    (x1, l1, e1), (x2, l2, e2) = out
    a1, a2 = x1 - l1[:, None], x2 - l2[:, None]
    p1, p2 = np.where(vis, np.exp(a1), 0.0), np.where(vis, np.exp(a2), 0.0)
    r = np.where(vis, a1 - a2, 0.0)
    kl = (p1 * r).sum(1)
    n = np.minimum(vis.sum(1), 64) + 16
    # sums of n terms and their logarithms; dKL = sum p1 (r - KL) dS1 + sum (p2 - p1) dS2
    bk = (p1 * np.abs(r - kl[:, None]) * (e1.max(1) + e2.max(1) + n * ref.F32)[:, None]).sum(1) + 2 * e2.max(1)
    bk = bk + 2 * n * ref.F32 * (1 + (p1 * np.abs(r)).sum(1))
    return kl, l1, l2, bk, *(e.max(1) + n * ref.F32 + 4 * ref.F32 * np.abs(l) for l, e in ((l1, e1), (l2, e2)))


def check_low(rows, p, low):
    for h in range(p["q1"].shape[1]):
        want = definition(p, 0, h, low)
        for g, w, b, what in zip(rows, want[:3], want[3:], ("KL", "LSE1", "LSE2")):
            within(f64(g)[0, h], w, b, f"{what}, head {h}")


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("side", ["1", "2", "12"])
@pytest.mark.parametrize("bias", [None, "one way"])
def test_raw_scores_far_below_zero_are_no_mask(bias, side, splits):
    """scale q.k between -8.3e5 and -7.7e5 for every pair: rows with one key and with many.  q.k is exact (small whole
    numbers)."""
    dev, kw, where, p = problem(seed=40, NQ=200, NK=420, bias1=bias, bias2=bias, scale1=1e4 if "1" in side else None,
                                scale2=1e4 if "2" in side else None)
    g = torch.Generator().manual_seed(1)
    for t in side:
        dev["q" + t][:] = 1.0
        dev["k" + t][:] = -1.25
        dev["k" + t][..., 0] = torch.randint(-3, 3, dev["k" + t].shape[:3], generator=g).to(torch.bfloat16).cuda()
        p["q" + t], p["k" + t] = f64(dev["q" + t]), f64(dev["k" + t])
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where, num_splits=splits)
    check_low(rows, p, side)
    # the gradients: a row's LSE holds its scores to 2^-24 of 8e5, so P is known to 5 % only; here they are not lost
    dkl = torch.ones_like(rows[0])
    for m in (skl.STREAMKL_GRAD_P1, skl.STREAMKL_GRAD_P2):
        dq, dk, _ = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, m, **where)
        assert torch.isfinite(dq).all() and torch.isfinite(dk).all() and dk.any()


def test_one_key_far_below_zero():
    """A causal row with a single key has KL 0 and the key's score as LSE, however low."""
    dev, kw, where, p = problem(seed=41, NQ=1, NK=1, scale1=1e4)
    dev["q1"][:] = 1.0
    dev["k1"][:] = -1.25
    kl, l1, l2 = skl.streamkl_fwd_mod(*sides(dev, kw), **where)
    assert torch.all(kl.abs() < 1e-6) and torch.all((l1 + 8e5).abs() <= 4 * ref.F32 * 8e5) and torch.isfinite(l2).all()


def test_steep_slopes_are_no_mask():
    """Slopes that take a row's nearest key below -6.9e5 (ids keep the near ones away).  Slopes and products are small
    whole numbers, so the scores are exact."""
    dev, kw, where, p = problem(seed=42, NQ=300, NK=300, bias1="slopes", bias2="slopes", docs="packed", scale1=1.0, scale2=1.0)
    for t in "12":
        kw[t]["slopes"][:] = torch.tensor([8192.0, 4096.0], device="cuda")
        p["slopes" + t] = f64(kw[t]["slopes"])
        for x in "qk":
            dev[x + t].round_()
            p[x + t] = f64(dev[x + t])
    where["doc_q"].fill_(1)
    where["doc_k"][:] = (torch.arange(300, device="cuda") < 40).int()
    p["doc_q"], p["doc_k"] = where["doc_q"].cpu().numpy(), where["doc_k"].cpu().numpy()
    rows = skl.streamkl_fwd_mod(*sides(dev, kw), **where)
    assert rows[1].min() < -7e5 and torch.isfinite(rows[1]).all()
    check_low(rows, p, "12")


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("lowest", [-3.4028234663852886e38, -math.inf, -1e30, -1e9, -1e6])
def test_a_tables_mask_is_one_on_one_side_alone(lowest, splits):
    """The first rows see only keys which one side's table masks; beside raw scores of some -100 on the other side."""
    dev, kw, where, p = problem(seed=48, NQ=300, NK=300, H=2, bias1="one way", bias2="one way", scale2=20.0)
    kw["1"]["table"][1, :8] = lowest  # head 1 only
    rows = skl.streamkl_fwd_mod(*sides(dev, kw), **where, num_splits=splits)
    gone = torch.zeros(300, dtype=torch.bool, device="cuda")
    gone[:8] = True
    for t, w in zip(rows, (0.0, -math.inf, -math.inf)):
        assert torch.all(t[0, 1, gone] == w)
        assert torch.isfinite(t[0, 1, ~gone]).all() and torch.isfinite(t[0, 0]).all()


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("low", [-1e3, -1e4, -65504.0, -3e5])
@pytest.mark.parametrize("kind", ["far both ways", "near one way", "far both ways, capped", "near one way, ids"])
def test_finite_masks_cost_the_other_keys_nothing(kind, low, splits):
    """A row whose first keys in the kernel's order are masked by a large finite entry: the later keys' scores keep
    their own accuracy."""
    both = "both" in kind
    case = dict(NQ=500, NK=500, H=1, causal=not both, bias1="both ways" if both else "one way",
                bias2="both ways" if both else "one way")
    if "capped" in kind:
        case.update(cap1=30.0, cap2=50.0)
    if "ids" in kind:
        case.update(docs="packed")
    dev, kw, where, p = problem(seed=43, **case)
    for t in "12":
        tab = kw[t]["table"]
        if both:
            tab[:, 15] = tab[:, 31] = low
        else:
            tab[:, :8] = low
        p["table" + t] = f64(tab)
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p, num_splits=splits)
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode)


def test_steep_slopes_to_the_right():
    """The kernel's first keys are the farthest: 1500 positions x slope 60 below the nearest."""
    dev, kw, where, p = problem(seed=44, NQ=100, NK=1500, H=1, bias1="slopes", bias2="slopes", causal=False)
    for t in "12":
        kw[t]["slopes"][:] = 60.0
        p["slopes" + t] = f64(kw[t]["slopes"])
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode)


@pytest.mark.parametrize("side", ["1", "2"])
def test_finite_masks_on_one_side(side):
    """The other side's weight on the masked keys stays: its sum, of another reference, must not be taken for empty."""
    for low in (-2e3, -65504.0):
        dev, kw, where, p = problem(seed=49, NQ=500, NK=500, H=1, bias1="one way", bias2="one way")
        kw[side]["table"][:, :8] = low
        p["table" + side] = f64(kw[side]["table"])
        p1, p2 = sides(dev, kw)
        rows = check_forward(p1, p2, where, p)
        check_backward(p1, p2, where, p, rows, "2")


@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e-42, 1e-300])
def test_a_cap_far_above_tiny_scores(scale):
    """Capped scores that are all but zero: every visible key weighs the same."""
    dev, kw, where, p = problem(seed=45, NQ=150, NK=200, cap1=1e6, cap2=1e6, scale1=scale, scale2=scale)
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    check_backward(p1, p2, where, p, rows, "2")


@pytest.mark.parametrize("capped", ["1", "2"])
def test_large_products_beside_a_capped_side(capped):
    """q.k near 1e21 on the side without a cap, whose scale brings the scores back to a few units."""
    other = "2" if capped == "1" else "1"
    dev, kw, where, p = problem(seed=46, NQ=150, NK=200, **{"cap" + capped: 30.0, "scale" + other: 1e-21})
    for x in "qk":
        dev[x + other].mul_(2.0 ** 34)  # exact in bf16
        p[x + other] = f64(dev[x + other])
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode)


@pytest.mark.parametrize("d", range(16, 129, 16))
def test_the_scale_is_the_callers(d):
    """Rows that see one key each, whose products q.k are exact: LSE is scale q.k.  Beside the scale's own rounding
    (of scale log2 e to 32 bits, the same for all), what a row adds is the rounding of its score and of its LSE, evenly
    spread within 2^-24 each: over 1024 rows their mean is below 2^-24 / 16 (ten standard deviations)."""
    n, heads = 128, 8
    q = torch.ones(1, heads, n, d) * (1 + torch.arange(heads)[None, :, None, None] / 8)
    k = torch.ones(1, heads, n, d) * (64 + torch.arange(n)[None, None, :, None] / 2)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    q, k, scale = q.bfloat16().cuda(), k.bfloat16().cuda(), 1 / math.sqrt(d)
    side = skl.AttnSide(q, k, scale)
    kl, l1, l2 = skl.streamkl_fwd_mod(side, side, doc_q=ids, doc_k=ids)
    want = scale * (f64(q) * f64(k)).sum(3)
    rounded = float(np.float32(scale * math.log2(math.e))) / (scale * math.log2(math.e)) - 1
    for got in (l1, l2):
        assert abs((f64(got) / want - 1).mean() - rounded) < ref.F32 / 16 + 3e-9  # (ln 2 in 32 bits: 2.7e-9)
    assert torch.all(kl.abs() < 1e-6)
