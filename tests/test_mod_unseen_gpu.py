"""Query rows that see no key (LSE -inf) in the backward over modified scores:
whatever their q and dkl hold, they get zeros and no other gradient changes."""

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl
import mod_reference as ref
from test_mod_gpu import f64, problem, sides, within

pytestmark = pytest.mark.gpu


def ids_nobody_has(dev, kw, where, p):
    """Every third query carries an id that no key has."""
    q = where["doc_q"]
    q[:, ::3] = 77
    p["doc_q"] = q.cpu().numpy()


def keys_all_later(dev, kw, where, p):
    """Rows 40 to 59 share an id only with keys that lie behind them in time."""
    where["doc_q"][:, 40:60] = 5
    where["doc_k"].clamp_(max=4)
    where["doc_k"][:, 150:] = 5
    p["doc_q"], p["doc_k"] = where["doc_q"].cpu().numpy(), where["doc_k"].cpu().numpy()


def nearest_masked(dev, kw, where, p):
    """The first rows see near keys only, which the table masks."""
    for t in "12":
        kw[t]["table"][:, :8] = -3.4028234663852886e38
        p["table" + t][:, :8] = np.float64(np.float32(-3.4028234663852886e38))


CASES = {
    "more rows than keys": (dict(NQ=300, NK=170), None),
    "more rows than keys, capped": (dict(NQ=300, NK=170, cap1=30.0, cap2=20.0, H=4, HK2=2), None),
    "more rows than keys, table": (dict(NQ=300, NK=170, bias1="slopes", bias2="one way", d1=128, d2=128), None),
    "more rows than keys, tables": (dict(NQ=260, NK=131, bias1="one way", bias2="one way", cap1=30.0), None),
    "an id no key has": (dict(docs="packed", NQ=200, NK=260, causal=False, B=2, bias2="both ways", bias1="slopes"), ids_nobody_has),
    "an id no key has, capped": (dict(docs="shuffled", NQ=200, NK=200, causal=False, cap2=30.0), ids_nobody_has),
    "ids of later keys": (dict(docs="packed", NQ=200, NK=200, bias2="one way", H=4, HK1=2, HK2=2), ids_nobody_has),
    "keys all later": (dict(docs="packed", NQ=200, NK=200, bias1="one way", bias2="slopes"), keys_all_later),
    "masked by the table": (dict(NQ=200, NK=200, bias1="one way", bias2="one way"), nearest_masked),
    "masked by the table, capped": (dict(NQ=400, NK=400, bias1="one way", bias2="one way", cap1=30.0, cap2=30.0),
                                    nearest_masked),
}


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("name", list(CASES))
def test_unseen_rows_may_hold_anything(name, junk):
    case, change = CASES[name]
    dev, kw, where, p = problem(seed=30, **case)
    if change is not None:
        change(dev, kw, where, p)
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    empty = torch.isinf(rows[1])
    assert empty.any() and not empty.all() and torch.equal(empty, torch.isinf(rows[2]))
    assert np.array_equal(empty.cpu().numpy(), np.isinf(ref.forward(p)[1]))
    g = torch.Generator().manual_seed(31)
    dkl = (torch.rand(rows[0].shape, generator=g) * 2 - 0.5).cuda()
    clean = f64(dkl)
    dev["q1"][empty] = junk
    dev["q2"][empty] = junk
    dkl[empty] = junk
    for mode, det in (("1", False), ("2", False), ("1", True), ("2", True)):
        got = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2,
                                   **where, deterministic=det)
        want = list(ref.backward(p, *(f64(t) for t in rows), clean, mode))
        if det:
            want[3] = want[3] + (1 + ref.BF16) * ref.grid_error(p, f64(rows[0]), clean, mode)
        for x, w, b, what in zip(got, want[:3], want[3:], ("dq", "dk", "dtable")):
            if w is not None:
                within(x, w, b, f"mode P{mode} {what}")
        assert not got[0][empty].any()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
