"""The calls over modified scores at lengths of thousands of keys: far buckets
of the largest table, many key tiles in the fixed order of the deterministic
mode, single tokens of a long cache, offsets past 32 bits; and two host threads
that both have to finish."""

import threading

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl
import mod_reference as ref
from test_mod_gpu import check_backward, check_forward, f64, problem, sides, within

pytestmark = pytest.mark.gpu

CASES = {
    "largest table, far behind": dict(NQ=200, NK=4300, bias1="one way", bias2="one way", nb=64, maxd=4096, H=1),
    "largest table, both ways, far behind": dict(NQ=150, NK=4400, causal=False, bias2="both ways", nb=64, maxd=4096, cap1=30.0),
    "largest table, both ways, far ahead": dict(NQ=4400, NK=150, causal=False, bias1="both ways", bias2="slopes", nb=64,
                                                maxd=4096, H=1),
    "table in a long sequence": dict(NQ=2300, NK=2300, H=1, bias1="one way", bias2="one way", cap2=30.0),
    "packed, long": dict(NQ=2500, NK=2500, H=1, docs="packed", bias1="slopes", bias2="slopes", d1=128),
    "prefix, long": dict(NQ=500, NK=4100, H=2, prefix=[3900], cap1=30.0, cap2=30.0, d1=96, d2=96),
    "few rows, long": dict(NQ=5, NK=8100, H=8, HK1=2, HK2=2, cap1=30.0, bias2="slopes", d1=128, d2=128),
}


@pytest.mark.parametrize("name", list(CASES))
def test_long(name):
    dev, kw, where, p = problem(seed=60, **CASES[name])
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)
    if name.startswith("largest"):  # the last bucket of each direction in use is met
        r = np.arange(p["k1"].shape[2])[None] - np.arange(p["q1"].shape[2])[:, None] - (p["k1"].shape[2] - p["q1"].shape[2])
        met = set(np.unique(ref.bucket(r, 64, 4096, "both" in name)))
        assert (63 in met) or (31 in met and "behind" in name)
    for mode in "12":
        check_backward(p1, p2, where, p, rows, mode)


@pytest.mark.parametrize("mode", "12")
@pytest.mark.parametrize("case", [dict(NQ=300, NK=3300, H=4, HK1=1, HK2=1, cap1=30.0, cap2=30.0),
                                  dict(NQ=700, NK=2900, H=6, HK1=2, HK2=3, bias1="one way", bias2="one way", nb=64, maxd=2500),
                                  dict(NQ=1300, NK=1300, H=4, HK1=2, HK2=2, B=2, docs="packed", bias1="both ways",
                                       bias2="both ways", causal=False)])
def test_deterministic_over_many_tiles(case, mode):
    dev, kw, where, p = problem(seed=61, **case)
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    one, dkl = check_backward(p1, p2, where, p, rows, mode, deterministic=True)
    m = skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2
    for _ in range(6):
        two = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, m, **where, deterministic=True)
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("kw", [dict(cap1=50.0, cap2=50.0), dict(bias1="one way", bias2="slopes", nb=64, maxd=4000),
                                dict(docs="shuffled", causal=False)])
@pytest.mark.parametrize("nq", [1, 3])
def test_last_tokens_of_a_long_cache(nq, kw):
    """The library's own splits over 30011 keys."""
    dev, kws, where, p = problem(seed=62, H=8, HK1=2, HK2=2, NQ=nq, NK=30011, d1=128, d2=64, **kw)
    check_forward(*sides(dev, kws), where, p)


def test_offsets_past_32_bits():
    """K and dk inside caches whose second batch begins 2^31 elements in, and whose heads lie 2^30 apart."""
    dev, kw, where, p = problem(seed=63, B=2, H=2, NQ=140, NK=300, bias2="one way", d2=64)
    p1, p2 = sides(dev, kw)
    rows = check_forward(p1, p2, where, p)

    def cache(t):
        big = torch.empty(2 ** 31 + 2 ** 30 + 300 * 64, dtype=torch.bfloat16, device="cuda")
        v = big.as_strided(t.shape, (2 ** 31, 2 ** 30, 64, 1))
        v.copy_(t)
        return v

    far = dict(dev, k2=cache(dev["k2"]))
    q1, q2 = sides(far, kw)
    got = skl.streamkl_fwd_mod(q1, q2, **where)
    assert all(torch.equal(a, b) for a, b in zip(got, rows))
    dk = cache(torch.full_like(dev["k2"], 7.0))
    dkl = torch.ones_like(rows[0])
    want = skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True)
    out = skl.streamkl_bwd_mod(q1, q2, *rows, dkl, **where, deterministic=True, dk=dk)
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and out[1] is dk


def test_both_threads_finish():
    """Two host threads at once, on a stream each, through the same kernels; each says that it is done."""
    work = []
    for seed, case in ((64, dict(NQ=260, NK=260, bias1="one way", bias2="one way", maxd=20)),
                       (65, dict(NQ=200, NK=400, bias1="one way", bias2="one way", maxd=900, H=4, HK1=2, HK2=2))):
        dev, kw, where, p = problem(seed=seed, **case)
        p1, p2 = sides(dev, kw)
        rows = skl.streamkl_fwd_mod(p1, p2, **where)
        one = torch.ones_like(rows[0])
        want = [t.clone() for t in list(rows) + list(skl.streamkl_bwd_mod(p1, p2, *rows, one, **where, deterministic=True))]
        work.append((p1, p2, where, one, want))
    torch.cuda.synchronize()
    said = [None, None]

    def go(n, p1, p2, where, one, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                same = True
                for _ in range(20):
                    rows = skl.streamkl_fwd_mod(p1, p2, **where)
                    got = list(rows) + list(skl.streamkl_bwd_mod(p1, p2, *rows, one, **where, deterministic=True))
                    same = same and all(torch.equal(a, b) for a, b in zip(got, want))
                torch.cuda.current_stream().synchronize()
            said[n] = "same" if same else "results differ"
        except Exception as e:  # noqa: BLE001
            said[n] = repr(e)

    threads = [threading.Thread(target=go, args=(n, *w)) for n, w in enumerate(work)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and said == ["same", "same"]
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
