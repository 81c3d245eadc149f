"""The attention KL over selected blocks on the GPU against the float64
definitions, element by element within the bounds of mod_reference.py: head
layouts, lengths from one token on, lists with empty, repeated and foreign
entries, masks that leave rows empty, strides, streams, graphs."""

import math

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl
import mod_reference as dense
import sel_reference as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def problem(seed=0, B=1, H=2, HK1=None, HK2=None, HS=1, NQ=150, NK=150, d1=64, d2=64, bs=32, T=3, sd=1.5, causal=True,
            prefix=None, docs=None, bshd=False, lists="mixed"):
    """(sides' tensors, blocks, where, float64 problem).  lists: "mixed" (random
    blocks, some empty, repeated, unseen or not there), "all" (every block),
    "none"."""
    g = torch.Generator().manual_seed(seed)
    HK1, HK2 = HK1 or H, HK2 or H

    def x(h, n, d):
        t = (sd * torch.randn((B, h, n, d), generator=g)).to(torch.bfloat16)
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if bshd else t.cuda()

    dev = dict(q1=x(H, NQ, d1), k1=x(HK1, NK, d1), q2=x(H, NQ, d2), k2=x(HK2, NK, d2))
    nb = -(-NK // bs)
    if lists == "all":
        idx = torch.arange(nb, dtype=torch.int32).expand(B, HS, NQ, nb).contiguous()
    elif lists == "none":
        idx = torch.full((B, HS, NQ, T), -1, dtype=torch.int32)
    else:
        idx = torch.randint(-1, nb + 1, (B, HS, NQ, T), generator=g, dtype=torch.int32)
        if T > 1:
            idx[..., 1] = torch.where(torch.rand(idx[..., 1].shape, generator=g) < 0.2, idx[..., 0], idx[..., 1])
        idx[:, :, ::17] = -1
        idx[:, :, 5::23, -1] = 2 ** 31 - 1
        idx[:, :, 6::23, 0] = -2 ** 31
    ids = None
    if docs is not None:
        if docs == "packed":
            q = torch.sort(torch.randint(0, 4, (B, NQ), generator=g), dim=1)[0]
            k = q if NQ == NK else torch.sort(torch.randint(0, 4, (B, NK), generator=g), dim=1)[0]
            q, k = q.clone(), k.clone()
            q[:, NQ - NQ // 9:] = -1
            k[:, NK - NK // 9:] = -1
        else:
            q = torch.randint(-2, 6, (B, NQ), generator=g)
            k = torch.randint(-2, 6, (B, NK), generator=g)
        ids = q.int(), k.int()
    p = {k: f64(v) for k, v in dev.items()}
    for t, d in (("1", d1), ("2", d2)):
        p.update({"scale" + t: 1 / math.sqrt(d), "cap" + t: 0.0, "slopes" + t: None, "table" + t: None})
    p.update(blocks=idx.numpy(), bs=bs, causal=causal, prefix=None if prefix is None else np.array(prefix),
             doc_q=None if ids is None else ids[0].numpy(), doc_k=None if ids is None else ids[1].numpy())
    where = dict(causal=causal, prefix=None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
                 doc_q=None if ids is None else ids[0].cuda(), doc_k=None if ids is None else ids[1].cuda())
    return dev, idx.cuda(), where, p


def sides(dev):
    return tuple(skl.AttnSide(dev["q" + t], dev["k" + t], 1 / math.sqrt(dev["q" + t].shape[3])) for t in "12")


def within(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    same = np.isinf(want) & (got == want)
    err = np.abs(np.where(same, 0.0, got) - np.where(same, 0.0, want))
    assert np.all(np.isfinite(err)), f"{what}: not finite where the definition is"
    over = err - bound - 1e-30
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what} at {at}: {got[at]} for {want[at]}, error {err[at]:.3g}, bound {bound[at]:.3g}"


def check_forward(dev, idx, where, p, **kw):
    got = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where, **kw)
    torch.cuda.synchronize()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    want = ref.forward(p)
    for g, w, b, what in zip(got, want[:3], want[3:], ("KL", "LSE1", "LSE2")):
        within(g, w, b, what)
    return got


def check_backward(dev, idx, where, p, rows, mode, seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    dkl = (torch.rand(rows[0].shape, generator=g) * 2 - 0.5).cuda()
    got = skl.streamkl_bwd_sel(*sides(dev), idx, p["bs"], *rows, dkl,
                               skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2, **where, **kw)
    torch.cuda.synchronize()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    want = list(ref.backward(p, *(f64(t) for t in rows), f64(dkl), mode))
    # every block's contribution to dq is rounded to the row's grid: as grid_error for tiles of 128, with a slot each
    slots = p["blocks"].shape[3]
    tiles = -(-p["k1"].shape[2] // 128)
    want[2] = want[2] + (1 + dense.BF16) * dense.grid_error(p, f64(rows[0]), f64(dkl), mode) * slots / tiles
    for g_, w, b, what in zip(got, want[:2], want[2:], ("dq", "dk")):
        within(g_, w, b, f"mode P{mode} {what}")
    return got, dkl


CASES = {
    "one token": dict(H=1, NQ=1, NK=1, T=1),
    "one row": dict(H=4, HK1=1, HK2=1, NQ=1, NK=300, T=4),
    "heads apart": dict(B=2, H=3, HS=3, NQ=200, NK=200),
    "one list for all heads": dict(B=2, H=6, HK1=2, HK2=3, HS=1, NQ=100, NK=140, T=5),
    "groups of three": dict(H=6, HK1=2, HK2=2, HS=2, NQ=130, NK=333, T=6, bs=64),
    "grouped": dict(H=8, HK1=2, HK2=2, HS=2, NQ=300, NK=300, T=4, bs=64, d1=128, d2=128),
    "student with its own heads": dict(H=8, HK1=2, HK2=8, HS=2, NQ=260, NK=260, T=2, bs=128, d1=128, d2=64),
    "lists finer than keys": dict(H=8, HK1=1, HK2=2, HS=8, NQ=90, NK=257, T=4, d1=64, d2=128),
    "more heads than a tile": dict(H=192, HK1=1, HK2=1, HS=1, NQ=9, NK=70, T=3, d1=16, d2=32),
    "odd head dims": dict(H=2, NQ=77, NK=190, d1=80, d2=112, bs=128, T=2),
    "narrow": dict(H=2, NQ=77, NK=190, d1=16, d2=48, T=7),
    "last block short": dict(H=2, NQ=64, NK=129, bs=128, T=2),
    "not causal": dict(H=4, HK1=2, HK2=2, NQ=190, NK=500, causal=False, bs=64, T=5, bshd=True),
    "more queries than keys": dict(H=2, NQ=300, NK=100, T=3),
    "prefix": dict(B=3, H=2, NQ=150, NK=260, prefix=[0, 77, 260], T=5),
    "packed": dict(B=2, H=4, HK1=2, HK2=2, HS=2, NQ=300, NK=300, docs="packed", T=6, bshd=True),
    "shuffled ids": dict(B=2, H=2, NQ=200, NK=170, docs="shuffled", T=4, bs=64),
    "ids and prefix": dict(B=2, H=2, NQ=200, NK=200, docs="packed", prefix=[60, 130], T=4),
    "33 slots": dict(H=2, NQ=70, NK=900, T=33),
    "128 slots": dict(H=2, HS=2, NQ=40, NK=700, T=128, causal=False),
    "every block": dict(H=2, NQ=300, NK=300, lists="all"),
    "no block": dict(H=2, NQ=100, NK=100, lists="none"),
    "many blocks": dict(H=1, NQ=200, NK=20000, T=9, d1=64, d2=64),
    "many rows": dict(H=16, HK1=2, HK2=2, HS=2, NQ=1500, NK=1500, T=5, bs=64, d1=128, d2=128, bshd=True),
    "peaked": dict(H=2, NQ=200, NK=400, T=6, sd=6.0),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    check_forward(*problem(**CASES[name]))


@pytest.mark.parametrize("mode", ["1", "2"])
@pytest.mark.parametrize("name", CASES)
def test_backward(name, mode):
    dev, idx, where, p = problem(**CASES[name])
    rows = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    got, dkl = check_backward(dev, idx, where, p, rows, mode)
    again, _ = check_backward(dev, idx, where, p, rows, mode)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_every_block_is_the_dense_forward():
    dev, idx, where, p = problem(H=4, HK1=2, HK2=2, NQ=333, NK=333, bs=64, lists="all", d1=128, d2=128)
    got = check_forward(dev, idx, where, p)
    dense = skl.streamkl_fwd_mod(*sides(dev), **where)
    for g, d in zip(got, dense):
        assert (g - d).abs().max() <= 1e-4


def test_hidden_keys_hold_anything():
    dev, idx, where, p = problem(B=1, H=2, NQ=200, NK=200, docs="packed", T=2, lists="mixed")
    want = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    idx[idx == 3] = -1
    p["blocks"] = idx.cpu().numpy()
    want = check_forward(dev, idx, where, p)
    pad = where["doc_k"][0] < 0
    for t in "12":
        dev["k" + t][:, :, pad] = float("nan")
        dev["k" + t][:, :, 96:128] = float("inf")     # block 3, which nobody selects
    got = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    # keys after a causal query
    dev, idx, where, p = problem(H=1, NQ=64, NK=64, T=1, lists="all")
    want = skl.streamkl_fwd_sel(*sides(dev), idx, 32, **where)
    dev["k1"][:, :, 40:] = float("nan")
    got = skl.streamkl_fwd_sel(*sides(dev), idx, 32, **where)
    for g, w in zip(got, want):
        assert torch.equal(g[..., :40], w[..., :40])


def test_nan_queries_stay_with_their_rows():
    dev, idx, where, p = problem(H=4, HK1=2, HK2=2, NQ=100, NK=100)
    want = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    dev["q1"][0, 1, 50] = float("nan")
    got = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    for g, w in zip(got, want):
        same = g == w
        same[0, 1, 50] = True
        assert same.all()
    assert torch.isnan(got[0][0, 1, 50])


def test_strides():
    """Heads and tokens inside larger tensors, and strides whose common divisor is below the head dim."""
    dev, idx, where, p = problem(B=2, H=4, HK1=2, HK2=2, NQ=70, NK=90, d1=64, d2=80)
    want = skl.streamkl_fwd_sel(*sides(dev), idx, p["bs"], **where)
    for pad_n, pad_h, pad_b in ((0, 0, 0), (8, 0, 0), (0, 40, 0), (16, 8, 24)):
        other = {}
        for name, t in dev.items():
            B, H, N, d = t.shape
            sn = d + pad_n
            sh, sb = N * sn + pad_h, 0
            sb = H * sh + pad_b
            buf = torch.full((B * sb,), float("nan"), dtype=torch.bfloat16, device="cuda")
            v = buf.as_strided((B, H, N, d), (sb, sh, sn, 1))
            v.copy_(t)
            other[name] = v
        got = skl.streamkl_fwd_sel(*sides(other), idx, p["bs"], **where)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_repeatable_and_order_free():
    dev, idx, where, p = problem(H=8, HK1=2, HK2=2, HS=2, NQ=700, NK=700, T=6, bs=32)
    want = skl.streamkl_fwd_sel(*sides(dev), idx, 32, **where)
    for _ in range(3):
        for g, w in zip(skl.streamkl_fwd_sel(*sides(dev), idx, 32, **where), want):
            assert torch.equal(g, w)
    turned = idx.flip(3).contiguous()
    p["blocks"] = turned.cpu().numpy()
    check_forward(dev, turned, where, p)


def test_outputs_workspace_streams_and_graphs():
    dev, idx, where, p = problem(H=4, HK1=2, HK2=2, NQ=200, NK=200, T=4)
    p1, p2 = sides(dev)
    want = skl.streamkl_fwd_sel(p1, p2, idx, 32, **where)
    need = skl.streamkl_fwd_sel_workspace_bytes(p1, p2, idx, 32, **where)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(w, float("nan")) for w in want]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = skl.streamkl_fwd_sel(p1, p2, idx, 32, **where, workspace=ws, kl=out[0], lse1=out[1], lse2=out[2], stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(g is o for g, o in zip(got, out))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    with pytest.raises(skl.StreamKLError):
        skl.streamkl_fwd_sel(p1, p2, idx, 32, **where, workspace=ws[: need - 16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = skl.streamkl_fwd_sel(p1, p2, idx, 32, **where)
    dev["q2"].copy_(torch.randn_like(dev["q2"], dtype=torch.float32))
    idx.copy_(idx.roll(1, 2))
    graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(again, skl.streamkl_fwd_sel(p1, p2, idx, 32, **where)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("bs", [32, 64, 128])
@pytest.mark.parametrize("d1,d2", [(96, 128), (128, 96), (48, 128), (128, 48), (80, 112)])
def test_nan_queries_stay_with_their_rows_beside_a_narrower_side(d1, d2, bs):
    """The sides' tiles take turns in the same memory, where the narrower one leaves columns of the other: many tiles a
    CTA, so that each place is used by both."""
    dev, idx, where, p = problem(H=16, HK1=2, HK2=2, HS=2, NQ=2000, NK=2000, T=6, bs=bs, d1=d1, d2=d2)
    bad = torch.arange(11, 2000, 97, device="cuda")
    idx[:, :, bad] = -1
    idx[:, :, bad, 0] = 0  # what these rows reach: block 0
    want = skl.streamkl_fwd_sel(*sides(dev), idx, bs, **where)
    dkl = torch.ones_like(want[0])
    grads = {m: skl.streamkl_bwd_sel(*sides(dev), idx, bs, *want, dkl, m, **where)
             for m in (skl.STREAMKL_GRAD_P1, skl.STREAMKL_GRAD_P2)}
    others = torch.ones(2000, dtype=torch.bool, device="cuda")
    others[bad] = False
    for side in "12":
        q = dev["q" + side].clone()
        dev["q" + side][:, :, bad] = float("nan")
        got = skl.streamkl_fwd_sel(*sides(dev), idx, bs, **where)
        for g, w in zip(got, want):
            assert torch.equal(g[:, :, others], w[:, :, others])
        assert torch.isnan(got[0][:, :, bad]).all()
        for m, (dq, dk) in grads.items():
            a, b = skl.streamkl_bwd_sel(*sides(dev), idx, bs, *got, dkl, m, **where)
            assert torch.equal(a[:, :, others], dq[:, :, others])
            assert torch.equal(b[:, :, bs:], dk[:, :, bs:])
        dev["q" + side].copy_(q)
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK


ANYTHING = {
    "packed": dict(B=2, H=4, HK1=2, HK2=2, HS=2, NQ=300, NK=300, docs="packed", T=5),
    "shuffled ids, large blocks": dict(B=2, H=4, HK1=1, HK2=4, HS=1, NQ=200, NK=333, docs="shuffled", T=2, bs=128, d1=128, d2=96),
    "shuffled ids, blocks of 64": dict(B=2, H=6, HK1=2, HK2=3, HS=2, NQ=260, NK=400, docs="shuffled", T=3, bs=64, d1=48, d2=64),
    "more queries than keys": dict(H=2, NQ=300, NK=100, T=3),
    "few lists": dict(H=4, HK1=2, HK2=2, NQ=400, NK=400, T=2, d1=80, d2=128),
}


@pytest.mark.parametrize("mode", ["1", "2"])
@pytest.mark.parametrize("name", ANYTHING)
def test_what_nobody_sees_may_hold_anything(name, mode):
    """Rows that see nothing (padded, before the first key, without a list, or whose blocks hold no key of theirs): q and
    dkl; keys with a negative id: k.  The results are those of zeros there, and theirs are zeros."""
    dev, idx, where, p = problem(**ANYTHING[name])
    bs, flag = p["bs"], skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2
    rows = skl.streamkl_fwd_sel(*sides(dev), idx, bs, **where)
    blind = torch.isinf(rows[1])  # [B, H, NQ]
    assert blind.any() and torch.equal(blind, torch.isinf(rows[2])) and not blind.all()
    hidden = where["doc_k"] < 0 if where["doc_k"] is not None else torch.zeros_like(dev["k1"][:, 0, :, 0], dtype=torch.bool)
    dkl = torch.rand(rows[0].shape, generator=torch.Generator().manual_seed(2)).cuda() + 0.5
    results = []
    for junk in (0.0, float("nan"), float("inf"), -3.0e38):
        x = {n: t.clone() for n, t in dev.items()}
        w = dkl.clone()
        for t in "12":
            x["q" + t][blind] = junk
            k = x["k" + t]
            k[hidden[:, None].expand(k.shape[:3])] = junk
        w[blind] = junk
        got = skl.streamkl_fwd_sel(*sides(x), idx, bs, **where)
        for g, v in zip(got, rows):
            assert torch.equal(g, v)
        results.append(skl.streamkl_bwd_sel(*sides(x), idx, bs, *got, w, flag, **where))
    for dq, dk in results:
        assert torch.equal(dq, results[0][0]) and torch.equal(dk, results[0][1])
        assert not dq[blind].any() and not dk[hidden[:, None].expand(dk.shape[:3])].any()
        assert dq.isfinite().all() and dk.isfinite().all() and dq.any() and dk.any()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK


@pytest.mark.parametrize("mode", ["1", "2"])
def test_backward_workspace_streams_and_graphs(mode):
    dev, idx, where, p = problem(H=4, HK1=2, HK2=2, NQ=200, NK=200, T=4)
    p1, p2 = sides(dev)
    flag = skl.STREAMKL_GRAD_P1 if mode == "1" else skl.STREAMKL_GRAD_P2
    rows = skl.streamkl_fwd_sel(p1, p2, idx, 32, **where)
    dkl = torch.ones_like(rows[0])
    want = skl.streamkl_bwd_sel(p1, p2, idx, 32, *rows, dkl, flag, **where)
    need = skl.streamkl_bwd_sel_workspace_bytes(p1, p2, idx, 32, flag, **where)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(w, float("nan")) for w in want]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = skl.streamkl_bwd_sel(p1, p2, idx, 32, *rows, dkl, flag, **where, dq=out[0], dk=out[1], workspace=ws[:need], stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(g is o for g, o in zip(got, out)) and (ws[need:] == 255).all()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    for less in (need - 1, need - 16, 16):
        with pytest.raises(skl.StreamKLError):
            skl.streamkl_bwd_sel(p1, p2, idx, 32, *rows, dkl, flag, **where, workspace=ws[:less])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = skl.streamkl_bwd_sel(p1, p2, idx, 32, *rows, dkl, flag, **where)
    idx.copy_(idx.roll(1, 2))
    dkl.copy_(torch.rand_like(dkl))
    graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(again, skl.streamkl_bwd_sel(p1, p2, idx, 32, *rows, dkl, flag, **where)):
        assert torch.equal(g, w)
