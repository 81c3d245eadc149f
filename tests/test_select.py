"""Selected blocks against float64 scores: the same lists, ties to the lowest
block, forced and masked ones, and the refusals, without a GPU."""

import os

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl

A = 4096
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(skl.library_path):
        import __graft_entry__
        __graft_entry__.build()
    return skl.lib()


def seen(causal=0, prefix=None, doc_q=None, doc_k=None):
    return skl._Visible(causal, prefix, doc_q, doc_k)


def call(L, q=None, kb=None, vis=None, B=1, H=4, heads=2, NQ=100, NK=300, d=64, block=32, count=4, sink=1, local=1, out=A,
         ws=A, ws_bytes=1 << 40):
    v = skl._View(A, 1 << 20, 1 << 16, d)
    return L.streamkl_select_blocks(q or v, kb or v, vis or seen(), B, H, heads, NQ, NK, d, block, count, sink, local, out,
                                    ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(vis=seen(2)), 1), (dict(vis=seen(0, A)), 1), (dict(vis=seen(0, None, A)), 1), (dict(vis=seen(1, A + 1)), 1),
    (dict(block=48), 1), (dict(block=0), 1), (dict(count=0), 1), (dict(count=129), 1), (dict(sink=-1), 1),
    (dict(local=-1), 1), (dict(sink=3, local=2), 1), (dict(sink=5, local=0), 1), (dict(heads=3), 1), (dict(heads=0), 1),
    (dict(heads=8), 1), (dict(d=8), 2), (dict(d=72), 2), (dict(d=144), 2), (dict(NK=32 * 4096 + 1), 2), (dict(NK=0), 1),
    (dict(NQ=-1), 1), (dict(out=0), 1), (dict(out=A + 2), 1), (dict(ws=0), 1), (dict(ws=A + 8), 1), (dict(ws_bytes=64), 1),
    (dict(q=skl._View(0, 64, 64, 64)), 1), (dict(kb=skl._View(A, 64, 64, 4)), 1), (dict(B=20000), 1),
    (dict(NK=2 ** 31 - 1, H=1, heads=1), 2),
])
def test_refusals(L, kw, status):
    assert call(L, **kw) == status


def test_empty_and_workspace(L):
    assert call(L, NQ=0, out=0, ws=0) == 0 and call(L, B=0, out=0, ws=0) == 0
    f = skl.streamkl_select_blocks_workspace_bytes
    assert f(1, 4, 2, 100, 300, 64, 32, 4) >= 2 * 128 * 16 * 4
    assert f(1, 4, 2, 100, 300, 64, 32, 0) == 0
    assert f(1, 4, 2, 100, 300, 64, 32, 4, ids=True) > f(1, 4, 2, 100, 300, 64, 32, 4)
    assert f(1, 32, 8, 1 << 17, 1 << 17, 128, 32, 16) < 160 << 20  # strips


def expected(q, kb, T, bs, NK, causal, prefix, ids, sink, local):
    q, kb = q.double().cpu().numpy(), kb.double().cpu().numpy()
    B, H, NQ, _ = q.shape
    hs, nb = kb.shape[1], kb.shape[2]
    out = np.full((B, hs, NQ, T), -1, np.int32)
    for b in range(B):
        for h in range(hs):
            g = H // hs
            score = q[b, h * g:(h + 1) * g].sum(0) @ kb[b, h].T
            for i in range(NQ):
                first = np.arange(nb) * bs
                can = np.ones(nb, bool)
                if causal:
                    can = first <= i + NK - NQ
                    if prefix is not None:
                        can |= first < prefix[b]
                if ids is not None:
                    x = ids[0][b, i]
                    k = np.concatenate([ids[1][b], np.full(nb * bs - NK, -1)]).reshape(nb, bs)
                    lo = np.where(k >= 0, k, 2 ** 31 - 1).min(1)
                    can &= (x >= 0) & (lo <= x) & (x <= k.max(1))
                c = np.nonzero(can)[0]
                forced = set(c[:sink]) | set(c[len(c) - local:] if local else [])
                rest = sorted((j for j in c if j not in forced), key=lambda j: (-score[i, j], j))
                take = sorted(list(forced) + rest[:max(0, T - len(forced))])
                out[b, h, i, :len(take)] = take
    return out


def run(B=1, H=4, HS=2, NQ=100, NK=300, d=64, bs=32, T=4, causal=True, prefix=None, docs=None, sink=1, local=1, bshd=False,
        seed=0, make=None):
    g = torch.Generator().manual_seed(seed)
    nb = -(-NK // bs)
    q = torch.randn((B, H, NQ, d), generator=g)
    kb = torch.randn((B, HS, nb, d), generator=g)
    if make:
        q, kb = make(q, kb)
    q, kb = q.to(torch.bfloat16), kb.to(torch.bfloat16)
    ids = None
    if docs == "packed":
        k = torch.sort(torch.randint(0, 4, (B, NK), generator=g), dim=1)[0]
        k[:, NK - NK // 9:] = -1
        ids = k[:, NK - NQ:].int().contiguous(), k.int()
    elif docs == "shuffled":
        ids = torch.randint(-2, 9, (B, NQ), generator=g).int(), torch.randint(-5, 9, (B, NK), generator=g).int()
    lay = (lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if bshd else (lambda t: t.cuda())
    kw = dict(causal=causal, prefix=None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
              doc_q=None if ids is None else ids[0].cuda(), doc_k=None if ids is None else ids[1].cuda(), sink=sink,
              local=local)
    got = skl.streamkl_select_blocks(lay(q), lay(kb), T, bs, NK, **kw)
    torch.cuda.synchronize()
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK
    want = expected(q, kb, T, bs, NK, causal, prefix, None if ids is None else [x.numpy() for x in ids], sink, local)
    assert np.array_equal(got.cpu().numpy(), want)
    return lay(q), lay(kb), kw, got


CASES = {
    "one token": dict(H=1, HS=1, NQ=1, NK=1, T=1, sink=0),
    "one query": dict(H=8, HS=2, NQ=1, NK=1000, T=8),
    "grouped": dict(H=8, HS=2, NQ=300, NK=1500, T=6, d=128),
    "heads apart": dict(B=2, H=3, HS=3, NQ=130, NK=600, T=5, bshd=True),
    "one list for all": dict(H=6, HS=1, NQ=129, NK=900, T=7, d=80, bs=64),
    "not causal": dict(H=4, HS=4, NQ=70, NK=2000, T=12, causal=False, bs=64, sink=0, local=0),
    "no forced": dict(NQ=300, NK=300, T=3, sink=0, local=0),
    "all forced": dict(NQ=300, NK=300, T=4, sink=2, local=2),
    "fewer candidates than places": dict(NQ=200, NK=200, T=16),
    "more queries than keys": dict(NQ=300, NK=100, T=3),
    "prefix": dict(B=3, NQ=150, NK=400, prefix=[0, 177, 400], T=5),
    "packed": dict(B=2, NQ=400, NK=400, docs="packed", T=4),
    "packed, few queries": dict(B=2, NQ=40, NK=700, docs="packed", T=4, sink=2),
    "shuffled ids": dict(B=2, NQ=100, NK=500, docs="shuffled", T=4, causal=False),
    "300 blocks": dict(H=2, HS=1, NQ=40, NK=300 * 32, T=32),
    "600 blocks": dict(H=2, HS=1, NQ=40, NK=600 * 32 - 5, T=16, causal=False),
    "1500 blocks": dict(H=2, HS=2, NQ=20, NK=1500 * 32, T=24, docs="packed"),
    "4096 blocks": dict(H=1, HS=1, NQ=5, NK=4096 * 32, T=128, causal=False, d=16),
    "128 places": dict(H=1, HS=1, NQ=50, NK=200 * 32, T=128, d=32),
    "large blocks": dict(NQ=500, NK=5000, bs=128, T=9, d=112),
}


@gpu
@pytest.mark.parametrize("name", CASES)
def test_lists(name):
    run(**CASES[name])


def whole_numbers(q, kb):
    """Small whole numbers: many exact ties."""
    return q.round().clamp(-1, 1), kb.round().clamp(-1, 1)


def equal_keys(q, kb):
    kb[:, :, 3:] = kb[:, :, 3:4]
    return q, kb


def zeros(q, kb):
    q[:, :, ::2] = 0
    kb[:, :, 5::3] = 0
    return q, kb


def near(q, kb):
    """Keys one rounding apart: sums of fp32 do not tell all of them apart."""
    kb[:] = kb[:, :, :1]
    bump = torch.zeros_like(kb)
    at = torch.arange(kb.shape[2]) % kb.shape[3]
    bump[:, :, torch.arange(kb.shape[2]), at] = 2.0 ** -7
    return q, kb * (1 + bump)


def cancelling(q, kb):
    """Large products that cancel, and what is left decides."""
    q[..., 1::2] = -q[..., ::2]
    kb[..., ::2] = 64.0
    kb[..., 1::2] = 64.0
    kb[..., 0] += torch.randn(kb.shape[:3], generator=torch.Generator().manual_seed(1))
    return q, kb


@gpu
@pytest.mark.parametrize("make", [whole_numbers, equal_keys, zeros, near, cancelling])
@pytest.mark.parametrize("shape", [dict(NQ=200, NK=2000, T=6), dict(NQ=60, NK=40000, T=16, causal=False, H=2, HS=1)])
def test_ties_and_close_scores(make, shape):
    run(make=make, **shape)


@gpu
def test_sizes_of_scores():
    run(make=lambda q, kb: (q * 1e10, kb * 1e10))
    run(make=lambda q, kb: (q * 1e-12, kb * 1e-8))


@gpu
def test_not_finite_queries_stay_in_bounds():
    q, kb, kw, want = run(NQ=64, NK=2000, T=6, causal=False)
    q[0, 0, 5] = float("nan")
    q[0, 2, 7, 3] = float("inf")
    kw["causal"] = False
    got = skl.streamkl_select_blocks(q, kb, 6, 32, 2000, **kw)
    assert got.min() >= -1 and got.max() < 63
    same = torch.ones(64, dtype=torch.bool)
    same[[5, 7]] = False
    assert torch.equal(got[:, :, same], want[:, :, same])


@gpu
def test_strips_streams_and_graphs():
    q, kb, kw, want = run(H=2, HS=1, NQ=300, NK=900, T=5, bshd=True)
    need = skl.streamkl_select_blocks_workspace_bytes(1, 2, 1, 300, 900, 64, 32, 5, causal=True)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(want, 7)
    assert skl.streamkl_select_blocks(q, kb, 5, 32, 900, **kw, out=out, workspace=ws[16:], stream=st) is out
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, want)
    with pytest.raises(skl.StreamKLError):
        skl.streamkl_select_blocks(q, kb, 5, 32, 900, **kw, workspace=ws[: need - 16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = skl.streamkl_select_blocks(q, kb, 5, 32, 900, **kw)
    q.copy_(torch.randn(q.shape, device="cuda"))
    graph.replay()
    assert torch.equal(again, skl.streamkl_select_blocks(q, kb, 5, 32, 900, **kw))
    # more queries than one strip holds: 128 MB of scores
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn((1, 2, 24000, 32), generator=g, device="cuda").to(torch.bfloat16)
    kb = torch.randn((1, 2, 1875, 32), generator=g, device="cuda").to(torch.bfloat16)
    whole = skl.streamkl_select_blocks(q, kb, 4, 32, 60000)
    for i0 in range(0, 24000, 8000):
        part = skl.streamkl_select_blocks(q[:, :, i0:i0 + 8000], kb, 4, 32, 60000)
        assert torch.equal(part, whole[:, :, i0:i0 + 8000])


# Many rows of up to 256 blocks: their lists come from where the scores are made.
MANY = dict(B=19, H=32, HS=16, NQ=7, d=32)
MANY_CASES = {
    "one token": dict(NQ=1, NK=1, T=1, sink=0),
    "grouped": dict(H=64, NQ=9, NK=1500, T=6, d=128),
    "odd head dim": dict(H=16, NK=900, T=7, d=80, bs=64, bshd=True),
    "not causal": dict(NK=8192, T=12, causal=False, sink=0, local=0),
    "no forced": dict(NK=300, T=3, sink=0, local=0),
    "all forced": dict(NK=300, T=4, sink=2, local=2),
    "one place": dict(NK=3000, T=1, sink=0, local=0),
    "fewer candidates than places": dict(NQ=40, NK=200, T=16),
    "more queries than keys": dict(NQ=150, NK=40, T=3),
    "prefix": dict(NQ=12, NK=1000, prefix=[0, 177, 400, 1000, 31, 32, 33] * 2 + [999, 1, 500, 64, 65], T=5),
    "63 places": dict(NK=200 * 32, T=63),
    "64 places": dict(NK=200 * 32, T=64),
    "128 places": dict(NK=256 * 128 - 7, bs=128, T=128),
    "tiles": dict(B=4, H=8, HS=8, NQ=1250, NK=2500, T=6, bs=128),
}


@gpu
@pytest.mark.parametrize("name", MANY_CASES)
def test_lists_of_many_rows(name):
    run(**{**MANY, **MANY_CASES[name]})


@gpu
@pytest.mark.parametrize("make", [whole_numbers, equal_keys, zeros, near, cancelling])
@pytest.mark.parametrize("shape", [dict(NK=2000, T=6), dict(NK=8000, T=40, causal=False, HS=16)])
def test_ties_and_close_scores_of_many_rows(make, shape):
    run(make=make, **{**MANY, **shape})


@gpu
def test_many_rows_whose_numbers_are_not_finite():
    """Rows with such numbers stay in bounds, the others as they were; and so with those of a block."""
    q, kb, kw, want = run(**MANY, NK=2000, T=6)
    q[0, 0, 5] = float("nan")
    q[3, 9, 2, 3] = float("inf")
    got = skl.streamkl_select_blocks(q, kb, 6, 32, 2000, **kw)
    assert got.min() >= -1 and got.max() < 63
    same = torch.ones(want.shape[:3], dtype=torch.bool)
    same[0, 0, 5] = same[3, 4, 2] = False
    assert torch.equal(got[same], want[same])
    kb[18, 15, 40] = float("nan")
    got = skl.streamkl_select_blocks(q, kb, 6, 32, 2000, **kw)
    assert got.min() >= -1 and got.max() < 63
    same[18, 15] = False
    assert torch.equal(got[same], want[same])


@gpu
def test_many_rows_or_few_are_the_same():
    """A part of the batch, by the other way, has the same lists; replayed too, with other queries."""
    q, kb, kw, want = run(**MANY, NK=3000, T=9, bshd=True)
    assert torch.equal(skl.streamkl_select_blocks(q[:3], kb[:3], 9, 32, 3000, **kw), want[:3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = skl.streamkl_select_blocks(q, kb, 9, 32, 3000, **kw)
    q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(3)))
    graph.replay()
    now = skl.streamkl_select_blocks(q[4:6], kb[4:6], 9, 32, 3000, **kw)
    assert torch.equal(again[4:6], now) and not torch.equal(again, want)
    need = skl.streamkl_select_blocks_workspace_bytes(19, 32, 16, 7, 3000, 32, 32, 9, causal=True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(skl.streamkl_select_blocks(q, kb, 9, 32, 3000, **kw, workspace=ws), again)
    with pytest.raises(skl.StreamKLError):
        skl.streamkl_select_blocks(q, kb, 9, 32, 3000, **kw, workspace=ws[: need - 16])


def best_blocks(q, kb, T, bs, NK):
    """Lists of causal queries from scores in float64 on the GPU, the first and last candidate forced."""
    B, H, NQ, d = q.shape
    nb = kb.shape[2]
    s = q.double().reshape(B, kb.shape[1], -1, NQ, d).sum(2) @ kb.double().transpose(2, 3)
    at = torch.arange(nb, device=q.device)
    last = (torch.arange(NQ, device=q.device) + NK - NQ)[:, None].clamp(max=NK - 1) // bs
    s = torch.where((at == 0) | (at == last), float("inf"), torch.where(at <= last, s, -float("inf")))
    top, idx = torch.sort(s, dim=3, descending=True, stable=True)
    idx = torch.where(top[..., :T] > -float("inf"), idx[..., :T], nb).sort(3)[0]
    return torch.where(idx < nb, idx, -1).int()


@gpu
@pytest.mark.parametrize("T", [3, 16, 40, 63])
def test_lists_of_full_tiles_keep_their_error_bound(T):
    """All four warps of a tile hold rows: their lists go where the last queries were, from which |q| is found.  Keys one
    rounding apart, so that a |q| of anything else gives other lists."""
    g = torch.Generator().manual_seed(T)
    q, kb = near(torch.randn((5, 32, 500, 32), generator=g), torch.randn((5, 16, 64, 32), generator=g))
    q, kb = q.to(torch.bfloat16).cuda(), kb.to(torch.bfloat16).cuda()
    want = best_blocks(q, kb, T, 32, 2048)
    for _ in range(3):
        assert torch.equal(skl.streamkl_select_blocks(q, kb, T, 32, 2048, causal=True), want)
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK


def many_heads(H, d, bump, early):
    """Equal heads on one list, whose fp32 sums grow to 2^19 and more: there they lose what block 1 has ahead of block 0,
    a little for each head; block 2 is ahead by a gain of the first heads, which they keep."""
    q, kb = torch.ones((1, H, 1, d)), torch.ones((1, 1, 4, d))
    q[:, :H // 2 + 200, :, 0] = 0.0
    q[:, early:, :, 1] = 0.0
    kb[:, :, 1, 0] += bump * 2.0 ** -7
    kb[:, :, 2, 1] += 2.0 ** -3
    return q.to(torch.bfloat16).cuda(), kb.to(torch.bfloat16).cuda()


@gpu
@pytest.mark.parametrize("H,d,bump,early", [(65535, 16, 6, 8800), (65535, 16, 6, 12000), (65535, 16, 7, 12000),
                                            (65535, 32, 14, 10400), (4096, 128, 3, 700)])
def test_many_equal_heads_on_one_list(H, d, bump, early):
    q, kb = many_heads(H, d, bump, early)
    score = (q.double().sum(1) @ kb[0].double().transpose(1, 2)).flatten()
    got = skl.streamkl_select_blocks(q, kb, 1, 32, 128, sink=0, local=0)
    assert got.item() == score.argmax().item()


@gpu
@pytest.mark.parametrize("shape", [dict(H=64, HS=1, NQ=60, NK=2000, T=6), dict(B=19, H=64, HS=16, NQ=7, NK=2000, T=6, d=32)])
@pytest.mark.parametrize("make", [near, cancelling, whole_numbers])
def test_close_scores_of_many_heads(make, shape):
    """Heads that point the same way: their terms add up to the root of their number times the norm of all of them."""
    def alike(q, kb):
        q[:] = q[:, :1]
        return make(q, kb)
    run(make=alike, **shape)


def test_ends_taken_by_default(L):
    assert skl._ends(4, None, None) == (1, 1) and skl._ends(2, None, None) == (1, 1)
    assert skl._ends(1, None, None) == (0, 1)
    assert skl._ends(4, 4, None) == (4, 0) and skl._ends(4, None, 4) == (0, 4) and skl._ends(3, 2, None) == (2, 1)
    assert skl._ends(4, 3, 2) == (3, 2)  # refused by the library
    f = skl.streamkl_select_blocks_workspace_bytes
    assert f(1, 4, 2, 100, 300, 64, 32, 1) > 0
    assert f(1, 4, 2, 100, 300, 64, 32, 1, sink=1, local=1) == 0


@gpu
def test_one_place_by_default():
    """The last candidate, as the defaults say; the best with none forced."""
    q, kb, kw, _ = run(NQ=100, NK=300, T=1, sink=0, local=0)
    del kw["sink"], kw["local"]
    got = skl.streamkl_select_blocks(q, kb, 1, 32, 300, **kw)
    assert torch.equal(got.flatten(0, 1).squeeze(2).cpu(), ((torch.arange(100) + 200) // 32).int().expand(2, 100))


@gpu
def test_a_candidate_may_hold_no_key_of_the_query():
    """Ids out of order: a block whose smallest and largest enclose the query's is a candidate, one beside them is not."""
    ids = torch.tensor([[0] * 16 + [2] * 16 + [1] * 32 + [3] * 32 + [-1] * 16 + [1] * 16], dtype=torch.int32, device="cuda")
    doc_q = torch.tensor([[1, 0, 3, -1, 2]], dtype=torch.int32, device="cuda")
    q = torch.ones((1, 1, 5, 16), dtype=torch.bfloat16, device="cuda")
    kb = torch.ones((1, 1, 4, 16), dtype=torch.bfloat16, device="cuda")
    got = skl.streamkl_select_blocks(q, kb, 4, 32, 128, doc_q=doc_q, doc_k=ids)
    assert got[0, 0].tolist() == [[0, 1, 3, -1], [0, -1, -1, -1], [2, -1, -1, -1], [-1] * 4, [0, -1, -1, -1]]
