"""The calls over modified scores, without a GPU: refusals (every call here
fails validation before any CUDA call), workspace sizes, and the float64
definitions the GPU tests rely on, checked by finite differences."""

import ctypes
import os

import numpy as np
import pytest

import attention_distillation_kl_gb300 as skl
import mod_reference as ref

A = 4096  # a 16-byte aligned fake address: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(skl.library_path):
        import __graft_entry__
        __graft_entry__.build()
    return skl.lib()


def view(data=A, n=128, heads=2, d=64):
    return skl._View(data, heads * n * d, n * d, d)


def side(**kw):
    a = dict(q=view(), k=view(), d=64, HK=2, scale=0.125, softcap=0.0, slopes=None, table=None, num_buckets=0,
             max_distance=0, bidirectional=0)
    a.update(kw)
    return skl._Side(*(a[f] for f, _ in skl._Side._fields_))


def seen(causal=0, prefix=None, doc_q=None, doc_k=None):
    return skl._Visible(causal, prefix, doc_q, doc_k)


def fwd(L, s1=None, s2=None, vis=None, B=1, H=2, NQ=128, NK=128, splits=1, ws=A, ws_bytes=1 << 40, out=(A, A, A)):
    return L.streamkl_fwd_mod(s1 or side(), s2 or side(), vis or seen(), B, H, NQ, NK, splits, ws, ws_bytes, *out, None)


def bwd(L, s1=None, s2=None, vis=None, B=1, H=2, NQ=128, NK=128, rows=(A, A, A, A), mode=0, det=0, dq=None, dk=None,
        dtable=None, ws=A, ws_bytes=1 << 40):
    return L.streamkl_bwd_mod(s1 or side(), s2 or side(), vis or seen(), B, H, NQ, NK, *rows, mode, det, dq or view(),
                              dk or view(), dtable, ws, ws_bytes, None)


TABLE = dict(table=A, num_buckets=32, max_distance=128)

BAD_SIDES = [
    (dict(scale=0.0), skl.STREAMKL_INVALID_ARG), (dict(scale=float("nan")), skl.STREAMKL_INVALID_ARG),
    (dict(scale=2e4), skl.STREAMKL_INVALID_ARG), (dict(softcap=-1.0), skl.STREAMKL_INVALID_ARG),
    (dict(softcap=float("inf")), skl.STREAMKL_INVALID_ARG), (dict(softcap=1e-5), skl.STREAMKL_INVALID_ARG),
    (dict(HK=0), skl.STREAMKL_INVALID_ARG), (dict(HK=3), skl.STREAMKL_INVALID_ARG),
    (dict(d=8), skl.STREAMKL_UNSUPPORTED), (dict(d=72), skl.STREAMKL_UNSUPPORTED),
    (dict(d=144), skl.STREAMKL_UNSUPPORTED),
    (dict(slopes=A, **TABLE), skl.STREAMKL_INVALID_ARG), (dict(slopes=A + 2), skl.STREAMKL_INVALID_ARG),
    (dict(TABLE, num_buckets=1), skl.STREAMKL_INVALID_ARG), (dict(TABLE, num_buckets=65), skl.STREAMKL_INVALID_ARG),
    (dict(TABLE, num_buckets=31, bidirectional=1), skl.STREAMKL_INVALID_ARG),
    (dict(TABLE, num_buckets=2, bidirectional=1), skl.STREAMKL_INVALID_ARG),
    (dict(TABLE, bidirectional=2), skl.STREAMKL_INVALID_ARG),
    (dict(TABLE, max_distance=16), skl.STREAMKL_INVALID_ARG),  # half of the buckets hold one distance each
    (dict(TABLE, max_distance=5000), skl.STREAMKL_INVALID_ARG),
    (dict(q=view(0)), skl.STREAMKL_INVALID_ARG), (dict(k=view(A + 8)), skl.STREAMKL_INVALID_ARG),
    (dict(q=skl._View(A, 0, 128 * 64, 60)), skl.STREAMKL_INVALID_ARG),    # stride not a multiple of 8
    (dict(q=skl._View(A, 0, 0, 64)), skl.STREAMKL_INVALID_ARG),           # heads broadcast
    (dict(k=skl._View(A, 0, -64, 64)), skl.STREAMKL_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_SIDES)
def test_bad_sides_are_refused(L, kw, status):
    for pair in ((side(**kw), None), (None, side(**kw))):
        assert fwd(L, *pair) == status
        assert bwd(L, *pair) == status


@pytest.mark.parametrize("kw", [
    dict(vis=seen(causal=2)), dict(vis=seen(prefix=A)), dict(vis=seen(causal=1, prefix=A + 1)),
    dict(vis=seen(doc_q=A)), dict(vis=seen(doc_k=A)), dict(vis=seen(doc_q=A, doc_k=A + 2)),
    dict(B=-1), dict(NK=0), dict(NQ=-1), dict(B=70000), dict(ws=None, s1=side(**TABLE)),
    dict(ws=A + 8, s1=side(**TABLE)), dict(ws_bytes=8, s1=side(**TABLE)),
])
def test_bad_calls_are_refused(L, kw):
    assert fwd(L, **kw) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, **kw) == skl.STREAMKL_INVALID_ARG


def test_forward_refusals(L):
    assert fwd(L, splits=-1) == skl.STREAMKL_INVALID_ARG
    assert fwd(L, splits=1025) == skl.STREAMKL_INVALID_ARG
    assert fwd(L, splits=4, ws_bytes=5 * 4 * 4 * 2 * 128 - 1) == skl.STREAMKL_INVALID_ARG
    for out in ((0, A, A), (A, A + 4, A), (A, A, 0)):
        assert fwd(L, out=out) == skl.STREAMKL_INVALID_ARG
    assert L.streamkl_fwd_mod(None, side(), seen(), 1, 2, 128, 128, 1, A, 1 << 40, A, A, A, None) == \
        skl.STREAMKL_INVALID_ARG


def test_backward_refusals(L):
    assert bwd(L, mode=2) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, det=2) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, dtable=A) == skl.STREAMKL_INVALID_ARG                            # side 2 has no table
    assert bwd(L, dtable=A, s1=side(**TABLE)) == skl.STREAMKL_INVALID_ARG          # nor does the other side's count
    assert bwd(L, dtable=A + 2, s2=side(**TABLE)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, dq=view(0)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, dk=view(A + 2)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, rows=(A, 0, A, A)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, ws=None) == skl.STREAMKL_INVALID_ARG
    need = L.streamkl_bwd_mod_workspace_bytes(side(), side(), seen(), 1, 2, 128, 128, 0, 0, 0)
    assert need >= 2 * 128 * 64 * 4 and bwd(L, ws_bytes=need - 1) == skl.STREAMKL_INVALID_ARG


def test_empty_problems_do_nothing(L):
    none = side(q=view(0), k=view(0))
    assert fwd(L, none, none, NQ=0, ws=None, out=(0, 0, 0)) == skl.STREAMKL_OK
    assert fwd(L, none, none, B=0, ws=None, out=(0, 0, 0)) == skl.STREAMKL_OK
    assert bwd(L, none, none, B=0, ws=None, rows=(0, 0, 0, 0)) == skl.STREAMKL_OK


def test_workspace_bytes(L):
    f, b = L.streamkl_fwd_mod_workspace_bytes, L.streamkl_bwd_mod_workspace_bytes
    assert f(side(), side(), seen(), 1, 2, 128, 128, 1) == 0
    assert f(side(softcap=50.0), side(slopes=A), seen(1, A), 1, 2, 128, 128, 1) == 0
    assert f(side(), side(), seen(), 1, 2, 100, 300, 3) == 5 * 4 * 3 * 2 * 100
    # a lookup row per head over 2 (128 + 256) + 1 positions, and two more
    assert f(side(**TABLE), side(), seen(), 1, 2, 128, 128, 1) == -(-2 * 771 * 4 // 16) * 16
    ids = f(side(), side(), seen(0, None, A, A), 3, 2, 130, 130, 1)
    assert ids == 2 * 3 * 256 * 4 + 2 * 3 * 2 * 16
    assert f(side(scale=0.0), side(), seen(), 1, 2, 128, 128, 1) == 0
    assert f(side(), side(), seen(), 1, 2, 128, 128, 2000) == 0
    plain = b(side(), side(), seen(), 1, 2, 128, 128, 0, 0, 1)
    assert plain == 2 * 128 * 64 * 4                                   # table_grad without a table asks for nothing
    shared = b(side(), side(HK=1), seen(), 1, 2, 128, 128, 0, 0, 0)
    assert shared == plain + 128 * 64 * 4                              # and dK of the shared key head
    assert b(side(), side(HK=1), seen(), 1, 2, 128, 128, 1, 0, 0) == plain
    assert b(side(), side(), seen(), 1, 2, 128, 128, 2, 0, 0) == 0


def test_structures_match_the_header():
    """The field order of the ctypes structures, against the header's text."""
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "streamkl.h")).read()
    for name, struct in (("view", skl._View), ("side", skl._Side), ("visible", skl._Visible)):
        body = re.search(r"typedef struct streamkl_%s \{(.*?)\} streamkl_%s;" % (name, name), text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.strip().lstrip("*") for decl in body.split(";") if decl.strip()
                  for f in re.sub(r"^\s*(const\s+)?(long long|\w+)\s*", "", decl).replace("*", "").split(",")]
        assert fields == [f for f, _ in struct._fields_], name
    assert ctypes.sizeof(skl._View) == 32 and ctypes.sizeof(skl._Visible) == 32


def test_binding_checks_its_tensors():
    import torch
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        skl.AttnSide(x, x, 0.125)


# ------------------------------------------------------------------ the definitions


def small(seed, **kw):
    g = np.random.default_rng(seed)
    B, H, HK1, HK2, NQ, NK, d = 1, 2, 2, 1, 5, 9, 8
    p = dict(q1=g.normal(size=(B, H, NQ, d)), k1=g.normal(size=(B, HK1, NK, d)), q2=g.normal(size=(B, H, NQ, d)),
             k2=g.normal(size=(B, HK2, NK, d)), causal=True, prefix=None, doc_q=None, doc_k=None)
    for t in "12":
        p.update({"scale" + t: 0.7, "cap" + t: 0.0, "slopes" + t: None, "table" + t: None, "maxd" + t: 8,
                  "both" + t: False})
    p.update(kw)
    return p, g


CASES = {
    "capped": dict(cap1=2.0, cap2=1.5),
    "slopes": dict(slopes1=np.array([0.5, 0.1]), slopes2=np.array([0.3, 0.7]), causal=False),
    "table": dict(table2=np.linspace(-1, 1, 16).reshape(2, 8), cap1=3.0),
    "both ways": dict(table1=np.linspace(-1, 1, 16).reshape(2, 8), both1=True, table2=np.ones((2, 8)), both2=True,
                      causal=False),
    "prefix": dict(prefix=np.array([6]), cap2=1.0),
    "ids": dict(doc_q=np.array([[0, 1, -1, 1, 2]]), doc_k=np.array([[0, 0, 1, 1, -1, 1, 3, 1, 1]]), causal=False),
}


@pytest.mark.parametrize("mode", ["1", "2"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_gradients_are_the_differences(name, mode):
    p, g = small(3, **CASES[name])
    w = g.uniform(0.5, 1.5, size=(1, 2, 5))
    kl, l1, l2 = ref.forward(p)[:3]
    got = ref.backward(p, kl, l1, l2, w, mode)

    def loss():
        return float((w * ref.forward(p)[0]).sum())

    h = 1e-6
    for key, grad in (("q" + mode, got[0]), ("k" + mode, got[1]), ("table" + mode, got[2])):
        if p[key] is None:
            continue
        p[key] = p[key].astype(np.float64)
        for _ in range(12):
            at = tuple(int(g.integers(n)) for n in p[key].shape)
            old = p[key][at]
            p[key][at] = old + h
            up = loss()
            p[key][at] = old - h
            down = loss()
            p[key][at] = old
            # a central difference errs by h^2 and by the loss's rounding over h
            assert abs((up - down) / (2 * h) - grad[at]) < 1e-7 + 1e-6 * abs(grad[at])


def test_buckets_at_their_borders():
    # 32 buckets up to 128, one direction: distances 0 .. 15 each their own, 16 (2^(i/16 * 3)) on
    d = np.arange(0, 200)
    b = ref.bucket(-d, 32, 128, False)
    assert list(b[:17]) == list(range(17)) and b[127] == 31 and b[128] == 31 and b[199] == 31
    assert all(np.diff(b) >= 0) and all(ref.bucket(d[1:], 32, 128, False) == 0)
    # both directions, 16 each: whole distances at a border (16, 32, 64) begin their bucket
    b = ref.bucket(-d, 32, 128, True)
    assert [b[15], b[16], b[31], b[32], b[63], b[64]] == [9, 10, 11, 12, 13, 14]
    assert all(ref.bucket(d[1:], 32, 128, True) == b[1:] + 16)


def test_a_row_that_sees_nothing():
    p, _ = small(5, doc_q=np.array([[0, -1, 4, 1, 1]]), doc_k=np.array([[0, 0, 0, 1, 1, 1, 1, -1, -1]]))
    kl, l1, l2 = ref.forward(p)[:3]
    assert np.all(kl[:, :, 1:3] == 0) and np.all(np.isinf(l1[:, :, 1:3])) and np.all(np.isinf(l2[:, :, 1:3]))
    dq = ref.backward(p, kl, l1, l2, np.ones_like(kl), "2")[0]
    assert np.all(dq[:, :, 1:3] == 0) and np.all(np.isfinite(dq))
