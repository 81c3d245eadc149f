"""The calls over selected blocks, without a GPU: refusals (every call here
fails validation before any CUDA call), empty problems, structures."""

import os
import re

import numpy as np
import pytest

import attention_distillation_kl_gb300 as skl
from test_mod_cpu import A, L, seen, side, view  # noqa: F401


def blocks(selected=A, heads=1, count=4, block=32):
    return skl._Blocks(selected, heads, count, block)


def fwd(L, s1=None, s2=None, vis=None, sel=None, B=1, H=2, NQ=128, NK=128, ws=A, ws_bytes=1 << 40, out=(A, A, A)):
    return L.streamkl_fwd_sel(s1 or side(), s2 or side(), vis or seen(), sel or blocks(), B, H, NQ, NK, ws, ws_bytes,
                              *out, None)


def bwd(L, s1=None, s2=None, vis=None, sel=None, B=1, H=2, NQ=128, NK=128, ws=A, ws_bytes=1 << 40, rows=(A, A, A, A),
        mode=0, dq=None, dk=None):
    return L.streamkl_bwd_sel(s1 or side(), s2 or side(), vis or seen(), sel or blocks(), B, H, NQ, NK, *rows, mode,
                              dq or view(), dk or view(), ws, ws_bytes, None)


BAD = [
    (dict(s1=side(HK=1), s2=side(HK=1), sel=blocks(heads=1), H=1, NQ=1, NK=2 ** 31 - 1), skl.STREAMKL_INVALID_ARG),
    (dict(sel=blocks(selected=0)), skl.STREAMKL_INVALID_ARG), (dict(sel=blocks(selected=A + 2)), skl.STREAMKL_INVALID_ARG),
    (dict(sel=blocks(heads=0)), skl.STREAMKL_INVALID_ARG), (dict(sel=blocks(heads=3)), skl.STREAMKL_INVALID_ARG),
    (dict(sel=blocks(heads=4)), skl.STREAMKL_INVALID_ARG), (dict(sel=blocks(count=0)), skl.STREAMKL_INVALID_ARG),
    (dict(sel=blocks(count=129)), skl.STREAMKL_INVALID_ARG), (dict(sel=blocks(block=16)), skl.STREAMKL_INVALID_ARG),
    (dict(sel=blocks(block=96)), skl.STREAMKL_INVALID_ARG), (dict(sel=blocks(block=256)), skl.STREAMKL_INVALID_ARG),
    (dict(NK=32 * 4096 + 1), skl.STREAMKL_UNSUPPORTED),
    (dict(s1=side(softcap=30.0)), skl.STREAMKL_UNSUPPORTED), (dict(s2=side(slopes=A)), skl.STREAMKL_UNSUPPORTED),
    (dict(s2=side(table=A, num_buckets=32, max_distance=128)), skl.STREAMKL_UNSUPPORTED),
    (dict(s1=side(scale=0.0)), skl.STREAMKL_INVALID_ARG), (dict(s1=side(d=72)), skl.STREAMKL_UNSUPPORTED),
    (dict(s1=side(q=view(A + 8))), skl.STREAMKL_INVALID_ARG), (dict(s2=side(k=view(0))), skl.STREAMKL_INVALID_ARG),
    (dict(vis=seen(causal=2)), skl.STREAMKL_INVALID_ARG), (dict(vis=seen(prefix=A)), skl.STREAMKL_INVALID_ARG),
    (dict(vis=seen(doc_q=A)), skl.STREAMKL_INVALID_ARG),
    (dict(ws=0), skl.STREAMKL_INVALID_ARG), (dict(ws=A + 8), skl.STREAMKL_INVALID_ARG), (dict(ws_bytes=16), skl.STREAMKL_INVALID_ARG),
    (dict(B=-1), skl.STREAMKL_INVALID_ARG), (dict(NK=0), skl.STREAMKL_INVALID_ARG), (dict(B=70000), skl.STREAMKL_INVALID_ARG),
    (dict(NQ=1 << 25, H=1, s1=side(HK=1), s2=side(HK=1)), skl.STREAMKL_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_calls_are_refused(L, kw, status):  # noqa: F811
    assert fwd(L, **kw) == status
    assert bwd(L, **kw) == status


def test_backward_refusals(L):  # noqa: F811
    assert bwd(L, mode=2) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, rows=(A, 0, A, A)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, rows=(A, A, A, A + 4)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, dq=view(0)) == skl.STREAMKL_INVALID_ARG
    assert bwd(L, dk=view(A + 2)) == skl.STREAMKL_INVALID_ARG
    need = L.streamkl_bwd_sel_workspace_bytes(side(), side(), seen(), blocks(), 1, 2, 128, 128, 0)
    assert need >= 2 * 128 * 64 * 4 and bwd(L, ws_bytes=need - 1) == skl.STREAMKL_INVALID_ARG
    assert L.streamkl_bwd_sel_workspace_bytes(side(), side(), seen(), blocks(), 1, 2, 128, 128, 2) == 0


@pytest.mark.parametrize("mode", ["1", "2"])
def test_reference_gradients_by_differences(mode):
    """The float64 definitions that the GPU tests compare with: forward and backward fit together."""
    import sel_reference as ref
    g = np.random.default_rng(4)
    H, NQ, NK, d = 2, 7, 11, 3
    p = {n: g.standard_normal((1, h, n_, d)) for n, h, n_ in (("q1", H, NQ), ("k1", 1, NK), ("q2", H, NQ), ("k2", H, NK))}
    for t in "12":
        p.update({"scale" + t: 0.7, "cap" + t: 0.0, "slopes" + t: None, "table" + t: None})
    p.update(blocks=g.integers(-1, 4, (1, 2, NQ, 2)), bs=4, causal=True, prefix=None, doc_q=None, doc_k=None)
    w = g.standard_normal((1, H, NQ))
    rows = ref.forward(p)[:3]
    grads = dict(zip(("q", "k"), ref.backward(p, *rows, w, mode)[:2]))
    h = 1e-5
    for name, grad in grads.items():
        x = p[name + mode]
        for at in list(np.ndindex(x.shape))[::5]:
            old = x[at]
            x[at] = old + h
            up = (w * ref.forward(p)[0]).sum()
            x[at] = old - h
            down = (w * ref.forward(p)[0]).sum()
            x[at] = old
            # central differences: an error of h^2 / 6 times a third derivative (of order 10 here), and 2^-53 / h
            assert abs((up - down) / (2 * h) - grad[at]) <= 1e-7


def test_forward_outputs_are_checked(L):  # noqa: F811
    for out in ((0, A, A), (A, A + 4, A), (A, A, 0)):
        assert fwd(L, out=out) == skl.STREAMKL_INVALID_ARG


def test_empty_problems_do_nothing(L):  # noqa: F811
    none = side(q=view(0), k=view(0))
    for kw in (dict(NQ=0), dict(B=0)):
        assert fwd(L, none, none, sel=blocks(selected=0), ws=0, out=(0, 0, 0), **kw) == skl.STREAMKL_OK
    assert bwd(L, none, none, sel=blocks(selected=0), ws=0, rows=(0, 0, 0, 0), B=0) == skl.STREAMKL_OK


def test_workspace_bytes(L):  # noqa: F811
    f = L.streamkl_fwd_sel_workspace_bytes
    small = f(side(), side(), seen(), blocks(), 1, 2, 128, 128)
    assert small >= 20 * 2 * 128 * 4
    assert f(side(), side(), seen(), blocks(count=0), 1, 2, 128, 128) == 0
    assert f(side(), side(), seen(), blocks(), 1, 2, 0, 128) == 0
    assert f(side(), side(), seen(0, None, A, A), blocks(), 1, 2, 128, 128) == small + 2 * 128 * 4 + 2 * 16


def test_structures_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "streamkl.h")).read()
    for name, struct in (("blocks", skl._Blocks), ("rotary", skl._Rotary)):
        body = re.search(r"typedef struct streamkl_%s \{(.*?)\} streamkl_%s;" % (name, name), text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = []
        for decl in body.split(";"):
            for part in decl.split(","):
                m = re.search(r"(\w+)\s*(?:\[\d+\])?\s*$", part.strip())
                if m:
                    fields.append(m.group(1))
        assert fields == [f for f, _ in struct._fields_], name


def test_calls_take_their_arguments_by_name():
    import torch
    x = torch.zeros((1, 1, 8, 16), dtype=torch.bfloat16)  # not on a GPU: refused for that, behind the wrappers
    with pytest.raises(TypeError, match="x must be a CUDA"):
        skl.streamkl_rotate(rotary=None, x=x)
    with pytest.raises(TypeError, match="k must be a CUDA"):
        skl.streamkl_pool_blocks(k=x, block=32)
    with pytest.raises(TypeError, match="q must be a CUDA"):
        skl.streamkl_select_blocks(q=x, kb=x, count=4, block=32, NK=100)
    with pytest.raises(TypeError, match="missing"):
        skl.streamkl_pool_blocks()


@pytest.mark.gpu
def test_results_of_arguments_by_name():
    import torch
    q = torch.randn((1, 4, 100, 32), device="cuda").to(torch.bfloat16)
    k = torch.randn((1, 2, 100, 32), device="cuda").to(torch.bfloat16)
    kb = skl.streamkl_pool_blocks(k=k, block=32)
    assert torch.equal(kb, skl.streamkl_pool_blocks(k, 32))
    assert torch.equal(skl.streamkl_select_blocks(q=q, kb=kb, count=3, block=32, NK=100),
                       skl.streamkl_select_blocks(q, kb, 3, 32, 100))
