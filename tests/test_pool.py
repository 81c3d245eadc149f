"""The key of each block of keys: means against float64, padded keys left out."""

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


def call(L, k=None, ids=None, B=1, HK=2, NK=100, d=64, block=32, kb=None):
    return L.streamkl_pool_blocks(k or skl._View(A, 0, NK * d, d), ids, B, HK, NK, d, block,
                                  kb or skl._View(2 * A, 0, 4 * d, d), None)


@pytest.mark.parametrize("kw,status", [
    (dict(block=0), skl.STREAMKL_INVALID_ARG), (dict(block=48), skl.STREAMKL_INVALID_ARG),
    (dict(block=256), skl.STREAMKL_INVALID_ARG), (dict(d=8), skl.STREAMKL_UNSUPPORTED),
    (dict(d=144), skl.STREAMKL_UNSUPPORTED), (dict(ids=A + 2), skl.STREAMKL_INVALID_ARG),
    (dict(k=skl._View(0, 0, 64, 64)), skl.STREAMKL_INVALID_ARG), (dict(kb=skl._View(A, 0, 64, 4)), skl.STREAMKL_INVALID_ARG),
    (dict(NK=-1), skl.STREAMKL_INVALID_ARG), (dict(B=70000), skl.STREAMKL_INVALID_ARG),
])
def test_refusals(L, kw, status):
    assert call(L, **kw) == status


def test_empty_is_no_op(L):
    none = skl._View(0, 0, 0, 0)
    assert call(L, k=none, kb=none, NK=0) == skl.STREAMKL_OK


@gpu
@pytest.mark.parametrize("B,HK,NK,d,block,bshd,ids", [
    (1, 1, 1, 16, 32, False, False), (2, 3, 32, 64, 32, True, False), (1, 8, 1000, 128, 64, True, False),
    (3, 5, 531, 96, 32, False, True), (2, 2, 129, 112, 128, True, True), (1, 2, 4097, 48, 128, False, False),
    (2, 1, 300, 32, 64, True, True),
])
def test_means(B, HK, NK, d, block, bshd, ids):
    g = torch.Generator().manual_seed(NK)
    k = (torch.randn((B, HK, NK, d), generator=g) + 0.5).to(torch.bfloat16)
    doc = torch.randint(-1, 3, (B, NK), generator=g, dtype=torch.int32) if ids else None
    if ids:  # a block without a key, and padded keys that hold anything
        doc[0, :block] = -1
        k[(doc < 0)[:, None, :].expand(B, HK, NK)] = float("nan")
    dev = k.transpose(1, 2).contiguous().cuda().transpose(1, 2) if bshd else k.cuda()
    got = skl.streamkl_pool_blocks(dev, block, doc_k=None if doc is None else doc.cuda()).float().cpu().double().numpy()
    k = k.double().numpy()
    keep = np.ones((B, NK), bool) if doc is None else (doc >= 0).numpy()
    for j in range(-(-NK // block)):
        part, on = k[:, :, j * block:(j + 1) * block], keep[:, j * block:(j + 1) * block]
        part = np.where(on[:, None, :, None], part, 0.0)
        n = np.maximum(on.sum(1), 1)[:, None, None]
        want = part.sum(2) / n
        # one rounding to bf16; an fp32 sum of at most 128 values and a division
        tol = 2.0 ** -8 * np.abs(want) + (block + 2) * 2.0 ** -24 * np.abs(part).sum(2) / n
        assert np.all(np.abs(got[:, :, j] - want) <= tol)


@gpu
def test_out_and_stream():
    k = torch.randn((1, 2, 200, 64), device="cuda").to(torch.bfloat16)
    want = skl.streamkl_pool_blocks(k, 64)
    out = torch.zeros((1, 4, 2, 80), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    skl.streamkl_pool_blocks(k, 64, out=out[..., :64].transpose(1, 2), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out[..., :64].transpose(1, 2), want) and not out[..., 64:].any()
    with pytest.raises(ValueError):
        skl.streamkl_pool_blocks(k, 48)
    with pytest.raises(ValueError):
        skl.streamkl_pool_blocks(k, 64, doc_k=torch.zeros((1, 199), dtype=torch.int32, device="cuda"))
