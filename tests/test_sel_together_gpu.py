"""Distilling attention over selected blocks as it is used: queries and keys
without positions are turned, a key is made for each block, blocks are selected,
the KL over them is taken and its gradient goes back to the unturned ones; all
against float64 and its autograd, over the same lists."""

import math

import numpy as np
import pytest
import torch

import attention_distillation_kl_gb300 as skl

pytestmark = pytest.mark.gpu


def turn64(x, pos, freq, sections):
    """x [B, H, N, d] in float64, pairs (p, p + R)."""
    R = freq.shape[0]
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    a = (pos.double()[axis].permute(1, 2, 0) * freq.double())[:, None]
    u, v = x[..., :R], x[..., R:2 * R]
    return torch.cat((u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos(), x[..., 2 * R:]), 3)


def setting(B=1, H=8, HK=2, N=500, d=64, bs=32, T=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = {n: torch.randn((B, h, N, d), generator=g).to(torch.bfloat16).cuda()
         for n, h in (("q1", H), ("k1", HK), ("q2", H), ("k2", HK))}
    n = torch.arange(N)
    pos = torch.stack((n // 64, n // 8 % 8, n % 8)).int()[:, None].expand(3, B, N).cuda()
    sections = [8, 12, 8]
    freq = (1000.0 ** (-torch.arange(28) / 28)).float().cuda()
    return x, pos, sections, freq


def test_the_whole_way():
    x, pos, sections, freq = setting()
    bs, T, scale = 32, 5, 1 / 8
    rot = skl.Rotary(freq, pos, sections)
    sides = [skl.AttnSide(x["q" + t], x["k" + t], scale, rotary_q=rot, rotary_k=rot) for t in "12"]
    p1, p2 = sides
    kb = skl.streamkl_pool_blocks(p2.k, bs)
    blocks = skl.streamkl_select_blocks(p2.q, kb, T, bs, 500, causal=True)
    rows = skl.streamkl_fwd_sel(p1, p2, blocks, bs, causal=True)
    dkl = torch.ones_like(rows[0])
    got = {t: skl.streamkl_bwd_sel(p1, p2, blocks, bs, *rows, dkl, m, causal=True)
           for t, m in (("1", skl.STREAMKL_GRAD_P1), ("2", skl.STREAMKL_GRAD_P2))}
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK

    leaf = {n: v.double().requires_grad_() for n, v in x.items()}
    n = torch.arange(500, device="cuda")
    on = torch.zeros((1, 2, 500, 17), dtype=torch.bool, device="cuda")
    on.scatter_(3, torch.where(blocks >= 0, blocks, 16).long(), True)
    vis = on[..., :16].repeat_interleave(bs, 3)[..., :500].repeat_interleave(4, 1) & (n[None, :] <= n[:, None])
    lp = []
    for t in "12":
        q, k = (turn64(leaf[c + t], pos, freq, sections) for c in "qk")
        s = scale * q @ k.repeat_interleave(4, 1).transpose(2, 3)
        lp.append(torch.log_softmax(s.masked_fill(~vis, -1e30), 3))
    kl = torch.where(vis, lp[0].exp() * (lp[0] - lp[1]), 0.0).sum(3)
    # one rounding of q and k to bf16 after they are turned: scores off by 2 sqrt(d) 2^-9 of |q||k| / d at most in
    # the mean, some 0.01 here; KL, of size 1, by twice that
    assert (rows[0].double() - kl).abs().mean() <= 0.02 and (rows[0].double() - kl).norm() <= 0.03 * kl.norm()
    kl.sum().backward()
    for t in "12":
        for g, name in zip(got[t], "qk"):
            want = leaf[name + t].grad
            # the turned q and k, dS and the gradient twice are rounded to bf16 (2^-9 in the mean each), and P moves
            # with the scores
            assert (g.double() - want).norm() <= 0.05 * want.norm(), (t, name)


def test_turned_sides_are_the_rotated_tensors():
    x, pos, sections, freq = setting(N=300)
    rot = skl.Rotary(freq, pos[..., :300], sections)
    by_hand = {n: skl.streamkl_rotate(v, rot) for n, v in x.items()}
    turned = [skl.AttnSide(x["q" + t], x["k" + t], 0.125, rotary_q=rot, rotary_k=rot) for t in "12"]
    plain = [skl.AttnSide(by_hand["q" + t], by_hand["k" + t], 0.125) for t in "12"]
    blocks = torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 1, 300, 3).contiguous()
    for fwd, bwd, args in ((skl.streamkl_fwd_sel, skl.streamkl_bwd_sel, (blocks, 64)),
                           (skl.streamkl_fwd_mod, skl.streamkl_bwd_mod, ())):
        a, b = (fwd(*s, *args, causal=True) for s in (turned, plain))
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        kw = {} if args else dict(deterministic=True)
        da, db = (bwd(*s, *args, *a, torch.ones_like(a[0]), causal=True, **kw) for s in (turned, plain))
        for u, v in zip(da[:2], db[:2]):
            assert torch.equal(u, skl.streamkl_rotate(v, rot, inverse=True))
    # only q turned, on a stream of its own
    st = torch.cuda.Stream()
    half = skl.AttnSide(x["q2"], by_hand["k2"], 0.125, rotary_q=rot)
    st.wait_stream(torch.cuda.current_stream())
    rows = skl.streamkl_fwd_sel(plain[0], half, blocks, 64, causal=True, stream=st)
    dq, dk = skl.streamkl_bwd_sel(plain[0], half, blocks, 64, *rows, torch.ones_like(rows[0]), causal=True, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    want = skl.streamkl_bwd_sel(*plain, blocks, 64, *rows, torch.ones_like(rows[0]), causal=True)
    assert torch.equal(dq, skl.streamkl_rotate(want[0], rot, inverse=True)) and torch.equal(dk, want[1])
    with pytest.raises(ValueError):
        skl.AttnSide(x["q1"], x["k1"], 0.125, rotary_q=skl.Rotary(freq, pos[..., :299], sections))


def test_captured_steps_in_turn():
    """Two captured steps that share nothing, replayed in turn, give what they gave alone."""
    graphs, outs, data = [], [], []
    for seed in (1, 2):
        x, pos, sections, freq = setting(N=256, seed=seed)
        rot = skl.Rotary(freq, pos[..., :256], sections)

        def step():
            p1, p2 = (skl.AttnSide(x["q" + t], x["k" + t], 0.125, rotary_q=rot, rotary_k=rot) for t in "12")
            kb = skl.streamkl_pool_blocks(p2.k, 32)
            blocks = skl.streamkl_select_blocks(p2.q, kb, 4, 32, 256, causal=True)
            rows = skl.streamkl_fwd_sel(p1, p2, blocks, 32, causal=True)
            return rows[0], *skl.streamkl_bwd_sel(p1, p2, blocks, 32, *rows, torch.ones_like(rows[0]), causal=True)

        alone = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append(graph)
        outs.append(out)
        data.append((alone, x, rot))  # a graph reads its inputs where they were
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for out, (alone, *_) in zip(outs, data):
        assert [torch.equal(a, b) for a, b in zip(out, alone)] == [True] * 3


def far(t, at):
    """t with its heads 2^31 values and more apart (and the whole of `at` behind)."""
    B, H, N, d = t.shape
    y = FAR.as_strided((B, H, N, d), (H * 2 ** 31, 2 ** 31 + 64, d, 1), at)
    y.copy_(t)
    return y


def test_strides_beyond_32_bits():
    """Heads further apart than 32 bits count: the results of dense tensors."""
    global FAR
    FAR = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    x, pos, sections, freq = setting(H=2, HK=2, N=200)
    rot = skl.Rotary(freq, pos[..., :200], sections)
    results = []
    for place in (lambda t, n: t, lambda t, n: far(t, n * 2 ** 16)):
        q1, k1, q2, k2 = (place(x[n], at) for at, n in enumerate(("q1", "k1", "q2", "k2")))

        def empty(at, n=200):
            return place(torch.zeros_like(x["q1"][:, :, :n]), at)

        turned = [skl.streamkl_rotate(t, rot, out=empty(4 + at)) for at, t in enumerate((q1, k1, q2, k2))]
        kb = skl.streamkl_pool_blocks(turned[3], 32, out=empty(8, 7))
        blocks = skl.streamkl_select_blocks(turned[2], kb, 3, 32, 200, causal=True)
        p1, p2 = skl.AttnSide(turned[0], turned[1], 0.125), skl.AttnSide(turned[2], turned[3], 0.125)
        rows = skl.streamkl_fwd_sel(p1, p2, blocks, 32, causal=True)
        grads = skl.streamkl_bwd_sel(p1, p2, blocks, 32, *rows, torch.ones_like(rows[0]), causal=True,
                                     dq=empty(9), dk=empty(10))
        results.append([t.clone() for t in (*turned, kb, blocks, *rows, *grads)])
    assert [torch.equal(a, b) for a, b in zip(*results)] == [True] * len(results[0])
    del FAR


def test_threads_with_streams_of_their_own():
    """Calls at once from several threads, each on its stream, give what they give alone."""
    import threading
    work = []
    for seed in range(3):
        x, pos, sections, freq = setting(N=300 + 100 * seed, seed=seed)
        rot = skl.Rotary(freq, pos, sections)

        def step(x=x, rot=rot, N=300 + 100 * seed):
            p1, p2 = (skl.AttnSide(x["q" + t], x["k" + t], 0.125, rotary_q=rot, rotary_k=rot) for t in "12")
            blocks = skl.streamkl_select_blocks(p2.q, skl.streamkl_pool_blocks(p2.k, 32), 4, 32, N, causal=True)
            rows = skl.streamkl_fwd_sel(p1, p2, blocks, 32, causal=True)
            return *rows, *skl.streamkl_bwd_sel(p1, p2, blocks, 32, *rows, torch.ones_like(rows[0]), causal=True)

        work.append((step, [t.clone() for t in step()]))
    torch.cuda.synchronize()
    wrong, rounds = [], 20

    def loop(step, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(rounds):
                    got = step()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append("another result")
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and skl.streamkl_get_device_status() == skl.STREAMKL_OK


def test_gradients_by_differences():
    """A step along a gradient, forward and back, moves the KL as the gradient says (the blocks held fixed)."""
    x, pos, sections, freq = setting(H=4, N=300, d=64, seed=5)
    rot = skl.Rotary(freq, pos, sections)
    w = torch.rand((1, 4, 300), generator=torch.Generator().manual_seed(6)).cuda()

    def sides(**other):
        y = {**x, **other}
        return [skl.AttnSide(y["q" + t], y["k" + t], 0.125, rotary_q=rot, rotary_k=rot) for t in "12"]

    p1, p2 = sides()
    blocks = skl.streamkl_select_blocks(p2.q, skl.streamkl_pool_blocks(p2.k, 32), 4, 32, 300, causal=True)
    rows = skl.streamkl_fwd_sel(p1, p2, blocks, 32, causal=True)
    for t, mode in (("1", skl.STREAMKL_GRAD_P1), ("2", skl.STREAMKL_GRAD_P2)):
        grads = skl.streamkl_bwd_sel(p1, p2, blocks, 32, *rows, w, mode, causal=True)
        for name, g in zip("qk", grads):
            at = x[name + t]
            # Steps of 0.5 % of the values, as far as bf16 takes them: what is counted is the step after rounding.  Scores
            # then move by 0.04 in the mean and some 0.1 where the gradient is large, and the third derivative's share is
            # a sixth of that squared, times a few: 0.5 %.  Rounding the turned q and k moves the difference by
            # 2^-9 |g x| against 0.01 |g| |x|, of 76800 or 19200 independent values: below 0.2 %.
            step = 0.005 * at.float().norm() / g.float().norm() * g.float()
            up, down = (at.float() + step).bfloat16(), (at.float() - step).bfloat16()
            ends = [(skl.streamkl_fwd_sel(*sides(**{name + t: y}), blocks, 32, causal=True)[0].double() * w).sum()
                    for y in (up, down)]
            says = (g.double() * (up.double() - down.double())).sum()
            assert abs((ends[0] - ends[1]) - says) <= 0.02 * abs(says), (name, t)
