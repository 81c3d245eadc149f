"""The calls over modified scores handed another stream than the current one:
what they allocate belongs to that stream.  (Memory that the current stream
has freed may still be in use there, and `stream` does not wait for that.)"""

import contextlib
import types

import pytest
import torch

import attention_distillation_kl_gb300 as skl


def test_a_calls_own_tensors_are_made_on_its_stream(monkeypatch):
    where, made, marked = [None], [], []

    @contextlib.contextmanager
    def on(stream):
        where[0] = stream
        yield
        where[0] = None

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "here")
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(where[0]) or empty(*a, **k))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append(s))
    cpu, other = torch.device("cpu"), types.SimpleNamespace(cuda_stream=1)
    skl._mod_workspace(None, 64, cpu, other)
    skl._mod_rows((None, None, None), ("kl", "lse1", "lse2"), (1, 2, 3), cpu, other)
    assert made == [other] * 4
    assert marked == ["here"] * 3  # the outputs go on on the caller's stream; the workspace does not
    # a given output is the caller's
    made.clear(), marked.clear()
    given = empty(1, 2, 3)
    out = skl._mod_rows((given, None, None), ("kl", "lse1", "lse2"), (1, 2, 3), cpu, other)
    assert out[0] is given and made == [other] * 2 and marked == ["here"] * 2


def test_a_stream_of_another_device_is_refused():
    one = types.SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(ValueError):
        skl._check_stream(one, torch.device("cuda:0"))
    skl._check_stream(types.SimpleNamespace(device=torch.device("cuda:0")), torch.device("cuda:0"))
    skl._check_stream(None, torch.device("cuda:0"))


@pytest.mark.gpu
def test_work_pending_on_the_current_stream_does_not_reach_the_results():
    """Freed memory of the current stream with a late write still queued there: the calls on another stream must not
    be given it."""
    from test_mod_gpu import problem, sides
    dev, kw, where, p = problem(seed=50, B=2, docs="packed", NQ=300, NK=300, H=4, HK2=2, bias2="one way")
    p1, p2 = sides(dev, kw)
    rows = skl.streamkl_fwd_mod(p1, p2, **where)
    dkl = torch.ones_like(rows[0])
    want = [t.clone() for t in list(rows) + list(skl.streamkl_bwd_mod(p1, p2, *rows, dkl, **where, deterministic=True))]
    sizes = [t.numel() * t.element_size() for t in want] + \
        [skl.streamkl_fwd_mod_workspace_bytes(p1, p2, **where), skl.streamkl_bwd_mod_workspace_bytes(p1, p2, **where,
                                                                                                   deterministic=True)]
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # some 50 ms on the current stream
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x5a)  # written after that, freed now
        got = list(skl.streamkl_fwd_mod(p1, p2, **where, stream=s))
        got += skl.streamkl_bwd_mod(p1, p2, *got, dkl, **where, deterministic=True, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert skl.streamkl_get_device_status() == skl.STREAMKL_OK


PLAIN = ["streamkl_fwd", "streamkl_fwd_splitk", "streamkl_fwd_splitk_noalloc", "streamkl_bwd", "streamkl_fwd_scaled",
         "streamkl_fwd_splitk_scaled", "streamkl_bwd_scaled", "streamkl_fwd_gqa", "streamkl_fwd_splitk_gqa",
         "streamkl_bwd_gqa", "streamkl_bwd_gqa_ws", "streamkl_bwd_both"]


def test_the_plain_calls_run_on_their_stream_as_a_whole(monkeypatch):
    import inspect
    where, marked = [None], []

    @contextlib.contextmanager
    def on(stream):
        where[0] = stream
        yield
        where[0] = None

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "here")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append(s))

    @skl._on_its_stream
    def call(a, b=2, stream=None):
        return [torch.full((1,), float(where[0] is not None))]

    for out, n in ((call(1, 2, "other"), 1), (call(1, stream="other"), 1), (call(1), 0), (call(1, 2, None), 0)):
        assert float(out[0]) == n
    assert marked == ["here"] * 2
    for name in PLAIN:
        assert list(inspect.signature(getattr(skl, name)).parameters)[-1] == "stream"
        assert hasattr(getattr(skl, name), "__wrapped__"), name


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 4])
def test_work_pending_on_the_current_stream_does_not_reach_the_plain_results(splits):
    g = torch.Generator().manual_seed(3)
    x = [torch.randn((1, 4, 512, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    dkl = torch.ones((1, 4, 512), device="cuda")

    def calls(**kw):
        rows = skl.streamkl_fwd_splitk(*x, 0.125, True, splits, **kw) if splits else skl.streamkl_fwd(*x, 0.125, True, **kw)
        return list(rows) + list(skl.streamkl_bwd(*x, 0.125, True, *rows, dkl, deterministic=True, **kw))

    want = [t.clone() for t in calls()]
    sizes = [t.numel() * 4 for t in want] + [skl.streamkl_fwd_splitk_workspace_bytes(1, 4, 512, max(splits, 1))]
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x5a)
        got = calls(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def turned_side(made_on, q=True, k=True):
    t = [torch.zeros(1), torch.zeros(1)]
    return types.SimpleNamespace(device=torch.device("cuda:0"), q=t[0], k=t[1], made_on=made_on,
                                 rotary_q="r" if q else None, rotary_k="r" if k else None)


def test_turned_copies_are_kept_for_the_stream_that_uses_them(monkeypatch):
    marked = []
    here, other = types.SimpleNamespace(cuda_stream=1), types.SimpleNamespace(cuda_stream=2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: marked.append((t, s)))
    plain, same, away = turned_side(None, False, False), turned_side(1), turned_side(2, q=False)

    def marks(p1, p2, stream):
        marked.clear()
        skl._turned(p1, p2, stream)
        return [(id(t), s.cuda_stream) for t, s in marked]

    assert marks(plain, same, None) == []  # used where it was made
    assert marks(plain, away, None) == [(id(away.k), 1)]
    assert marks(same, plain, other) == [(id(same.q), 2), (id(same.k), 2)]
    assert marks(away, same, other) == [(id(same.q), 2), (id(same.k), 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("calls", ["mod", "sel"])
def test_a_side_dropped_while_another_stream_reads_its_copies(calls):
    """The current stream, not the one that the side was made on: its memory is not handed out before that is done."""
    n = torch.arange(256, dtype=torch.int32, device="cuda")[None]
    x = [torch.randn((1, 4, 256, 64), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(4)]
    rot = skl.Rotary((100.0 ** (-torch.arange(32, device="cuda") / 32)).float(), n)
    blocks = torch.arange(8, dtype=torch.int32, device="cuda").expand(1, 4, 256, 8).contiguous()

    def use(p1, p2):
        if calls == "mod":
            rows = skl.streamkl_fwd_mod(p1, p2, causal=True)
            return (*rows, *skl.streamkl_bwd_mod(p1, p2, *rows, torch.ones_like(rows[0]), causal=True, deterministic=True)[:2])
        rows = skl.streamkl_fwd_sel(p1, p2, blocks, 32, causal=True)
        return (*rows, *skl.streamkl_bwd_sel(p1, p2, blocks, 32, *rows, torch.ones_like(rows[0]), causal=True))

    def sides():
        return [skl.AttnSide(x[i], x[i + 1], 0.125, rotary_q=rot, rotary_k=rot) for i in (0, 2)]

    want = [t.clone() for t in use(*sides())]
    b = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        p1, p2 = sides()
        held = {t.data_ptr() for p in (p1, p2) for t in (p.q, p.k)}
        b.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(b):
            torch.cuda._sleep(100_000_000)  # some 50 ms before they are read
            got = use(p1, p2)
        del p1, p2
        new = [torch.empty_like(x[0]).fill_(float("nan")) for _ in range(8)]
        assert not held & {t.data_ptr() for t in new}
        torch.cuda.current_stream().wait_stream(b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.gpu
def test_sides_made_before_a_capture():
    n = torch.arange(256, dtype=torch.int32, device="cuda")[None]
    x = [torch.randn((1, 4, 256, 64), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(4)]
    rot = skl.Rotary((100.0 ** (-torch.arange(32, device="cuda") / 32)).float(), n)
    p1, p2 = (skl.AttnSide(x[i], x[i + 1], 0.125, rotary_q=rot, rotary_k=rot) for i in (0, 2))
    want = skl.streamkl_fwd_mod(p1, p2, causal=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = skl.streamkl_fwd_mod(p1, p2, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    del p1, p2
    torch.cuda.synchronize()
    torch.empty_like(x[0])
