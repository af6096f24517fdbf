"""Workspaces and tensors of the calls under graphs and on several streams."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_top_gb300 as m
    m.lib()
    return m


def _randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("default", [True, False])
def test_a_graph_keeps_its_workspace_when_a_larger_call_follows(moe, default, monkeypatch):
    """Captured, then a call that needs more, then other tensors in whatever memory is free,
    then replays: the results are the same and nobody else's memory has changed."""
    monkeypatch.setattr(moe, "_DEFAULT_WS", {})
    ws = None if default else moe.Workspace("cuda")
    x, w = _randn(64, 4096, seed=1), _randn(256, 4096, seed=2)
    gy = _randn(64, 256, seed=3)

    def step():
        y = moe.linear(x, w, workspace=ws)                       # the contraction is split: partial sums
        return y, *moe.linear_backward(gy, x, w, bias=x[0, :256], workspace=ws)

    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    used = (moe.default_workspace() if default else ws).buffers()
    big = torch.full((4096, 8192), 2.0, dtype=torch.bfloat16, device="cuda")     # 67 MB of dz
    moe.linear_backward(big, _randn(4096, 64, seed=4), _randn(8192, 64, seed=5), activation="silu", preact=big,
                        workspace=ws)
    torch.cuda.synchronize()
    after = moe.default_workspace() if default else ws
    assert after.buf.numel() > 67 * 2 ** 20 and all(any(b is c for c in after.buffers()) for b in after.captured)
    assert any(b is c for b in used for c in after.captured)
    others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [b.numel() for b in used] * 2 + [1 << 20] * 8]
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((o == 7).all()) for o in others)
    moe.workspace_status(after)


def test_an_error_is_reported_after_the_workspace_has_grown(moe):
    """An expert index out of range, then a call that needs a larger buffer, then the status."""
    ws = moe.Workspace("cuda")
    h = _randn(16, 128, seed=6)
    idx = torch.full((16, 1), 9, dtype=torch.int32, device="cuda")
    wgu, wd = _randn(4, 256, 128, seed=7), _randn(4, 128, 128, seed=8)
    moe.experts_forward(h, idx, torch.ones(16, 1, device="cuda"), wgu, wd, workspace=ws)
    before = ws.buf.numel()
    moe.linear(_randn(64, 64, seed=9), _randn(64, 64, seed=10), workspace=ws)
    assert ws.buf.numel() > before
    with pytest.raises(moe.MoEError) as e:
        moe.workspace_status(ws)
    assert e.value.status == 1
    moe.workspace_status(ws)


def test_streams_do_not_share_the_default_workspace(moe):
    """Split products and gradients on two streams at once give what they give one by one."""
    cases = [(_randn(64, 4096, seed=20 + i), _randn(256, 4096, seed=30 + i), _randn(64, 256, seed=40 + i))
             for i in range(2)]

    def step(x, w, gy):
        return moe.linear(x, w), *moe.linear_backward(gy, x, w, bias=w[:, 0].contiguous())

    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = []
    for s in streams:
        with torch.cuda.stream(s):
            spaces.append(moe.default_workspace())
    assert spaces[0] is not spaces[1] and moe.default_workspace() not in spaces
    got = [[], []]
    for _ in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    for ws in spaces:
        moe.workspace_status(ws)


MS = 2_000_000          # about a millisecond of the SM's clock


def _calls(moe):
    """Each call that takes stream=, small; -> [(name, call(stream) -> tensors)]"""
    x, w = _randn(64, 4096, seed=50), _randn(256, 4096, seed=51)
    gy, y = _randn(64, 256, seed=52), _randn(64, 4096, seed=53)
    logits = _randn(64, 256, seed=54, dtype=torch.float32)
    idx, p = moe.route_scored(logits, 4)
    gp = _randn(64, 4, seed=55, dtype=torch.float32)
    wgu, wd = _randn(4, 256, 4096, seed=56), _randn(4, 4096, 128, seed=57)
    few = (idx[:, :1] % 4).contiguous()     # one slot a token: the combine's order is not fixed
    return [
        ("linear", lambda s: (moe.linear(x, w, stream=s),)),
        ("linear preact", lambda s: moe.linear(x, w, activation="silu", preact=True, stream=s)),
        ("linear_backward", lambda s: moe.linear_backward(gy, x, w, bias=gy[0], stream=s)),
        ("block_norm", lambda s: moe.block_norm(x, y, post_norm=True, stream=s)),
        ("block_norm_backward", lambda s: moe.block_norm_backward(x, y, x, y, post_norm=True, pre_weight=w[0], stream=s)),
        ("route_scored", lambda s: moe.route_scored(logits, 4, stream=s)),
        ("route_scored_backward", lambda s: (moe.route_scored_backward(logits, idx, p, gp, stream=s),)),
        ("route", lambda s: moe.route(logits, 4, stream=s)),
        ("dispatch", lambda s: moe.dispatch(few, 4, stream=s)),
        ("experts_forward", lambda s: (moe.experts_forward(x, few, p[:, :1].contiguous(), wgu, wd, stream=s),)),
        ("quantize_fp8_blocks", lambda s: moe.quantize_fp8_blocks(w, stream=s)),
        ("quantize_fp4_blocks", lambda s: moe.quantize_fp4_blocks(w, stream=s)),
    ]


def _same(got, want):
    return all((a is None) == (b is None) and (a is None or torch.equal(a, b)) for a, b in zip(got, want))


def test_results_on_a_stream_do_not_take_memory_that_the_current_stream_still_writes(moe, monkeypatch):
    """The current stream is late: blocks that it has let go of are still to be written by it,
    and a new workspace's zeros would come after the kernel's partial sums."""
    side = torch.cuda.Stream()
    for name, call in _calls(moe):
        want = [None if t is None else t.clone() for t in call(None)]
        torch.cuda.synchronize()
        monkeypatch.setattr(moe, "_DEFAULT_WS", {})
        torch.cuda._sleep(20 * MS)
        for t in want:       # same sizes as the results, written late and free at once
            if t is not None:
                torch.empty_like(t).view(torch.uint8).fill_(99)
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert _same(got, want), name
        moe.workspace_status()


def test_results_on_a_stream_that_are_let_go_are_not_written_into_others(moe):
    """The side stream is late and its results are dropped at once: tensors that the current
    stream makes meanwhile keep their values."""
    side = torch.cuda.Stream()
    for name, call in _calls(moe):
        if name == "dispatch":
            continue            # it waits for its own status
        sizes = [t.numel() * t.element_size() for t in call(None) if t is not None]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20 * MS)
        call(side)
        kept = [torch.full((n,), 99, dtype=torch.uint8, device="cuda") for n in sizes * 3]
        torch.cuda.synchronize()
        assert all(bool((k == 99).all()) for k in kept), name


def test_arguments_on_a_stream_may_be_let_go(moe):
    side = torch.cuda.Stream()
    w = _randn(256, 4096, seed=61)
    x = _randn(64, 4096, seed=60)
    want = moe.linear(x, w)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20 * MS)
    x2 = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.linear(x2, w, stream=side)
    del x2
    junk = [torch.full((64, 4096), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


def test_results_on_a_stream_read_late_by_the_current_one(moe):
    """The current stream reads a result after the caller has let it go and the side stream goes on."""
    side = torch.cuda.Stream()
    x, w = _randn(64, 4096, seed=62), _randn(256, 4096, seed=63)
    want, minus = moe.linear(x, w), -x
    torch.cuda.synchronize()
    y = moe.linear(x, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20 * MS)
    copy = y.clone()
    del y
    later = [moe.linear(minus, w, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and all(torch.equal(t, -want) for t in later)


def test_a_workspace_used_on_another_stream_than_its_own(moe):
    """In order, as a shared workspace has to be; it is let go while the other stream still works on it."""
    x, w = _randn(64, 4096, seed=64), _randn(256, 4096, seed=65)
    ws = moe.Workspace("cuda")
    want = moe.linear(x, w, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20 * MS)
    got = moe.linear(x, w, workspace=ws, stream=side)
    n = ws.buf.numel()
    del ws
    kept = [torch.full((n,), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((k == 99).all()) for k in kept)


def test_the_status_of_every_default_workspace(moe, monkeypatch):
    monkeypatch.setattr(moe, "_DEFAULT_WS", {})
    side = torch.cuda.Stream()
    h, wgu, wd = _randn(16, 128, seed=6), _randn(4, 256, 128, seed=7), _randn(4, 128, 128, seed=8)
    idx, one = torch.full((16, 1), 9, dtype=torch.int32, device="cuda"), torch.ones(16, 1, device="cuda")
    moe.experts_forward(h, idx - 9, one, wgu, wd)
    torch.cuda.synchronize()
    moe.experts_forward(h, idx, one, wgu, wd, stream=side)
    moe.workspace_status(moe.default_workspace())
    with pytest.raises(moe.MoEError):
        moe.workspace_status()
    moe.workspace_status()
    moe.workspace_status(moe.default_workspace(stream=side))
