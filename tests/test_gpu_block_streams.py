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
