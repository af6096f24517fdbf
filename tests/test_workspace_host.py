"""The workspace's bookkeeping, without a GPU: its buffers are host tensors here and the
state of the stream is the test's."""
import weakref

import pytest
import torch

import mixture_experts_routed_top_gb300 as moe


@pytest.fixture
def stream(monkeypatch):
    """Whether the current stream is being captured, as the test sets it."""
    state = dict(capturing=False)
    monkeypatch.setattr(moe, "_capturing", lambda: state["capturing"], raising=False)
    monkeypatch.setattr(moe, "_stream", lambda stream=None: 7)
    return state


def test_a_captured_buffer_outlives_growth(stream):
    """A graph keeps the address it was captured with: a larger call gets another
    buffer, and the graph's is not given back."""
    ws = moe.Workspace("cpu")
    first = ws.get(2000)
    assert ws.get(100) is first
    stream["capturing"] = True
    assert ws.get(1500) is first              # the graph's from now on
    stream["capturing"] = False
    assert ws.get(1500) is first
    first = weakref.ref(first)                # nobody but the workspace holds it
    large = ws.get(50000)
    assert first() is not None and large is not first() and ws.buf is large
    assert any(b is first() for b in ws.buffers()) and any(b is large for b in ws.buffers())
    stream["capturing"] = True
    assert ws.get(40000) is large             # another graph, a larger call
    stream["capturing"] = False
    ws.get(90000)
    assert {b.numel() for b in ws.buffers()} == {2000, 50000, 90000}


def test_a_buffer_that_was_not_captured_is_given_back(stream):
    ws = moe.Workspace("cpu")
    for n in (2000, 4000, 8000):
        ws.get(n)
    assert [b.numel() for b in ws.buffers()] == [8000]


def test_a_buffer_allocated_in_a_capture_stays_the_graphs(stream):
    ws = moe.Workspace("cpu")
    own = ws.get(1024)
    stream["capturing"] = True
    g = ws.get(5000)
    assert g is not own and ws.get(4000) is g
    stream["capturing"] = False
    assert ws.get(1000) is own and ws.get(4000) is not g
    assert any(b is g for b in ws.buffers())


def test_buffers_start_zeroed(stream):
    ws = moe.Workspace("cpu")
    assert ws.buffers() == [] and ws.buf is None
    assert ws.get(1).numel() >= 1024 and not ws.get(1).any()


def test_errors_survive_growth(stream):
    """The error word of a buffer that is given back moves on; the counters behind it start
    at zero; a captured buffer keeps its own."""
    ws = moe.Workspace("cpu")
    ws.get(1024)[:12].view(torch.int32).copy_(torch.tensor([5, 3, 1]))
    assert ws.get(4096)[:12].view(torch.int32).tolist() == [5, 0, 0]
    stream["capturing"] = True
    kept = ws.get(100)
    stream["capturing"] = False
    assert not ws.get(9000).any()
    assert kept[:4].view(torch.int32).item() == 5 and any(b is kept for b in ws.buffers())


def test_default_workspaces_per_stream(stream, monkeypatch):
    """Each device and stream has its own; a capturing stream without one shares the device's
    first, so that nothing is allocated in the capture."""
    now = {}
    monkeypatch.setattr(moe, "_DEFAULT_WS", {})
    monkeypatch.setattr(moe, "_raw_stream", lambda dev: now["handle"])
    made = {}
    for dev, handle in ((0, 0), (0, 11), (1, 0)):     # handle 0: the default stream
        now["handle"] = handle
        made[dev, handle] = moe._default_ws(dev)
        assert moe._default_ws(dev) is made[dev, handle]
    assert len({id(w) for w in made.values()}) == 3
    stream["capturing"] = True
    now["handle"] = 99
    assert moe._default_ws(0) is made[0, 0] and moe._default_ws(1) is made[1, 0]
    now["handle"] = 11
    assert moe._default_ws(0) is made[0, 11]
    stream["capturing"] = False
    now["handle"] = 99
    assert moe._default_ws(0) not in made.values()


def test_calls_on_a_stream(monkeypatch):
    """stream= makes it the current one for the whole call, and both streams are recorded."""
    log = []

    class Stream:
        device = torch.device("cuda", 0)

        def __init__(self, name):
            self.name = name

    class Under:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            log.append(("enter", self.s.name))

        def __exit__(self, *exc):
            log.append(("leave", self.s.name))

    class Fake(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 0)

        def record_stream(self, s):
            log.append((self.label, s.name))

    def tensor(label):
        t = torch.zeros(2).as_subclass(Fake)
        t.label = label
        return t

    main, side = Stream("main"), Stream("side")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: main)
    monkeypatch.setattr(torch.cuda, "stream", Under)
    result = (tensor("y"), None)

    def call(x, k, *, out=None, bias=None):
        log.append(("call", k))
        return result

    args = dict(x=tensor("x"), k=3, out=(tensor("o"), None), bias=None, stream=side)
    assert moe._on_stream(call, args) is result
    assert log == [("enter", "side"), ("call", 3), ("leave", "side"), ("x", "side"), ("o", "side"), ("y", "main")]
    log.clear()
    moe._on_stream(call, dict(x=tensor("x"), k=4, stream=main))         # the current one: nothing to record
    assert log == [("enter", "main"), ("call", 4), ("leave", "main")]
    other = Stream("other")
    other.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        moe._on_stream(call, dict(x=tensor("x"), k=4, stream=other))
