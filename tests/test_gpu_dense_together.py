"""The operators of the dense half of a block together, as a model uses them: a training step
and a serving pass, in graphs, on other streams and with shared workspaces."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_routed_top_gb300 as m
    m.lib()
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _randn(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _near(got, ref, roundings):
    """Norm-wise: each bf16 rounding on the way is at most 2^-8 of what it rounds; fp32 is far below."""
    assert np.linalg.norm(_np(got) - ref) <= roundings * BF * np.linalg.norm(ref)


def _train(moe, p, r, y, grad, stream=None, ws=None):
    """norm -> gated feed-forward -> residual, and its gradients from dL/d(out)."""
    kw = dict(stream=stream)
    kww = dict(stream=stream, workspace=ws)
    s, n = moe.layer_norm(r, y, weight=p["nw"], bias=p["nb"], **kw)
    h, z = moe.gated_linear(n, p["wgu"], bias=p["bgu"], activation="gelu", preact=True, **kww)
    out = moe.linear(h, p["wd"], residual=s, **kww)
    dh, dwd, _ = moe.linear_backward(grad, h, p["wd"], **kww)
    dn, dwgu, dbgu = moe.gated_linear_backward(dh, n, p["wgu"], z, bias=p["bgu"], activation="gelu", **kww)
    dr, dy, dnw, dnb = moe.layer_norm_backward(grad, dn, s, weight=p["nw"], bias=p["nb"], need_y=True, **kww)
    return dict(out=out, dwd=dwd, dwgu=dwgu, dbgu=dbgu, dr=dr, dy=dy, dnw=dnw, dnb=dnb)


def _params(H, I, seed=1):
    return dict(nw=1 + _randn(H, seed=seed, dtype=torch.float32, scale=0.1), nb=_randn(H, seed=seed + 1, dtype=torch.float32, scale=0.1),
                wgu=_randn(2 * I, H, seed=seed + 2, scale=H ** -0.5), bgu=_randn(2 * I, seed=seed + 3, dtype=torch.float32, scale=0.1),
                wd=_randn(H, I, seed=seed + 4, scale=I ** -0.5))


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (7, 136, 72), (33, 264, 40), (300, 512, 384), (2100, 256, 776)])
def test_a_training_step(moe, T, H, I):
    """Every gradient against a 64-bit autograd of the whole block.  On the longest way (the stream's
    gradient) the sum, n, h, the result's gradient through dh, dz, dn and dr are rounded: 8 of 2^-8."""
    p = _params(H, I)
    r, y, grad = _randn(T, H, seed=11, scale=2.0), _randn(T, H, seed=12), _randn(T, H, seed=13)
    got = _train(moe, p, r, y, grad)
    v = {k: t.double().requires_grad_() for k, t in dict(p, r=r, y=y).items()}
    s = v["r"] + v["y"]
    n = torch.nn.functional.layer_norm(s, (H,), v["nw"], v["nb"], 1e-5)
    zg, zu = (n @ v["wgu"].t() + v["bgu"]).chunk(2, 1)
    out = s + (torch.nn.functional.gelu(zg) * zu) @ v["wd"].t()
    d = dict(zip(v, torch.autograd.grad(out, list(v.values()), grad.double())))
    _near(got["out"], out.detach().cpu().numpy(), 4)
    for name, key in (("dwd", "wd"), ("dwgu", "wgu"), ("dbgu", "bgu"), ("dr", "r"), ("dy", "y"), ("dnw", "nw"), ("dnb", "nb")):
        _near(got[name], d[key].cpu().numpy(), 8)
    moe.workspace_status(moe.default_workspace())


@pytest.mark.parametrize("T", [1, 9, 40, 600])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_a_serving_pass_in_8_bits(moe, T, fmt):
    """norm, its codes once for both projections, and the projection back onto the stream: each step
    against the oracle on what the step before it gave."""
    H, N = 256, 320
    r = _randn(T, H, seed=21, scale=2.0)
    w = [O.quantize_blocks(_np(_randn(384, H, seed=22 + i, scale=H ** -0.5)).astype(np.float32), 128, 128, fmt) for i in range(2)]
    w1 = [(torch.from_numpy(c[:N].copy()).cuda(), torch.from_numpy(s).cuda(), c[:N], sv) for c, s, sv in w]
    wb = O.quantize_blocks(_np(_randn(H, 384, seed=25, scale=384 ** -0.5)).astype(np.float32), 128, 128, fmt)
    _, n = moe.layer_norm(r)
    q, s = moe.quantize_fp8_rows(n, fmt)
    codes, stored, values = O.quantize_blocks(_np(n).astype(np.float32), 1, 128, fmt)
    assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), stored)
    acts = ("silu", None)
    a, b = (moe.linear_fp8(q, c, sc, x_scale=s, activation=act) for (c, sc, _, _), act in zip(w1, acts))
    for t, (_, _, c, sv), act in zip((a, b), w1, acts):
        ref, _, mag = B.linear_fp8(codes, values, c, sv, activation=act)
        err = np.abs(_np(t) - ref)
        assert (err <= BF * np.abs(ref) + 2.0 ** -16 * mag).all()
    h = torch.zeros(T, 384, dtype=torch.bfloat16, device="cuda")
    h[:, :N] = a * b
    y = moe.linear_fp8(h, torch.from_numpy(wb[0]).cuda(), torch.from_numpy(wb[1]).cuda(), residual=r)
    hc, _, hv = O.quantize_blocks(_np(h).astype(np.float32), 1, 128, fmt)
    ref, _, mag = B.linear_fp8(hc, hv, wb[0], wb[2], residual=_np(r))
    assert (np.abs(_np(y) - ref) <= BF * np.abs(ref) + 2.0 ** -16 * (mag + np.abs(_np(r)))).all()


def _serve(moe, x, w, ws, big, stream=None, workspace=None):
    y = moe.linear_fp8(x, w, ws, stream=stream, workspace=workspace)
    return y, moe.gated_linear(x, big, stream=stream, workspace=workspace)


@pytest.mark.parametrize("T", [3, 40, 2060])
def test_in_a_graph(moe, T):
    """Captured and replayed on new contents of the same tensors: what eager calls give on them."""
    H, I = 512, 768
    p = _params(H, I)
    r, y, grad = _randn(T, H, seed=31), _randn(T, H, seed=32), _randn(T, H, seed=33)
    w = torch.randint(0, 120, (2 * I, H), dtype=torch.uint8, device="cuda")
    ws = torch.rand(2 * I // 128, H // 128, device="cuda")

    def step():
        t = _train(moe, p, r, y, grad)
        return [*t.values(), *_serve(moe, r, w, ws, p["wgu"]), *moe.quantize_fp8_rows(y, "ue8m0")]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (41, 51):
        for i, t in enumerate((r, y, grad)):
            t.copy_(_randn(T, H, seed=seed + i))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    moe.workspace_status(moe.default_workspace())


def test_on_two_streams_at_once(moe):
    """Calls on two streams, by stream= and by the current one, give what they give one by one."""
    H, I, T = 1024, 512, 40          # split contractions: partial sums in the workspaces
    p = _params(H, I)
    sets = [[_randn(T, H, seed=60 + 10 * i + j) for j in range(3)] for i in range(2)]
    w = torch.randint(0, 120, (2 * I, H), dtype=torch.uint8, device="cuda")
    ws = torch.rand(2 * I // 128, H // 128, device="cuda")
    want = [[*_train(moe, p, *s).values(), *_serve(moe, s[0], w, ws, p["wgu"])] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = [[*_train(moe, p, *s, stream=st).values(), *_serve(moe, s[0], w, ws, p["wgu"], stream=st)]
               for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    mine = [moe.Workspace("cuda") for _ in sets]
    for _ in range(5):
        got = []
        for s, st, k in zip(sets, streams, mine):
            with torch.cuda.stream(st):
                got.append([*_train(moe, p, *s, ws=k).values(), *_serve(moe, s[0], w, ws, p["wgu"], workspace=k)])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_do_not_depend_on_the_call(moe):
    """The same bits from call to call, and rows of a batch behind which nothing is written."""
    T, H, I = 2050, 512, 768
    p = _params(H, I)
    r, y, grad = _randn(T, H, seed=71), _randn(T, H, seed=72), _randn(T, H, seed=73)
    w = torch.randint(0, 120, (1700, H), dtype=torch.uint8, device="cuda")
    ws = torch.rand(14, H // 128, device="cuda")
    a = [*_train(moe, p, r, y, grad).values(), moe.linear_fp8(r, w, ws)]
    for _ in range(3):
        b = [*_train(moe, p, r, y, grad).values(), moe.linear_fp8(r, w, ws)]
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    for call, N in ((lambda o: moe.gated_linear(r, p["wgu"], out=o), I), (lambda o: moe.linear_fp8(r, w, ws, out=o), 1700)):
        for dt in (torch.bfloat16, torch.float32):
            if N == I and dt == torch.float32:
                continue
            room = torch.full((T + 300, N + 24), 7.0, dtype=dt, device="cuda")
            call(room[:T, :N])
            assert (room[T:] == 7).all() and (room[:, N:] == 7).all()
