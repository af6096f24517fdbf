"""The operators of a routed-expert block next to the experts themselves: cases, inputs, plain forms.

``route``      routing by softmax or sigmoid scores with a balance bias, expert groups, renormalised and scaled weights
``norm``       the norms after and before a block in one pass with its gate and residual scale
``linear``     x w^T with bias, activation and residual in the epilogue
``*_grad``     the gradient of each

``run`` computes a case in elementary torch operations in 32 bits, or (``own``) by the calls a user makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step: group-limited sigmoid routing over 256 experts, latency alone counts
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             renorm=True, scale=2.5, dtype="f32"),
        # the same routing over a whole prefill batch
        dict(name="route prefill", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             renorm=True, scale=2.5, dtype="f32"),
        # softmax scores kept as they are (not renormalised), an expert count that is no power of two, odd token count, bf16 logits
        dict(name="route softmax odd", op="route", T=4099, E=60, k=4, score="softmax", bias=False, n_group=1, topk_group=1,
             renorm=False, scale=1.0, dtype="bf16"),
        # the router's training step: every expert's logit has a gradient
        dict(name="route grad", op="route_grad", T=8192, E=256, k=8, score="softmax", bias=True, renorm=False, scale=1.0,
             dtype="f32"),
        # one token between two blocks: post-norm, residual, pre-norm
        dict(name="norm one token", op="norm", T=1, H=7168, post=True, gate="none", scale=1.0, stream="bf16", wdtype="bf16"),
        # a prefill batch, sandwich norms with a learned gate per channel
        dict(name="norm prefill", op="norm", T=8192, H=7168, post=True, gate="channel", scale=0.5, stream="bf16", wdtype="bf16"),
        # residual stream kept in 32 bits, one gate a token, no post-norm, odd token count
        dict(name="norm wide stream", op="norm", T=4099, H=2048, post=False, gate="token", scale=1.0, stream="f32", wdtype="f32"),
        # the backward pass of the sandwich with all its reductions over tokens
        dict(name="norm grad", op="norm_grad", T=8192, H=7168, post=True, gate="channel", scale=0.5, stream="bf16", wdtype="bf16"),
        # one token through a shared expert's down projection, joined to the routed output
        dict(name="linear one token", op="linear", T=1, K=2048, N=7168, act="none", bias=False, residual=True, out="bf16", preact=False),
        # router logits of a prefill batch: narrow output in 32 bits, bound by reading the tokens
        dict(name="linear router", op="linear", T=8192, K=7168, N=256, act="none", bias=False, residual=False, out="f32", preact=False),
        # a dense projection with bias and activation at full width
        dict(name="linear prefill", op="linear", T=8192, K=7168, N=4096, act="gelu", bias=True, residual=False, out="bf16", preact=False),
        # its backward pass (three gradients) with an odd token count
        dict(name="linear grad", op="linear_grad", T=8191, K=7168, N=2048, act="silu", bias=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "norm", "norm_grad", "linear", "linear", "linear_grad"])
    if op.startswith("route"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384, 512, rng.randrange(9, 1025)])
        score = rng.choice(["softmax", "sigmoid"])
        c = dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randrange(1, min(E, 12) + 1), score=score, bias=rng.random() < 0.5,
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]), dtype=rng.choice(["f32", "f32", "bf16"]))
        if op == "route":
            fits = [(g, m) for g in (2, 4, 8) for m in range(1, g) if E % g == 0 and E // g >= 2 and m * (E // g) >= c["k"]]
            g, m = rng.choice(fits) if fits and rng.random() < 0.5 else (1, 1)
            c.update(n_group=g, topk_group=m)
        return c
    if op.startswith("norm"):
        H = rng.choice([2048, 4096, 7168, 8 * _log(rng, 16, 1024), _log(rng, 100, 8192)])
        return dict(op=op, T=_log(rng, 1, min(16384, 8192 * 7168 // H)), H=H, post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token", "element"]),
                    scale=rng.choice([1.0, 0.5, 0.125]), stream=rng.choice(["bf16", "bf16", "f32"]), wdtype=rng.choice(["bf16", "f32"]))
    T, K, N = _log(rng, 1, 8192), 8 * _log(rng, 16, 896), _log(rng, 1, 4096)
    if rng.random() < 0.5:
        N = max(8, N // 8 * 8)
    if op == "linear_grad":
        return dict(op=op, T=T, K=K, N=min(N, 2048), act=rng.choice(["none", "silu", "gelu", "relu"]), bias=rng.random() < 0.7, out="bf16")
    act = rng.choice(["none", "none", "silu", "gelu", "relu"])
    return dict(op=op, T=T, K=K, N=N, act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.4,
                out=rng.choice(["bf16", "bf16", "f32"]), preact=act != "none" and rng.random() < 0.4)


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * (c["E"] * size + 8 * c["k"]) + 4 * c["E"] * c["bias"], "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "route_grad":
        size = 4 if c["dtype"] == "f32" else 2
        dense = c["score"] == "softmax" and not c["renorm"]
        read = c["E"] * size if dense else c["k"] * size
        return {"bytes": c["T"] * (read + 12 * c["k"] + c["E"] * size), "flops": 4 * c["T"] * c["E"]}
    if c["op"].startswith("norm"):
        T, H, s = c["T"], c["H"], 4 if c["stream"] == "f32" else 2
        gate = {"none": 0, "channel": 4 * H, "token": 4 * T, "element": 2 * T * H}[c["gate"]]  # learned in 32 bits, or an activation
        w = (4 if c["wdtype"] == "f32" else 2) * H * (1 + c["post"])
        if c["op"] == "norm":
            return {"bytes": T * H * (2 * s + 4) + gate + w, "flops": 10 * T * H}
        return {"bytes": T * H * (3 * s + 6) + 2 * gate + w + 4 * H * (1 + c["post"]), "flops": 25 * T * H}
    T, K, N, o = c["T"], c["K"], c["N"], 4 if c["out"] == "f32" else 2
    if c["op"] == "linear":
        return {"bytes": 2 * (T * K + N * K) + T * N * o * (1 + c["residual"] + c["preact"]) + 2 * N * c["bias"], "flops": 2 * T * N * K}
    return {"bytes": 4 * (T * K + N * K) + 2 * T * N * (1 + (c["act"] != "none")) + 4 * N * c["bias"], "flops": 4 * T * N * K}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=c)
    if c["op"].startswith("route"):
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = (randn(T, E) * 1.5 + randn(E) * 0.5).to(DTYPES[c["dtype"]])
        # a balance bias as its update rule leaves it: many small equal steps
        s["bias"] = (randn(E) * 30).round() * 0.001 if c["bias"] else None
        if c["op"] == "route":
            s["out"] = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
        else:
            scores = _scores(s["logits"].float(), c["score"])
            choice = scores if s["bias"] is None else scores + s["bias"]
            s["idx"] = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
            w = scores.gather(1, s["idx"].long())
            s["w"] = ((w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]).contiguous()
            s["grad_w"] = randn(T, k)
            s["out"] = torch.empty_like(s["logits"])
        return s
    if c["op"].startswith("norm"):
        T, H = c["T"], c["H"]
        wd, sd = DTYPES[c["wdtype"]], DTYPES[c["stream"]]
        s["residual"] = (randn(T, H) * 2).to(sd)
        s["y"] = (randn(T, H) * (0.5 + torch.rand(T, 1, generator=g, device="cuda"))).to(torch.bfloat16)
        s["post_weight"] = (1 + 0.2 * randn(H)).to(wd) if c["post"] else None
        s["pre_weight"] = (1 + 0.2 * randn(H)).to(wd)
        s["gate"] = {"none": lambda: None, "channel": lambda: 1 + 0.3 * randn(H), "token": lambda: torch.sigmoid(randn(T)),
                     "element": lambda: torch.sigmoid(randn(T, H)).to(torch.bfloat16)}[c["gate"]]()
        if c["op"] == "norm":
            s["out"] = (torch.empty_like(s["residual"]), torch.empty_like(s["y"]))
        else:  # the stream after the block, and what comes back to it and to the next block's input
            s["grad_residual"] = randn(T, H).to(sd)
            s["grad_normed"] = randn(T, H).to(torch.bfloat16)
        return s
    T, K, N = c["T"], c["K"], c["N"]
    s["x"] = randn(T, K).to(torch.bfloat16)
    s["w"] = (randn(N, K) / math.sqrt(K)).to(torch.bfloat16)
    s["b"] = (randn(N) * 0.2).to(torch.bfloat16) if c["bias"] else None
    if c["op"] == "linear":
        s["residual"] = randn(T, N).to(DTYPES[c["out"]]) if c["residual"] else None
        s["out"] = torch.empty(T, N, dtype=DTYPES[c["out"]], device="cuda")
    else:
        s["preact"] = None
        if c["act"] != "none":
            z = s["x"] @ s["w"].t()
            s["preact"] = z if s["b"] is None else z + s["b"]
        s["grad_y"] = randn(T, N).to(DTYPES[c["out"]])
    return s


def run(state):
    return (_own if own else _plain)(state)


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import mixture_experts_routed_top_gb300 as moe

    c = s["case"]
    op = c["op"]
    if op == "route":
        return moe.route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_group=c["n_group"],
                                topk_group=c["topk_group"], renormalise=c["renorm"], scale=c["scale"], out=s["out"])
    if op == "route_grad":
        return moe.route_scored_backward(s["logits"], s["idx"], s["w"], s["grad_w"], score=c["score"], bias=s["bias"],
                                         renormalise=c["renorm"], scale=c["scale"], out=s["out"])
    if op == "norm":
        return moe.block_norm(s["residual"], s["y"], gate=s["gate"], scale=c["scale"], post_norm=c["post"],
                              post_weight=s["post_weight"], pre_weight=s["pre_weight"], eps=1e-6, out=s["out"])
    if op == "norm_grad":
        return moe.block_norm_backward(s["grad_residual"], s["grad_normed"], s["residual"], s["y"], gate=s["gate"], scale=c["scale"],
                                       post_norm=c["post"], post_weight=s["post_weight"], pre_weight=s["pre_weight"], eps=1e-6)
    act = None if c["act"] == "none" else c["act"]
    if op == "linear":
        return moe.linear(s["x"], s["w"], bias=s["b"], activation=act, residual=s["residual"], preact=c["preact"], out=s["out"])
    return moe.linear_backward(s["grad_y"], s["x"], s["w"], bias=s["b"], activation=act, preact=s["preact"])


# ------------------------------------------------------------------ plain forms
def _tree_sum(v):
    """Sum over the last axis by halves: the fixed order in which the softmax's normaliser is defined."""
    n = 1 << (v.shape[1] - 1).bit_length()
    if n > v.shape[1]:
        v = torch.cat([v, v.new_zeros(v.shape[0], n - v.shape[1])], 1)
    while n > 1:
        n //= 2
        v = v[:, :n] + v[:, n:]
    return v


def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.max(1, keepdim=True)[0])
    return e / _tree_sum(e)


def _plain_route(s):
    c = s["case"]
    scores = _scores(s["logits"].float(), c["score"])
    choice = scores if s["bias"] is None else scores + s["bias"]
    T, E = scores.shape
    if c["n_group"] > 1:
        groups = choice.view(T, c["n_group"], E // c["n_group"])
        best = torch.sort(groups, dim=2, descending=True)[0][:, :, :2].sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True)[1][:, : c["topk_group"]]
        kept = torch.zeros(T, c["n_group"], dtype=torch.bool, device="cuda").scatter_(1, keep, True)
        choice = torch.where(kept.unsqueeze(2), groups, -math.inf).view(T, E)
    idx = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, : c["k"]]
    w = scores.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), w * c["scale"]


def _plain_route_grad(s):
    c = s["case"]
    idx, g = s["idx"].long(), s["grad_w"] * c["scale"]
    p = _scores(s["logits"].float(), c["score"])
    ps = p.gather(1, idx)
    if c["renorm"]:
        total = ps.sum(1, keepdim=True)
        g = (g - (g * ps).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_(1, idx, g)
    if c["score"] == "sigmoid":
        return (ds * p * (1 - p)).to(s["logits"].dtype)
    return (p * (ds - (g * ps).sum(1, keepdim=True))).to(s["logits"].dtype)


def _rstd(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)


def _gate_of(s):
    g = s["gate"]
    return 1.0 if g is None else g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _plain_norm(s):
    c = s["case"]
    z = s["y"].float()
    if c["post"]:
        z = z * _rstd(z) * s["post_weight"].float()
    r = s["residual"].float() + c["scale"] * _gate_of(s) * z
    n = r * _rstd(r) * s["pre_weight"].float()
    return r.to(s["residual"].dtype), n.to(s["y"].dtype)


def _plain_norm_grad(s):
    c = s["case"]
    r, y, dn = s["residual"].float(), s["y"].float(), s["grad_normed"].float()
    rs = _rstd(r)
    q = dn * s["pre_weight"].float() * rs
    d = s["grad_residual"].float() + q - r * rs * rs * (q * r).mean(1, keepdim=True)
    d_pre = (dn * r * rs).sum(0)
    dz = c["scale"] * _gate_of(s) * d
    d_post, ys = None, y
    dy = dz
    if c["post"]:
        ry = _rstd(y)
        ys = y * ry * s["post_weight"].float()
        q = dz * s["post_weight"].float() * ry
        dy = q - y * ry * ry * (q * y).mean(1, keepdim=True)
        d_post = (dz * y * ry).sum(0)
    dg = None
    if c["gate"] == "channel":
        dg = (c["scale"] * ys * d).sum(0)
    elif c["gate"] == "token":
        dg = (c["scale"] * ys * d).sum(1)
    elif c["gate"] == "element":
        dg = (c["scale"] * ys * d).to(s["gate"].dtype)
    return d.to(s["residual"].dtype), dy.to(s["y"].dtype), dg, d_post, d_pre


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.where(z > 0, z, 0.0) if act == "relu" else z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return (z > 0).to(z.dtype)


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        y = y + s["b"].float()
    z, dt = y, DTYPES[s["case"]["out"]]
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(dt), z.to(dt)) if s["case"]["preact"] else y.to(dt)


def _plain_linear_grad(s):
    dz = s["grad_y"].float()
    if s["preact"] is not None:
        dz = dz * _act_slope(s["preact"].float(), s["case"]["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    db = None if s["b"] is None else dz.sum(0)
    return dx.to(s["x"].dtype), dw.to(s["w"].dtype), db


_FORMS = {"route": _plain_route, "route_grad": _plain_route_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
          "linear": _plain_linear, "linear_grad": _plain_linear_grad}


def _plain(s):
    return _FORMS[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    return globals()["_exact_" + c["op"]](c, {k: v for k, v in s.items() if k != "out"})


def _exact_scores(x, score):
    return torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)


def _exact_route(c, s):
    # which experts are taken is decided by the 32-bit scores (part of the definition); their weights are in 64 bits
    idx = _plain_route(s)[0].long()
    w = _exact_scores(s["logits"].double(), c["score"]).gather(1, idx)
    if c["renorm"]:
        w = torch.nn.functional.normalize(w, p=1, dim=1)
    return None, w * c["scale"]


def _exact_route_grad(c, s):
    x = s["logits"].double().requires_grad_()
    w = _exact_scores(x, c["score"]).gather(1, s["idx"].long())
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((w * c["scale"] * s["grad_w"].double()).sum(), x)[0]


def _exact_block(c, r, y, gate, w_post):
    if c["post"]:
        y = y / (y.square().mean(1, keepdim=True) + 1e-6).sqrt() * w_post
    if gate is not None:
        y = y * (gate[:, None] if c["gate"] == "token" else gate)
    return r + c["scale"] * y


def _exact_rows(c):
    return c["T"] * c["H"] <= 1 << 26


def _exact_norm(c, s):
    if not _exact_rows(c):
        return None
    v = {k: None if s[k] is None else s[k].double() for k in ("residual", "y", "gate", "post_weight", "pre_weight")}
    r = _exact_block(c, v["residual"], v["y"], v["gate"], v["post_weight"])
    return r, r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * v["pre_weight"]


def _exact_norm_grad(c, s):
    if not _exact_rows(c):
        return None
    v = {k: None if s[k] is None else s[k].double().requires_grad_() for k in ("residual", "y", "gate", "post_weight", "pre_weight")}
    # the pre-norm's own gradient at the stream given, then the block's at a residual that leads there
    out, w = v["residual"], v["pre_weight"]
    n = out / (out.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
    d, d_pre = torch.autograd.grad(n, (out, w), s["grad_normed"].double())
    d = d + s["grad_residual"].double()
    block = _exact_block(c, torch.zeros_like(d), v["y"], v["gate"], v["post_weight"])
    names = [k for k in ("y", "gate", "post_weight") if v[k] is not None]
    got = dict(zip(names, torch.autograd.grad(block, [v[k] for k in names], d)))
    return d, got["y"], got.get("gate"), got.get("post_weight"), d_pre


def _exact_act(z, act):
    f = torch.nn.functional
    return z if act == "none" else {"silu": f.silu, "gelu": f.gelu, "relu": f.relu}[act](z)


def _exact_linear(c, s):
    z = s["x"].double().mm(s["w"].double().t())
    if s["b"] is not None:
        z = z + s["b"].double()
    y = _exact_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, z) if c["preact"] else y


def _exact_linear_grad(c, s):
    dz = s["grad_y"].double()
    if s["preact"] is not None:
        z = s["preact"].double().requires_grad_()
        dz = torch.autograd.grad(_exact_act(z, c["act"]), z, dz)[0]
    return dz.mm(s["w"].double()), dz.t().mm(s["x"].double()), None if s["b"] is None else dz.sum(0)
