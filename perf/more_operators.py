"""The dense half of a routed-expert block: cases, inputs, plain forms.

``gated``       both projections of a gated feed-forward, activation and product: act(x wg^T + bg) (x wu^T + bu)
``fp8``         x w^T of e4m3 codes with a scale per 1 x 128 of x and per 128 x 128 of w, bias, activation, residual
``ln``          residual sum and layer norm in one pass
``*_grad``      the gradients of ``gated`` and ``ln``

``run`` computes a case in elementary torch operations in 32 bits, or (``own``) by the calls a user makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step through a shared expert's gate and up projections: the weights' bytes count
        dict(name="gated one token", op="gated", T=1, K=7168, I=2048, act="silu", bias=False, preact=False),
        # the shared expert over a prefill batch
        dict(name="gated prefill", op="gated", T=8192, K=7168, I=2048, act="silu", bias=False, preact=False),
        # a training step's forward pass, which keeps both pre-activations: biases, gelu, an odd token count
        dict(name="gated training", op="gated", T=4099, K=2048, I=1408, act="gelu", bias=True, preact=True),
        # the backward pass of a training step: input's, weights' and biases' gradients
        dict(name="gated grad", op="gated_grad", T=8191, K=7168, I=2048, act="silu", bias=True),
        # the same for a small batch of a small model
        dict(name="gated grad small", op="gated_grad", T=257, K=2048, I=1024, act="relu", bias=False),
        # one token through an 8-bit output projection that joins the residual stream; power-of-two scales
        dict(name="fp8 one token", op="fp8", T=1, K=2048, N=7168, fmt="ue8m0", codes=False, act="none", bias=False,
             residual=True, out="bf16"),
        # a prefill batch through an 8-bit projection with 32-bit scales; activations quantised within the call
        dict(name="fp8 prefill", op="fp8", T=8192, K=7168, N=4096, fmt="f32", codes=False, act="none", bias=False,
             residual=False, out="bf16"),
        # codes that another projection of the same input has made already, a width that ends inside a scale block
        dict(name="fp8 codes odd", op="fp8", T=4099, K=7168, N=2112, fmt="ue8m0", codes=True, act="gelu", bias=True,
             residual=False, out="f32"),
        # a decode batch between two blocks, with the residual sum
        dict(name="layer norm few tokens", op="ln", T=8, H=7168, add=True, stream="bf16", wdtype="bf16", bias=True),
        # a prefill batch
        dict(name="layer norm prefill", op="ln", T=8192, H=7168, add=True, stream="bf16", wdtype="bf16", bias=True),
        # a training step's backward pass with the weight's and bias' sums over tokens
        dict(name="layer norm grad", op="ln_grad", T=8192, H=7168, add=True, stream="bf16", wdtype="bf16", bias=True),
        # a stream kept in 32 bits, a width and a token count that are no multiples of anything
        dict(name="layer norm grad odd", op="ln_grad", T=4099, H=2050, add=True, stream="f32", wdtype="f32", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "fp8", "fp8", "ln", "ln_grad"])
    if op.startswith("gated"):
        I = _log(rng, 1, 2048)
        if rng.random() < 0.6:
            I = max(8, I // 8 * 8)
        c = dict(op=op, T=_log(rng, 1, 8191), K=8 * _log(rng, 16, 896), I=I, act=rng.choice(["silu", "silu", "gelu", "relu"]),
                 bias=rng.random() < 0.4)
        if op == "gated":
            c["preact"] = rng.random() < 0.5
        return c
    if op == "fp8":
        N = _log(rng, 1, 4096)
        if rng.random() < 0.5:
            N = max(64, N // 64 * 64)
        return dict(op=op, T=_log(rng, 1, 8192), K=128 * _log(rng, 1, 56), N=N, fmt=rng.choice(["f32", "ue8m0"]),
                    codes=rng.random() < 0.4, act=rng.choice(["none", "none", "silu", "gelu", "relu"]),
                    bias=rng.random() < 0.4, residual=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "f32"]))
    H = rng.choice([2048, 4096, 7168, 8 * _log(rng, 16, 1024), _log(rng, 100, 8192)])
    stream = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, T=_log(rng, 1, min(16384, (8192 if stream == "bf16" else 3584) * 7168 // H)), H=H, add=rng.random() < 0.6,
                stream=stream, wdtype=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.7)


def work(case):
    c = case
    if c["op"].startswith("gated"):
        T, K, I = c["T"], c["K"], c["I"]
        if c["op"] == "gated":
            return {"bytes": 2 * (T * K + 2 * I * K) + 2 * T * I * (3 if c["preact"] else 1) + 4 * I * c["bias"],
                    "flops": 4 * T * I * K}
        return {"bytes": 4 * (T * K + 2 * I * K) + 6 * T * I + 8 * I * c["bias"], "flops": 8 * T * I * K}
    if c["op"] == "fp8":
        T, K, N, o, s = c["T"], c["K"], c["N"], 4 if c["out"] == "f32" else 2, 4 if c["fmt"] == "f32" else 1
        x = T * (K + K // 128 * s) if c["codes"] else 2 * T * K
        return {"bytes": x + N * K + (N + 127) // 128 * (K // 128) * s + T * N * o * (1 + c["residual"]) + 2 * N * c["bias"],
                "flops": 2 * T * N * K}
    T, H, s, w = c["T"], c["H"], 4 if c["stream"] == "f32" else 2, 4 if c["wdtype"] == "f32" else 2
    if c["op"] == "ln":
        return {"bytes": T * H * (s + 2 + (s + 2) * c["add"]) + w * H * (1 + c["bias"]), "flops": 8 * T * H}
    # the stream, its gradient and the norm's in, the stream's gradient out (the block's too where it is another type)
    return {"bytes": T * H * (2 * s + 2 + s * c["add"] + 2 * (c["add"] and s == 4)) + w * H + 4 * H * (1 + c["bias"]),
            "flops": 16 * T * H}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=c)
    if c["op"].startswith("gated"):
        T, K, I = c["T"], c["K"], c["I"]
        s["x"] = randn(T, K).to(torch.bfloat16)
        s["w"] = (randn(2 * I, K) / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (randn(2 * I) * 0.2).to(torch.bfloat16) if c["bias"] else None
        if c["op"] == "gated":
            s["out"] = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
        else:
            z = s["x"] @ s["w"].t()
            s["preact"] = z if s["b"] is None else z + s["b"]
            s["grad_h"] = randn(T, I).to(torch.bfloat16)
        return s
    if c["op"] == "fp8":
        T, K, N = c["T"], c["K"], c["N"]
        # activations of tokens of different size, with a few channels that stand out
        x = (randn(T, K) * (0.5 + torch.rand(T, 1, generator=g, device="cuda"))
             * (1 + 7 * (torch.rand(K, generator=g, device="cuda") < 0.01))).to(torch.bfloat16)
        pad = -N % 128
        w = torch.cat([randn(N, K) / math.sqrt(K), torch.zeros(pad, K, device="cuda")])
        blocks = w.view((N + pad) // 128, 128, K // 128, 128)
        scale, s["w_scale"] = _scale(blocks.abs().amax((1, 3)), c["fmt"])
        s["w"] = _codes(blocks * (1 / scale)[:, None, :, None]).view(N + pad, K)[:N].contiguous()
        s["x"], s["x_scale"] = _quantise(x, c["fmt"]) if c["codes"] else (x, None)
        s["b"] = (randn(N) * 0.2).to(torch.bfloat16) if c["bias"] else None
        s["residual"] = randn(T, N).to(DTYPES[c["out"]]) if c["residual"] else None
        s["out"] = torch.empty(T, N, dtype=DTYPES[c["out"]], device="cuda")
        return s
    T, H, wd, sd = c["T"], c["H"], DTYPES[c["wdtype"]], DTYPES[c["stream"]]
    # a stream with a mean of its own in each token, as biases leave it
    s["residual"] = (randn(T, H) * 2 + randn(T, 1)).to(sd)
    s["y"] = randn(T, H).to(torch.bfloat16) if c["add"] else None
    s["weight"] = (1 + 0.2 * randn(H)).to(wd)
    s["b"] = (0.2 * randn(H)).to(wd) if c["bias"] else None
    if c["op"] == "ln":
        s["out"] = (torch.empty_like(s["residual"]) if c["add"] else None, torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
    else:
        s["grad_residual"] = randn(T, H).to(sd) if c["add"] else None
        s["grad_normed"] = randn(T, H).to(torch.bfloat16)
    return s


def run(state):
    return (_own if own else _plain)(state)


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import mixture_experts_routed_top_gb300 as moe

    c = s["case"]
    op = c["op"]
    if op == "gated":
        return moe.gated_linear(s["x"], s["w"], bias=s["b"], activation=c["act"], preact=c["preact"], out=s["out"])
    if op == "gated_grad":
        return moe.gated_linear_backward(s["grad_h"], s["x"], s["w"], s["preact"], bias=s["b"], activation=c["act"])
    if op == "fp8":
        return moe.linear_fp8(s["x"], s["w"], s["w_scale"], x_scale=s["x_scale"], bias=s["b"],
                              activation=None if c["act"] == "none" else c["act"], residual=s["residual"], out=s["out"])
    if op == "ln":
        return moe.layer_norm(s["residual"], s["y"], weight=s["weight"], bias=s["b"], eps=1e-5, out=s["out"])
    return moe.layer_norm_backward(s["grad_residual"], s["grad_normed"], s["residual"], weight=s["weight"], bias=s["b"],
                                   eps=1e-5, need_y=c["add"])


# ------------------------------------------------------------------ plain forms
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


def _plain_gated(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    gate, up = z[:, : c["I"]], z[:, c["I"]:]
    h = (_act(gate, c["act"]) * up).to(torch.bfloat16)
    return (h, z.to(torch.bfloat16)) if c["preact"] else h


def _plain_gated_grad(s):
    c = s["case"]
    z, dh = s["preact"].float(), s["grad_h"].float()
    gate, up = z[:, : c["I"]], z[:, c["I"]:]
    dz = torch.cat([dh * up * _act_slope(gate, c["act"]), dh * _act(gate, c["act"])], 1)
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    return dx.to(torch.bfloat16), dw.to(torch.bfloat16), None if s["b"] is None else dz.sum(0)


def _scale(amax, fmt):
    """amax / 448 in 32 bits, or the least power of two that is no smaller; as a number and as it is stored."""
    # by a tensor: a division by a number would become a product with its rounded reciprocal
    q = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448.0))
    if fmt == "f32":
        return q, q
    bits = q.view(torch.int32)
    e = ((bits >> 23) + ((bits & 0x7FFFFF) != 0)).clamp(1, 254)
    return (e << 23).view(torch.float32), e.to(torch.uint8)


def _codes(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _quantise(x, fmt):
    """-> e4m3 codes of x and the scales of its 1 x 128 blocks, as stored."""
    blocks = x.float().view(x.shape[0], -1, 128)
    scale, stored = _scale(blocks.abs().amax(2), fmt)
    return _codes(blocks * (1 / scale)[:, :, None]).view(x.shape), stored


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _scale_values(stored):
    return stored if stored.dtype == torch.float32 else (stored.to(torch.int32) << 23).view(torch.float32)


def _plain_fp8(s):
    c = s["case"]
    T, K, N = c["T"], c["K"], c["N"]
    codes, stored = (s["x"], s["x_scale"]) if c["codes"] else _quantise(s["x"], c["fmt"])
    x = (_values(codes).view(T, K // 128, 128) * _scale_values(stored)[:, :, None]).view(T, K)
    per_row = _scale_values(s["w_scale"])[torch.arange(N, device="cuda") // 128]
    w = (_values(s["w"]).view(N, K // 128, 128) * per_row[:, :, None]).view(N, K)
    y = x @ w.t()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _plain_ln(s):
    r = s["residual"].float()
    if s["y"] is not None:
        r = r + s["y"].float()
    d = r - r.mean(1, keepdim=True)
    n = d * torch.rsqrt((d * d).mean(1, keepdim=True) + 1e-5) * s["weight"].float()
    if s["b"] is not None:
        n = n + s["b"].float()
    return r.to(s["residual"].dtype), n.to(torch.bfloat16)


def _plain_ln_grad(s):
    r, dn = s["residual"].float(), s["grad_normed"].float()
    d = r - r.mean(1, keepdim=True)
    rs = torch.rsqrt((d * d).mean(1, keepdim=True) + 1e-5)
    n = d * rs
    q = dn * s["weight"].float()
    dr = rs * (q - q.mean(1, keepdim=True) - n * (q * n).mean(1, keepdim=True))
    if s["grad_residual"] is not None:
        dr = dr + s["grad_residual"].float()
    db = None if s["b"] is None else dn.sum(0)
    dy = dr.to(torch.bfloat16) if s["case"]["add"] else None
    return dr.to(s["residual"].dtype), dy, (dn * n).sum(0), db


_FORMS = {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "fp8": _plain_fp8, "ln": _plain_ln, "ln_grad": _plain_ln_grad}


def _plain(s):
    return _FORMS[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))


def _exact_act(z, act):
    f = torch.nn.functional
    return z if act == "none" else {"silu": f.silu, "gelu": f.gelu, "relu": f.relu}[act](z)


def _exact_halves(z, act):
    gate, up = z.tensor_split(2, 1)
    return _exact_act(gate, act).mul(up)


def _exact_gated(c, s):
    z = s["x"].double().mm(s["w"].double().t())
    if c["bias"]:
        z += s["b"].double()
    h = _exact_halves(z, c["act"])
    return (h, z) if c["preact"] else h


def _exact_gated_grad(c, s):
    z = s["preact"].double().requires_grad_()
    dz = torch.autograd.grad(_exact_halves(z, c["act"]), z, s["grad_h"].double())[0]
    return dz.mm(s["w"].double()), dz.t().mm(s["x"].double()), dz.sum(0) if c["bias"] else None


def _round_e4m3(v):
    """The nearest value of four exponent and three mantissa bits, ties to even (of 64-bit numbers of at most 448)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_fp8(c, s):
    T, K, N = c["T"], c["K"], c["N"]
    if c["codes"]:
        x = s["x"].view(torch.float8_e4m3fn).double().view(T, -1, 128)
        sx = s["x_scale"].double() if c["fmt"] == "f32" else torch.exp2(s["x_scale"].double() - 127)
    else:
        # the codes are part of the definition: each step rounds to 32 bits once
        x = s["x"].double().view(T, -1, 128)
        amax = x.abs().amax(2)
        sx = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, 448)).float().double()
        if c["fmt"] == "ue8m0":
            m, e = torch.frexp(sx)
            sx = torch.exp2((e - (m == 0.5).to(e.dtype)).double())
        inv = (1 / sx).float().double()
        x = _round_e4m3((x * inv[..., None]).float().double().clamp(-448, 448))
    sw = s["w_scale"].double() if c["fmt"] == "f32" else torch.exp2(s["w_scale"].double() - 127)
    w = s["w"].view(torch.float8_e4m3fn).double().view(N, -1, 128) * sw.repeat_interleave(128, 0)[:N, :, None]
    z = (x * sx[..., None]).view(T, K).mm(w.view(N, K).t())
    if c["bias"]:
        z += s["b"].double()
    y = _exact_act(z, c["act"])
    return y + s["residual"].double() if c["residual"] else y


def _exact_rows(c):
    return c["T"] * c["H"] <= 1 << 26


def _exact_norm(r, w, b):
    var, mean = torch.var_mean(r, 1, correction=0, keepdim=True)
    n = (r - mean) / (var + 1e-5).sqrt() * w
    return n if b is None else n + b


def _exact_ln(c, s):
    if not _exact_rows(c):
        return None
    r = s["residual"].double()
    if c["add"]:
        r = r + s["y"].double()
    return r, _exact_norm(r, s["weight"].double(), s["b"].double() if c["bias"] else None)


def _exact_ln_grad(c, s):
    if not _exact_rows(c):
        return None
    r, w = s["residual"].double().requires_grad_(), s["weight"].double().requires_grad_()
    dr, dw = torch.autograd.grad(_exact_norm(r, w, None), (r, w), s["grad_normed"].double())
    if c["add"]:
        dr = dr + s["grad_residual"].double()
    return dr, dr if c["add"] else None, dw, s["grad_normed"].double().sum(0) if c["bias"] else None
