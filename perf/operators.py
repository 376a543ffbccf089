"""The operators of a layer in training and serving: norm, linear products, 8-bit checkpoints.

A layer of the models whose weights the optimizer steps (hidden 2048 / 4096 /
5120, mlp 5504 / 11008 / 13824), on T tokens:

  norm         h = x + r, y = rms_norm(h) w, optionally y also held in 8 bits
  norm_grad    its gradient, with the gradient that reaches h past the norm
  pack         an activation held in 8 bits (e4m3, one power-of-two scale for
               32 columns of a row) and the values that this stands for
  linear       y = act(x W^T + b) + r, and z = x W^T + b for the backward pass
  act_grad     dz = dy act'(z) and the bias gradient
  linear_grad  dx = dz W and dW = dz^T x
  weight_grad  M <- M + dz^T x with x from its 8-bit checkpoint: the weight
               gradient summed into the optimizer's momentum

``own`` chooses between the plain form (elementary torch operations in 32
bits, each output rounded once) and this package's operators.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BLOCK = 32          # columns that share one scale

# multiplications of the largest listed case; drawn cases stay below it
MOST_WORK = 8192 * 11008 * 4096


def listed():
    return [
        # one token's norm in serving: latency
        {"name": "norm-1x4096", "op": "norm", "T": 1, "m": 4096, "dtype": "bf16", "pack": False},
        # a training batch's norm that also leaves the 8-bit checkpoint
        {"name": "norm-8192x4096-f8", "op": "norm", "T": 8192, "m": 4096, "dtype": "bf16",
         "pack": True},
        # the backward pass of that norm
        {"name": "norm_grad-8192x4096", "op": "norm_grad", "T": 8192, "m": 4096, "dtype": "bf16"},
        # the mlp's inner activation of a training batch, checkpointed
        {"name": "pack-8192x11008", "op": "pack", "T": 8192, "m": 11008, "dtype": "bf16"},
        # one token through the mlp's first product in serving: reads the weights once
        {"name": "linear-1x11008x4096", "op": "linear", "T": 1, "n": 11008, "m": 4096,
         "dtype": "bf16", "act": "silu", "bias": True, "residual": False, "preact": False},
        # a ragged prefill through the 1B mlp's second product, onto the residual stream
        {"name": "linear-1000x2048x5504", "op": "linear", "T": 1000, "n": 2048, "m": 5504,
         "dtype": "fp16", "act": "none", "bias": True, "residual": True, "preact": False},
        # a training batch through the 7B mlp's first product
        {"name": "linear-8192x11008x4096", "op": "linear", "T": 8192, "n": 11008, "m": 4096,
         "dtype": "bf16", "act": "gelu_tanh", "bias": True, "residual": False, "preact": True},
        # the activation's gradient of that product
        {"name": "act_grad-8192x11008", "op": "act_grad", "T": 8192, "n": 11008, "dtype": "bf16",
         "act": "gelu_tanh"},
        # both products of the backward pass of an attention projection
        {"name": "linear_grad-8192x4096x4096", "op": "linear_grad", "T": 8192, "n": 4096,
         "m": 4096, "dtype": "bf16"},
        # a short odd sequence through the backward pass of a layer of odd size
        {"name": "linear_grad-517x1000x515", "op": "linear_grad", "T": 517, "n": 1000, "m": 515,
         "dtype": "fp16"},
        # weight gradient of a small matrix from a long batch's checkpoint, into the momentum
        {"name": "weight_grad-16384x128x512", "op": "weight_grad", "T": 16384, "n": 128, "m": 512,
         "dtype": "bf16"},
        # weight gradient of the 1B mlp from a training batch's checkpoint, into the momentum
        {"name": "weight_grad-8192x5504x2048", "op": "weight_grad", "T": 8192, "n": 5504,
         "m": 2048, "dtype": "bf16"},
    ]


def draw(rng):
    """Another case of the same ranges: 1 to 16384 tokens, sides 100 to 13824, odd ones too."""
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        kind = rng.random()
        if kind < 0.4 and v >= 256:          # most sides of real layers
            v = v // 128 * 128
        elif kind < 0.7 and v >= 16:
            v = v // 8 * 8
        return max(lo, v)

    op = rng.choice(["norm", "norm_grad", "pack", "linear", "linear", "act_grad", "linear_grad",
                     "weight_grad"])
    case = {"op": op, "T": size(1, 16384), "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op in ("norm", "norm_grad", "pack"):
        case["m"] = size(100, 13824)
        if op == "norm":
            case["pack"] = rng.random() < 0.5
        return case
    case["n"] = size(100, 13824)
    if op == "act_grad":
        case["act"] = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        return case
    case["m"] = size(100, 13824)
    while case["T"] * case["n"] * case["m"] * (2 if op == "linear_grad" else 1) > MOST_WORK:
        case["T"] = case["T"] * 3 // 4
    if op == "linear":
        case["act"] = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        case["bias"] = rng.random() < 0.5
        case["residual"] = rng.random() < 0.5
        case["preact"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------- inputs

def _rand(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _activation(g, T, m, dtype):
    """Activations: N(0, 1) with a few columns far larger, as a residual stream has them."""
    gain = torch.ones(m, device="cuda")
    gain[torch.randint(0, m, (max(1, m // 256),), generator=g, device="cuda")] = 12.0
    x = torch.randn((T, m), generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DTYPES[case["dtype"]]
    op, T, m, n = case["op"], case["T"], case.get("m", 0), case.get("n", 0)
    s = {"case": case}
    if op == "norm":
        s["x"], s["r"] = _rand(g, (T, m), 0.5, t), _activation(g, T, m, t)
        s["w"] = 1.0 + _rand(g, (m,), 0.1, torch.float32)
    elif op == "norm_grad":
        s["h"] = _activation(g, T, m, t)
        s["dy"], s["dh"] = _rand(g, (T, m), 0.02, t), _rand(g, (T, m), 0.02, t)
        s["w"] = 1.0 + _rand(g, (m,), 0.1, torch.float32)
        # kept by the forward pass
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
    elif op == "pack":
        s["x"] = _activation(g, T, m, t)
    elif op == "linear":
        s["x"] = _activation(g, T, m, t)
        s["W"] = _rand(g, (n, m), 0.02, t)
        s["b"] = _rand(g, (n,), 0.1, torch.float32) if case["bias"] else None
        s["r"] = _activation(g, T, n, t) if case["residual"] else None
    elif op == "act_grad":
        s["z"], s["dy"] = _rand(g, (T, n), 1.5, t), _rand(g, (T, n), 0.02, t)
    else:
        s["dz"] = _rand(g, (T, n), 0.02, t)
        x = _activation(g, T, m, t)
        if op == "linear_grad":
            s["x"], s["W"] = x, _rand(g, (n, m), 0.02, t)
        else:                # the 8-bit checkpoint that the forward pass left, and the momentum
            s["q"], s["scale"] = _quantize(x)
            s["M"] = _rand(g, (n, m), 1.0, torch.float32)
    return s


# --------------------------------------------------------- the 8-bit format

def _pow2(e):
    """2^e in fp32 from the exponent's bits, exactly (-149 <= e <= 127)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).float()


def _quantize(x):
    """(q, scale): rows padded with zeros to whole blocks of 32 columns, q in
    e4m3, scale one byte e + 127 a block.  2^e is the smallest power of two
    that keeps the block's largest magnitude at or below 448."""
    T, m = x.shape
    mp = -(-m // BLOCK) * BLOCK
    v = torch.zeros((T, mp), device=x.device, dtype=torch.float32)
    v[:, :m] = x
    v = v.view(T, mp // BLOCK, BLOCK)
    mant, ex = torch.frexp(v.abs().amax(2))             # amax = mant 2^ex, 0.5 <= mant < 1
    e = ex - 9 + (mant > 0.875).to(ex.dtype)            # 448 = 0.875 2^9
    e = torch.where(mant == 0, torch.full_like(e, -127), e).clamp_min(-127)
    # the largest block of a type must not round up to past its largest value
    last = 8 if x.dtype == torch.float16 else 120
    most = torch.where(e == last, 240.0, 448.0).unsqueeze(2)
    u = v * _pow2(-e).unsqueeze(2)
    q = torch.minimum(torch.maximum(u, -most), most).to(torch.float8_e4m3fn)
    return q.view(T, mp), (e + 127).to(torch.uint8)


def _values(q, scale, m):
    """The fp32 values that (q, scale) stand for."""
    T, mp = q.shape
    v = q.float().view(T, mp // BLOCK, BLOCK)
    return (v * _pow2(scale.to(torch.int32) - 127).unsqueeze(2)).view(T, mp)[:, :m]


# ----------------------------------------------------------- the plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    op, t = case["op"], DTYPES[case["dtype"]]
    if op == "norm":
        h = (s["x"].float() + s["r"].float()).to(t)
        hf = h.float()
        rstd = 1 / torch.sqrt(hf.square().mean(1) + EPS)
        y = (hf * rstd.unsqueeze(1) * s["w"]).to(t)
        out = {"h": h, "y": y, "rstd": rstd}
        if case["pack"]:
            out["y8"] = _values(*_quantize(y), case["m"]).to(t)
        return out
    if op == "norm_grad":
        hat = s["h"].float() * s["rstd"].unsqueeze(1)
        dy = s["dy"].float()
        a = dy * s["w"]
        dx = s["rstd"].unsqueeze(1) * (a - hat * (a * hat).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(t), "dw": (dy * hat).sum(0)}
    if op == "pack":
        return _values(*_quantize(s["x"]), case["m"]).to(t)
    if op == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(t), "z": z.to(t)} if case["preact"] else {"y": y.to(t)}
    if op == "act_grad":
        d = s["dy"].float() * _act_slope(s["z"].float(), case["act"])
        return {"dz": d.to(t), "db": d.sum(0)}
    if op == "linear_grad":
        dz = s["dz"].float()
        return {"dx": (dz @ s["W"].float()).to(t), "dW": dz.t() @ s["x"].float()}
    s["M"] += s["dz"].float().t() @ _values(s["q"], s["scale"], case["m"])
    return s["M"]


# ------------------------------------------------------ the package's calls

def _own(s):
    import orthogonalizing_optimizer_amd as d3
    case = s["case"]
    op, t = case["op"], DTYPES[case["dtype"]]
    if op == "norm":
        y, h, rstd, packed = d3.add_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS,
                                             pack=case["pack"])
        out = {"h": h, "y": y, "rstd": rstd}
        if case["pack"]:
            out["y8"] = d3.unpack_f8(packed, t)
        return out
    if op == "norm_grad":
        dx, dw = d3.add_rms_norm_grad(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "pack":
        return d3.unpack_f8(d3.pack_f8(s["x"]), t)
    if op == "linear":
        y, z = d3.linear(s["x"], s["W"], bias=s["b"], act=case["act"], residual=s["r"],
                         return_preact=case["preact"])
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    if op == "act_grad":
        dz, db = d3.act_grad(s["dy"], s["z"], case["act"], bias=True)
        return {"dz": dz, "db": db}
    if op == "linear_grad":
        return {"dx": d3.linear_grad_input(s["dz"], s["W"]),
                "dW": d3.linear_grad_weight(s["dz"], s["x"])}
    return d3.linear_grad_weight(s["dz"], d3.PackedF8(s["q"], s["scale"], case["m"]), out=s["M"],
                                 accumulate=True)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the value in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, from the inputs' own values."""
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "norm":
        h = s["x"].to(f) + s["r"].to(f)
        stream = h.to(DTYPES[case["dtype"]]).to(f)   # the stream that goes on is the rounded one
        rstd = 1 / torch.sqrt(torch.sum(stream * stream, 1) / case["m"] + EPS)
        out = {"h": h, "y": stream * rstd[:, None] * s["w"].to(f), "rstd": rstd}
        if case["pack"]:
            # which of two 8-bit neighbours a value at a border takes hangs on
            # the rounding of y before it: no value of its own
            out["y8"] = None
        return out
    if op == "norm_grad":
        h, dy, w, r = s["h"].to(f), s["dy"].to(f), s["w"].to(f), s["rstd"].to(f)[:, None]
        inner = torch.sum(dy * w * h, 1, keepdim=True) / case["m"]
        return {"dx": r * dy * w - r ** 3 * h * inner + s["dh"].to(f),
                "dw": torch.sum(dy * h * r, 0)}
    if op == "pack":
        x = s["x"].to(f)
        T, m = x.shape
        pad = (-m) % BLOCK
        v = torch.cat([x, x.new_zeros((T, pad))], 1).reshape(T, -1, BLOCK)
        top = torch.amax(torch.abs(v), 2, keepdim=True)
        power = torch.tensor([2.0 ** k for k in range(-160, 161)], device=x.device, dtype=f)

        def two(k):                                                  # exactly 2^k
            return power[k.long() + 160]
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448))
        e = torch.where(two(e - 1) * 448 >= top, e - 1, e)          # log2 next to a whole number
        e = torch.where(two(e) * 448 < top, e + 1, e)
        u = v / two(e)
        # e4m3: 3 bits after the leading one, down to steps of 2^-9
        lead = torch.floor(torch.log2(torch.clamp(torch.abs(u), min=2.0 ** -9)))
        lead = torch.where(two(lead) > torch.abs(u), lead - 1, lead)
        lead = torch.where(two(lead + 1) <= torch.abs(u), lead + 1, lead)
        step = two(torch.clamp(lead, min=-6.0) - 3)
        u = torch.round(u / step) * step                             # ties to even
        return (u * two(e)).reshape(T, -1)[:, :m]
    if op == "linear":
        z = torch.matmul(s["x"].to(f), s["W"].to(f).T.contiguous())
        if case["bias"]:
            z = z + s["b"].to(f)
        act = case["act"]
        if act == "relu":
            y = torch.maximum(z, torch.zeros_like(z))
        elif act == "gelu":
            y = z * (1 + torch.special.erf(z / 2 ** 0.5)) / 2
        elif act == "gelu_tanh":
            y = z / 2 * (1 + torch.tanh((2 / math.pi) ** 0.5 * z * (1 + 0.044715 * z ** 2)))
        elif act == "silu":
            y = z * torch.special.expit(z)
        else:
            y = z
        if case["residual"]:
            y = y + s["r"].to(f)
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    if op == "act_grad":
        z = s["z"].to(f).requires_grad_(True)
        act = case["act"]
        with torch.enable_grad():
            y = {"relu": torch.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
                 "none": lambda v: v * 1}[act](z)
            d, = torch.autograd.grad(y, z, s["dy"].to(f))
        return {"dz": d, "db": torch.sum(d, 0)}
    dz = s["dz"].to(f)
    if op == "linear_grad":
        return {"dx": torch.matmul(dz, s["W"].to(f)),
                "dW": torch.matmul(dz.T.contiguous(), s["x"].to(f))}
    T, mp = s["q"].shape
    power = torch.tensor([2.0 ** k for k in range(-127, 129)], device=dz.device, dtype=f)
    two = power[s["scale"].long()]
    x = (s["q"].to(f).reshape(T, mp // BLOCK, BLOCK) * two[:, :, None]).reshape(T, mp)
    return s["M"].to(f) + torch.matmul(dz.T.contiguous(), x[:, :case["m"]].contiguous())


# ---------------------------------------------------------- the work of a pass

def work(case):
    op, T, m, n = case["op"], case["T"], case.get("m", 0), case.get("n", 0)
    f8 = 1 + 1 / BLOCK
    if op == "norm":      # x, r in, h, y (and y in 8 bits and its values) out
        return {"bytes": T * m * (8 + (f8 + 2 if case["pack"] else 0)) + 4 * (m + T),
                "flops": 6 * T * m}
    if op == "norm_grad":
        return {"bytes": 8 * T * m + 8 * m + 4 * T, "flops": 11 * T * m}
    if op == "pack":      # in, 8 bits out, their values out
        return {"bytes": T * m * (2 + f8 + 2), "flops": 3 * T * m}
    if op == "linear":
        outs = 1 + case["preact"] + case["residual"]
        return {"bytes": 2 * (T * m + n * m + outs * T * n) + 4 * n * case["bias"],
                "flops": 2 * T * n * m}
    if op == "act_grad":
        return {"bytes": 6 * T * n + 4 * n, "flops": 12 * T * n}
    if op == "linear_grad":
        return {"bytes": 2 * (T * n + T * m + n * m + T * m) + 4 * n * m, "flops": 4 * T * n * m}
    return {"bytes": 2 * T * n + f8 * T * m + 8 * n * m, "flops": 2 * T * n * m}
