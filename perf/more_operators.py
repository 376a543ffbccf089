"""The operators of a training step around the layers: both ends of a model, heads, clipping.

  embed        y = s W[tokens]: a model's first step
  embed_grad   its gradient, dW[v] = s sum of dy over the tokens v, in fp32
  heads        queries and keys normed per head and rotated by their positions
  heads_grad   its gradient, the norms' weights too
  logp         log probabilities of given tokens, with entropy and the best alternatives
  logp_grad    the gradient of the log probabilities (and the entropies) in the logits
  clip         the global norm of many gradients, and the clipped gradients in place
               or summed into the optimizer's momenta

Sizes are those of the layers whose weights the optimizer steps (hidden 2048 /
4096 / 5120 in heads of 128, mlp 5504) with vocabularies of the usual sizes.

``own`` chooses between the plain form (elementary torch operations in 32
bits, each output rounded once) and this package's operators.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6

# elements of the largest listed case of each kind; drawn cases stay below
MOST = {"embed": 8192 * 4096, "embed_grad": 32000 * 4096, "heads": 8192 * 40 * 128,
        "heads_grad": 8192 * 40 * 128, "logp": 8192 * 32000, "logp_grad": 8192 * 32000,
        "clip": 1 << 28}


def listed():
    return [
        # a training batch's tokens, fp32 weights to 16-bit activations
        {"name": "embed-8192x4096", "op": "embed", "T": 8192, "n": 32000, "m": 4096,
         "wtype": "fp32", "dtype": "bf16", "scale": 1.0},
        # the gradient of that: few rows have many tokens, most have none
        {"name": "embed_grad-8192x32000x4096", "op": "embed_grad", "T": 8192, "n": 32000,
         "m": 4096, "dtype": "bf16", "scale": 1.0, "sum": False},
        # a short odd sequence, summed into the gradient that a tied head left
        {"name": "embed_grad-517x50257x515", "op": "embed_grad", "T": 517, "n": 50257, "m": 515,
         "dtype": "fp16", "scale": 22.5, "sum": True},
        # one token in serving: latency
        {"name": "heads-1x32+8x128", "op": "heads", "T": 1, "hq": 32, "hk": 8, "D": 128, "r": 128,
         "dtype": "bf16", "interleaved": False, "far": 100000},
        # a training batch
        {"name": "heads-8192x32+8x128", "op": "heads", "T": 8192, "hq": 32, "hk": 8, "D": 128,
         "r": 128, "dtype": "bf16", "interleaved": False, "far": 0},
        # its backward pass
        {"name": "heads_grad-8192x32+8x128", "op": "heads_grad", "T": 8192, "hq": 32, "hk": 8,
         "D": 128, "r": 128, "dtype": "bf16", "interleaved": False, "far": 0},
        # four sequences' next tokens in serving, with the 20 best alternatives
        {"name": "logp-4x131072-top20", "op": "logp", "T": 4, "n": 131072, "dtype": "bf16",
         "scale": 1.25, "entropy": True, "top": 20, "masked": 0},
        # a scored text of odd length over an odd vocabulary, fp32 logits, 5 alternatives
        {"name": "logp-1000x50257-top5", "op": "logp", "T": 1000, "n": 50257, "dtype": "fp32",
         "scale": 1.0, "entropy": True, "top": 5, "masked": 0},
        # a training batch's loss
        {"name": "logp-8192x32000", "op": "logp", "T": 8192, "n": 32000, "dtype": "bf16",
         "scale": 1.0, "entropy": False, "top": 0, "masked": 0},
        # its gradient, with a bonus for the entropy
        {"name": "logp_grad-8192x32000", "op": "logp_grad", "T": 8192, "n": 32000, "dtype": "bf16",
         "scale": 1.0, "entropy": True, "masked": 0},
        # the gradients of one small layer, in place: latency
        {"name": "clip-9-small", "op": "clip", "shapes": "128x512,512x128,512,128,515", "count": 9,
         "dtype": "fp32", "into": False, "ratio": 0.5, "scale": 1.0},
        # 16-bit gradients of 6 layers of the 1B set, clipped and summed into the momenta
        {"name": "clip-42-layers-into", "op": "clip",
         "shapes": "2048x2048,2048x2048,2048x2048,2048x2048,5504x2048,5504x2048,2048x5504",
         "count": 42, "dtype": "bf16", "into": True, "ratio": 0.5, "scale": 1.0},
    ]


def draw(rng):
    """Another case of the same ranges, odd sizes among them."""
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        kind = rng.random()
        if kind < 0.4 and v >= 256:
            v = v // 128 * 128
        elif kind < 0.7 and v >= 16:
            v = v // 8 * 8
        return max(lo, v)

    op = rng.choice(["embed", "embed_grad", "heads", "heads_grad", "logp", "logp", "logp_grad",
                     "clip"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "clip":
        case["dtype"] = rng.choice(["fp32", "bf16", "fp16"])
        case["into"] = rng.random() < 0.5
        case["ratio"] = rng.choice([0.5, 2.0])
        case["scale"] = rng.choice([1.0, 2.0 ** -10]) if case["into"] else 1.0
        shapes, count = [], rng.randint(1, 40)
        for _ in range(rng.randint(1, 6)):
            a = size(64, 5504)
            shapes.append(str(a) if rng.random() < 0.3 else "%dx%d" % (a, size(64, 5504)))
        case["shapes"] = ",".join(shapes)
        while count > 1 and _elements(shapes, count) > MOST[op]:
            count -= 1
        case["count"] = count
        return case
    case["T"] = size(1, 8192)
    if op in ("embed", "embed_grad"):
        case["n"], case["m"] = size(1000, 131072), size(64, 5120)
        case["scale"] = rng.choice([1.0, math.sqrt(case["m"])])
        while case["T"] * case["m"] > MOST["embed"]:
            case["T"] = case["T"] * 3 // 4
        while case["n"] * case["m"] > MOST["embed_grad"]:
            case["n"] = case["n"] * 3 // 4
        if op == "embed":
            case["wtype"] = rng.choice(["fp32", case["dtype"]])
        else:
            case["sum"] = rng.random() < 0.5
        return case
    if op in ("heads", "heads_grad"):
        case["hk"] = rng.choice([1, 2, 4, 8, 16])
        case["hq"] = case["hk"] * rng.choice([1, 2, 4, 5])
        case["D"] = rng.choice([64, 80, 96, 128, 128, 192, 256])
        case["r"] = rng.choice([case["D"], case["D"], case["D"] // 2, 20])
        case["interleaved"] = rng.random() < 0.4
        case["far"] = rng.choice([0, 0, 4000, 1000000])
        while case["T"] * (case["hq"] + case["hk"]) * case["D"] > MOST[op]:
            case["T"] = case["T"] * 3 // 4
        return case
    case["n"] = size(1000, 131072)
    case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case["scale"] = rng.choice([1.0, 1.0, 0.7, 2.0])
    case["entropy"] = rng.random() < 0.5
    case["masked"] = rng.choice([0, 0, 1, 57])       # a padded vocabulary's last columns
    if op == "logp":
        case["top"] = rng.choice([0, 1, 5, 20])
    while case["T"] * case["n"] > MOST[op] // (4 if case.get("top") else 1):
        case["T"] = case["T"] * 3 // 4
    return case


def _shapes(texts, count):
    """The first ``count`` of the shapes in turn."""
    return [tuple(int(v) for v in texts[i % len(texts)].split("x")) for i in range(count)]


def _elements(texts, count):
    return sum(math.prod(s) for s in _shapes(texts, count))


# ------------------------------------------------------------------- inputs

def _rand(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _tokens(g, T, n):
    """Tokens as a text has them: the r-th most frequent of n one in r, in a shuffled order."""
    p = 1.0 / torch.arange(3, n + 3, device="cuda", dtype=torch.float32)
    rank = torch.multinomial(p, T, replacement=True, generator=g)
    return torch.randperm(n, generator=g, device="cuda")[rank]


def _logits(g, T, n, dtype, masked):
    """Logits of a trained model: a broad floor and a few likely tokens a row."""
    x = torch.randn((T, n), generator=g, device="cuda", dtype=torch.float32).mul_(2.0)
    at = torch.randint(0, n, (T, 8), generator=g, device="cuda")
    x.scatter_add_(1, at, 4 + 6 * torch.rand((T, 8), generator=g, device="cuda"))
    if masked:
        x[:, n - masked:] = -math.inf
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, t = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "clip":
        # one flat buffer, the gradients views of it, as training programs keep them
        shapes = _shapes(case["shapes"].split(","), case["count"])
        total = sum(math.prod(v) for v in shapes)
        s["flat"] = torch.empty(total, device="cuda", dtype=t)
        s["sums"] = torch.empty(total, device="cuda") if case["into"] else None
        s["grads"], s["into"], at = [], [] if case["into"] else None, 0
        for shape in shapes:
            n = math.prod(shape)
            s["flat"][at:at + n] = _rand(g, (n,), 0.02 / case["scale"], t)
            s["grads"].append(s["flat"][at:at + n].view(shape))
            if case["into"]:
                s["sums"][at:at + n].normal_(generator=g)
                s["into"].append(s["sums"][at:at + n].view(shape))
            at += n
        s["max_norm"] = case["ratio"] * 0.02 * math.sqrt(total)
        return s
    T = case["T"]
    if op in ("embed", "embed_grad"):
        n, m = case["n"], case["m"]
        s["tokens"] = _tokens(g, T, n)
        if op == "embed":
            s["W"] = _rand(g, (n, m), 0.02, DTYPES[case["wtype"]])
        else:
            s["dy"] = _rand(g, (T, m), 0.02, t)
            s["dW"] = _rand(g, (n, m), 0.02, torch.float32) if case["sum"] else None
    elif op in ("heads", "heads_grad"):
        hq, hk, D, r = case["hq"], case["hk"], case["D"], case["r"]
        # queries, keys and values of one product
        x = _rand(g, (T, (hq + 2 * hk) * D), 1.0, t)
        s["q"] = x[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = x[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
        s["wq"], s["wk"] = 1 + _rand(g, (D,), 0.1, torch.float32), 1 + _rand(g, (D,), 0.1, torch.float32)
        # sequences of up to 4096 tokens, one behind the other
        s["pos"] = case["far"] + torch.arange(T, device="cuda") % 4096
        s["freqs"] = 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        if op == "heads_grad":
            s["dq"], s["dk"] = _rand(g, (T, hq, D), 0.02, t), _rand(g, (T, hk, D), 0.02, t)
    else:
        n = case["n"]
        s["x"] = _logits(g, T, n, t, case["masked"])
        s["targets"] = torch.randint(0, n - case["masked"], (T,), generator=g, device="cuda")
        if op == "logp_grad":
            s["g"] = -torch.rand(T, generator=g, device="cuda") / T
            s["gh"] = (-0.01 / T) * torch.rand(T, generator=g, device="cuda") if case["entropy"] else None
            # what the forward pass left: the maximum, the log of the sum, the entropy
            m, e = [], []
            for part in s["x"].split(max(1, (1 << 27) // n)):
                z = part.double() * case["scale"]
                top = z.amax(1)
                d = z - top[:, None]
                l = torch.logsumexp(d, 1)
                p = torch.exp(d - l[:, None])
                m.append(torch.stack([top, l], 1))
                e.append(l - torch.where(p > 0, p * d, 0.0).sum(1))
            s["stats"], s["H"] = torch.cat(m).float(), torch.cat(e).float()
    return s


# ----------------------------------------------------------- the plain forms

def _turn(x, cos, sin, interleaved):
    """x [T, H, D], its first 2 len(cos) columns turned by the angles of cos, sin [T, 1, r / 2]."""
    h = cos.shape[-1]
    y = x.clone()
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    u, v = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = u, v
    else:
        y[..., :h], y[..., h:2 * h] = u, v
    return y


def _angles(s):
    a = s["pos"].double()[:, None, None] * s["freqs"]      # far positions: in 64 bits
    return torch.cos(a).float(), torch.sin(a).float()


def _plain(s):
    case = s["case"]
    op, t = case["op"], DTYPES[case["dtype"]]
    if op == "embed":
        return (s["W"][s["tokens"]].float() * case["scale"]).to(t)
    if op == "embed_grad":
        d = torch.zeros((case["n"], case["m"]), device="cuda")
        d.index_add_(0, s["tokens"], s["dy"].float() * case["scale"])
        if s["dW"] is None:
            return d
        s["dW"] += d
        return s["dW"]
    if op == "heads":
        cos, sin = _angles(s)
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x = s[name].float()
            u = x / torch.sqrt(x.square().mean(2, keepdim=True) + EPS) * w
            out[name] = _turn(u, cos, sin, case["interleaved"]).to(t)
        return out
    if op == "heads_grad":
        cos, sin = _angles(s)
        out = {}
        for name, w, dy in (("q", s["wq"], s["dq"]), ("k", s["wk"], s["dk"])):
            x = s[name].float()
            rstd = 1 / torch.sqrt(x.square().mean(2, keepdim=True) + EPS)
            hat = x * rstd
            du = _turn(dy.float(), cos, -sin, case["interleaved"])
            a = du * w
            out["d" + name] = (rstd * (a - hat * (a * hat).mean(2, keepdim=True))).to(t)
            out["dw" + name] = (du * hat).sum((0, 1))
        return out
    if op == "logp":
        z = s["x"].float() * case["scale"]
        top = z.amax(1, keepdim=True)
        d = z - top
        e = torch.exp(d)
        l = torch.log(e.sum(1, keepdim=True))
        out = {"logp": (d.gather(1, s["targets"][:, None]) - l)[:, 0],
               "lse": (top + l)[:, 0]}
        if case["entropy"]:
            p = e * torch.exp(-l)
            out["entropy"] = l[:, 0] - torch.where(p > 0, p * d, 0.0).sum(1)
        if case["top"]:
            at = torch.sort(s["x"], dim=1, descending=True, stable=True)[1][:, :case["top"]]
            out["top"], out["index"] = d.gather(1, at) - l, at
        return out
    if op == "logp_grad":
        z = s["x"].float() * case["scale"]
        q = z - s["stats"][:, :1] - s["stats"][:, 1:]               # log p
        p = torch.exp(q)
        d = -s["g"][:, None] * p
        if s["gh"] is not None:
            d = d - s["gh"][:, None] * torch.where(p > 0, p * (q + s["H"][:, None]), 0.0)
        d.scatter_add_(1, s["targets"][:, None], s["g"][:, None])
        return (d * case["scale"]).to(t)
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for v in s["grads"]:
        total = total + v.double().square().sum()
    norm = torch.sqrt(total) * case["scale"]
    c = torch.where(norm <= s["max_norm"], 1.0, s["max_norm"] / norm).float() * case["scale"]
    for i, v in enumerate(s["grads"]):
        if case["into"]:
            s["into"][i] += v.float() * c
        else:
            v.copy_(v.float() * c)
    return {"norm": norm.float(), "out": s["sums"] if case["into"] else s["flat"]}


# ------------------------------------------------------ the package's calls

def _own(s):
    import orthogonalizing_optimizer_amd as d3
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return d3.embedding(s["tokens"], s["W"], scale=case["scale"], dtype=DTYPES[case["dtype"]])
    if op == "embed_grad":
        return d3.embedding_grad(s["tokens"], s["dy"], case["n"], scale=case["scale"], out=s["dW"],
                                 accumulate=s["dW"] is not None)
    if op == "heads":
        q, k = d3.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"], eps=EPS,
                               interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "heads_grad":
        dq, dk, dwq, dwk = d3.qk_norm_rope_grad(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"],
                                                s["pos"], s["freqs"], eps=EPS,
                                                interleaved=case["interleaved"])
        return {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}
    if op == "logp":
        logp, stats, entropy, top, index = d3.log_probs(
            s["x"], s["targets"], scale=case["scale"], entropy=case["entropy"], top=case["top"])
        out = {"logp": logp, "lse": stats.sum(1)}
        if case["entropy"]:
            out["entropy"] = entropy
        if case["top"]:
            out["top"], out["index"] = top, index
        return out
    if op == "logp_grad":
        return d3.log_probs_grad(s["g"], s["x"], s["targets"], s["stats"], scale=case["scale"],
                                 entropy=s["H"], dentropy=s["gh"])
    norm = d3.clip_grad_norm(s["grads"], s["max_norm"], scale=case["scale"], into=s["into"])
    return {"norm": norm, "out": s["sums"] if case["into"] else s["flat"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- the value in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, from the inputs' own values."""
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op == "embed":
        return torch.index_select(s["W"], 0, s["tokens"]).to(f) * case["scale"]
    if op == "embed_grad":
        n, m = case["n"], case["m"]
        total = s["dW"].to(f) if case["sum"] else torch.zeros((n, m), device="cuda", dtype=f)
        order = torch.argsort(s["tokens"])
        rows, counts = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        ends = torch.cumsum(counts, 0)
        sums = torch.cat([torch.zeros((1, m), device="cuda", dtype=f),
                          torch.cumsum(s["dy"][order].to(f), 0)])
        total[rows] += case["scale"] * (sums[ends] - sums[ends - counts])
        return total
    if op in ("heads", "heads_grad"):
        h, D = case["r"] // 2, case["D"]
        # the rotation as a product with a complex number
        turn = torch.polar(torch.ones((), device="cuda", dtype=f), s["pos"].to(f)[:, None] * s["freqs"])
        lead = torch.arange(h, device="cuda")
        ia, ib = (2 * lead, 2 * lead + 1) if case["interleaved"] else (lead, lead + h)

        def rotate(v, by):
            z = torch.complex(v[..., ia].contiguous(), v[..., ib].contiguous()) * by[:, None]
            v = v.clone()
            v[..., ia], v[..., ib] = z.real, z.imag
            return v

        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x, w = s[name].to(f), w.to(f)
            r = (torch.sum(x * x, 2, keepdim=True) / D + EPS) ** -0.5
            if op == "heads":
                out[name] = rotate(x * r * w, turn)
                continue
            du = rotate(s["d" + name].to(f), turn.conj())
            inner = torch.sum(du * w * x, 2, keepdim=True) / D
            out["d" + name] = r * du * w - r ** 3 * x * inner
            out["dw" + name] = torch.sum(du * x * r, (0, 1))
        return out
    if op == "logp":
        parts = []
        for x, at in zip(s["x"].split(1024), s["targets"].split(1024)):
            lp = torch.log_softmax(x.to(f) * case["scale"], 1)
            part = {"logp": lp.gather(1, at[:, None])[:, 0],
                    "lse": torch.logsumexp(x.to(f) * case["scale"], 1)}
            if case["entropy"]:
                part["entropy"] = torch.special.entr(torch.exp(lp)).sum(1)
            if case["top"]:
                part["top"] = torch.topk(lp, case["top"], 1)[0]
            parts.append(part)
        out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
        if case["top"]:
            out["index"] = None
        return out
    if op == "logp_grad":
        parts = []
        for i in range(0, case["T"], 1024):
            rows = slice(i, i + 1024)
            lp = torch.log_softmax(s["x"][rows].to(f) * case["scale"], 1)
            p = torch.exp(lp)
            hot = torch.nn.functional.one_hot(s["targets"][rows], case["n"])
            d = s["g"][rows, None].to(f) * (hot - p)
            if case["entropy"]:
                e = torch.special.entr(p)
                d += s["gh"][rows, None].to(f) * (e - p * e.sum(1, keepdim=True))
            parts.append((d * case["scale"]).float())    # (whole rows of 64 bits: too many)
        return torch.cat(parts)
    norm = torch.linalg.vector_norm(s["flat"].to(f)) * case["scale"]
    c = torch.clamp(s["max_norm"] / norm, max=1.0) * case["scale"]
    v = s["flat"].to(f) * c
    return {"norm": norm, "out": v + s["sums"].to(f) if case["into"] else v}


# ---------------------------------------------------------- the work of a pass

SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "clip":
        n = _elements(case["shapes"].split(","), case["count"])
        return {"bytes": n * (e + 8) if case["into"] else 2 * n * e, "flops": 4 * n}
    T = case["T"]
    if op == "embed":
        n, m = case["n"], case["m"]
        return {"bytes": min(T, n) * m * SIZE[case["wtype"]] + T * m * e + 8 * T, "flops": T * m}
    if op == "embed_grad":       # a sum touches the rows that have tokens
        n, m = case["n"], case["m"]
        return {"bytes": T * m * e + (8 * min(T, n) if case["sum"] else 4 * n) * m + 8 * T,
                "flops": 2 * T * m}
    if op in ("heads", "heads_grad"):
        n = T * (case["hq"] + case["hk"]) * case["D"]
        return {"bytes": n * e * (2 if op == "heads" else 3) + 8 * T,
                "flops": n * (8 if op == "heads" else 16)}
    n = T * case["n"]
    if op == "logp":
        return {"bytes": n * e + T * (16 + 4 * case["entropy"] + 12 * case["top"]),
                "flops": (8 if case["entropy"] else 5) * n}
    return {"bytes": 2 * n * e + 24 * T, "flops": (8 if case["entropy"] else 4) * n}
