"""The rest of a model's layer around its products, as measured work.

Each kind of case is one operator of the framework:

  gated           Y = act(A x op(Bg) + bg) * (A x op(Bu) + bu), both products in one      (sgemm_gated)
  gated_grad      the gradients of A, Bg, Bu, bg and bu from Y's                          (sgemm_gated_backward)
  gated_e4m3      the gated block on 8-bit (e4m3) operands with their row scales          (gemm_e4m3_gated)
  layernorm       S = X + R; Y = (S - mean) / sqrt(var + eps) * w + b, in float32
                  or as 8-bit codes with one scale a row                                  (layernorm, layernorm_e4m3)
  layernorm_grad  the gradients of X (and R), w and b                                     (layernorm_backward)
  clip            the norm of all elements of many tensors, and the tensors scaled
                  down to a largest norm                                                  (clip_grad_norm)

With `own` false, run() computes them in elementary torch operations in 32
bits; with `own` true it calls the framework.
"""
import math

import torch

own = False

EPS = 1e-5
CLIP_EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale (the smallest normal float32)
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


def listed():
    return [
        # one token through the widening half of a layer, both weights in one tensor of one row per output:
        # the weights' stream
        {"name": "gated 1x8192x2048", "kind": "gated", "M": 1, "N": 8192, "K": 2048, "tb": True, "merged": True,
         "act": "silu", "bias": False, "pre": False, "pad": 0},
        # the widening half of a training step on 2048 tokens, which keeps its pre-activations for the gradient
        {"name": "gated 2048x8192x2048", "kind": "gated", "M": 2048, "N": 8192, "K": 2048, "tb": False,
         "merged": False, "act": "gelu", "bias": True, "pre": True, "pad": 0},
        # the gradient of a small layer of odd sizes with two weight tensors
        {"name": "gated_grad 515x2051x1023", "kind": "gated_grad", "M": 515, "N": 2051, "K": 1023, "tb": True,
         "merged": False, "act": "gelu_tanh", "pad": 0},
        # the gradient of that half of a training step
        {"name": "gated_grad 2048x8192x2048", "kind": "gated_grad", "M": 2048, "N": 8192, "K": 2048, "tb": False,
         "merged": True, "act": "silu", "pad": 0},
        # one token through a small layer with 8-bit weights: latency
        {"name": "gated_e4m3 1x2048x512", "kind": "gated_e4m3", "M": 1, "N": 2048, "K": 512, "merged": True,
         "act": "silu", "bias": False, "pad": 0},
        # a long prompt through a layer with 8-bit weights
        {"name": "gated_e4m3 4096x8192x8192", "kind": "gated_e4m3", "M": 4096, "N": 8192, "K": 8192, "merged": False,
         "act": "gelu_tanh", "bias": True, "pad": 0},
        # one token, added to the residual stream
        {"name": "layernorm 1x8192", "kind": "layernorm", "rows": 1, "D": 8192, "residual": True, "bias": True,
         "e4m3": False, "pad": 0},
        # a long prompt before an 8-bit layer, with the residual stream written back
        {"name": "layernorm 8192x8192 e4m3", "kind": "layernorm", "rows": 8192, "D": 8192, "residual": True,
         "bias": True, "e4m3": True, "pad": 0},
        # a short batch of odd width
        {"name": "layernorm_grad 515x2051", "kind": "layernorm_grad", "rows": 515, "D": 2051, "stream": False,
         "pad": 0},
        # a training step on 8192 tokens, with the gradient that comes down the residual stream
        {"name": "layernorm_grad 8192x4096", "kind": "layernorm_grad", "rows": 8192, "D": 4096, "stream": True,
         "pad": 0},
        # the gradients of a small network: many little tensors
        {"name": "clip 2x96x250", "kind": "clip", "layers": 2, "width": 96, "inner": 250, "max_norm": 1.0, "pad": 0},
        # the gradients of eight layers
        {"name": "clip 8x2048x8192", "kind": "clip", "layers": 8, "width": 2048, "inner": 8192, "max_norm": 1.0,
         "pad": 0},
    ]


# The cost of the largest listed case of a kind: the operations of its products, rows*D of a row operator, elements.
MOST_PRODUCT = {"gated": 4 * 2048 * 8192 * 2048, "gated_grad": 4 * 2048 * 8192 * 2048,
                "gated_e4m3": 4 * 4096 * 8192 * 8192}
MOST_ROWS = {"layernorm": 8192 * 8192, "layernorm_grad": 8192 * 4096}


def _shapes(layers, width, inner):
    """The parameters of a stack of layers: per layer the projections of the
    mixing half, the two halves of a gated block in one tensor, the way back,
    and the vectors of two norms and two biases."""
    one = [(width, 4 * width), (width, 2 * inner), (inner, width), (width,), (width,), (2 * inner,), (width,)]
    return one * layers


def _elements(case):
    return sum(math.prod(s) for s in _shapes(case["layers"], case["width"], case["inner"]))


MOST_ELEMENTS = _elements({"layers": 8, "width": 2048, "inner": 8192})


def _size(rng, low, high):
    """Spread over the logarithm; half of them rounded to a multiple of 64 where large enough."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))
    if n >= 128 and rng.random() < 0.5:
        n = n // 64 * 64
    return max(low, min(high, n))


def draw(rng):
    kind = rng.choice(["gated", "gated_grad", "gated_e4m3", "layernorm", "layernorm_grad", "clip"])
    pad = rng.choice([0, 0, 1, 4, 16])  # elements between the end of a row and the next
    if kind == "clip":
        while True:
            case = {"kind": kind, "layers": _size(rng, 1, 48), "width": _size(rng, 16, 4096),
                    "inner": _size(rng, 16, 8192), "max_norm": rng.choice([0.5, 1.0, 1e6]), "pad": pad}
            if _elements(case) <= MOST_ELEMENTS:
                return case
    if kind in MOST_ROWS:
        while True:
            rows, d = _size(rng, 1, 8192), _size(rng, 64, 16384)
            if rows * d <= MOST_ROWS[kind]:
                break
        case = {"kind": kind, "rows": rows, "D": d, "pad": pad}
        if kind == "layernorm_grad":
            return case | {"stream": rng.random() < 0.5}
        return case | {"residual": rng.random() < 0.7, "bias": rng.random() < 0.7, "e4m3": rng.random() < 0.5}
    while True:
        m, n, k = _size(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 8192)
        if 4 * m * n * k <= MOST_PRODUCT[kind]:
            break
    case = {"kind": kind, "M": m, "N": n, "K": k, "pad": pad, "merged": rng.random() < 0.5,
            "act": rng.choice(ACTIVATIONS[1:] + ("silu", "silu") + ACTIVATIONS[:1])}
    if kind == "gated_e4m3":
        return case | {"bias": rng.random() < 0.4}
    case |= {"tb": rng.random() < 0.5}
    if kind == "gated_grad":
        return case
    return case | {"bias": rng.random() < 0.4, "pre": rng.random() < 0.4}


def _rows(make, rows, cols, pad):
    """A rows x cols matrix whose rows are `pad` elements apart."""
    return make(rows, cols + pad)[:, :cols]


def _halves(make, n, k, tb, merged, pad):
    """The two weights: stored (n, k) or (k, n), in one tensor or in two."""
    if not merged:
        shape = (n, k) if tb else (k, n)
        return _rows(make, *shape, pad), _rows(make, *shape, pad)
    both = _rows(make, 2 * n, k, pad) if tb else _rows(make, k, 2 * n, pad)
    return (both[:n], both[n:]) if tb else (both[:, :n], both[:, n:])


def _codes(x, pad):
    """Rows of x in 8 bits, with the scale of each: what a program keeps of its weights."""
    scale = (x.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    codes = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=torch.uint8, device=x.device)
    codes = codes.view(torch.float8_e4m3fn)[:, :x.shape[1]]
    codes.copy_((x / scale[:, None]).to(torch.float8_e4m3fn))
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    c, pad = case, case["pad"]
    s = {"case": dict(c)}
    if c["kind"] in ("gated", "gated_grad"):
        m, n, k = c["M"], c["N"], c["K"]
        s["A"] = _rows(normal, m, k, pad)
        # weights scaled as at a layer's start, so that pre-activations are of order one
        s["Bg"], s["Bu"] = (b.mul_(k ** -0.5) for b in _halves(normal, n, k, c["tb"], c["merged"], pad))
        if c["kind"] == "gated":
            s["bg"], s["bu"] = (normal(n).mul_(0.5), normal(n).mul_(0.5)) if c["bias"] else (None, None)
        else:
            s["dY"], s["G"], s["U"] = (_rows(normal, m, n, pad) for _ in range(3))
    elif c["kind"] == "gated_e4m3":
        m, n, k = c["M"], c["N"], c["K"]
        s["A"], s["sa"] = _codes(normal(m, k), pad)
        both, scale = _codes(normal(2 * n, k) * k ** -0.5, pad)
        s["Bg"], s["Bu"], s["sg"], s["su"] = both[:n], both[n:], scale[:n], scale[n:]
        if not c["merged"]:
            s["Bu"], s["su"] = _rows(lambda r, w: torch.zeros(r, w, dtype=torch.uint8, device="cuda")
                                     .view(torch.float8_e4m3fn), n, k, pad).copy_(s["Bu"]), s["su"].clone()
        s["bg"], s["bu"] = (normal(n).mul_(0.5), normal(n).mul_(0.5)) if c["bias"] else (None, None)
    elif c["kind"] == "clip":
        # gradients of unlike size; the buffers that the scaled ones go to are the program's own
        shapes = _shapes(c["layers"], c["width"], c["inner"])
        s["x"] = [(_rows(normal, *shape, pad) if len(shape) == 2 else normal(*shape)).mul_(10.0 ** -(i % 4))
                  for i, shape in enumerate(shapes)]
        s["out"] = [torch.empty_like(x) for x in s["x"]]
    else:
        rows, d = c["rows"], c["D"]
        # rows of unlike size, with a mean, as tokens of a residual stream are
        s["X"] = _rows(normal, rows, d, pad).add_(normal(rows, 1)).mul_(torch.exp(normal(rows, 1)))
        s["w"] = 1.0 + 0.1 * normal(d)
        if c["kind"] == "layernorm":
            s["R"] = _rows(normal, rows, d, pad) if c["residual"] else None
            s["b"] = normal(d).mul_(0.1) if c["bias"] else None
        else:
            s["dY"] = _rows(normal, rows, d, pad)
            s["dS"] = _rows(normal, rows, d, pad) if c["stream"] else None
    return s


# ---- the plain forms -----------------------------------------------------------------


def _act(z, name):
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 3 * GELU_A * z * z)
    sig = 1.0 / (1.0 + torch.exp(-z))
    return sig * (1.0 + z * (1.0 - sig))


def _plain_gated(s, c):
    if c["kind"] == "gated_e4m3":
        a = s["A"].float()
        gate = (a @ s["Bg"].float().T) * s["sa"][:, None] * s["sg"]
        up = (a @ s["Bu"].float().T) * s["sa"][:, None] * s["su"]
    else:
        gate = s["A"] @ (s["Bg"].T if c["tb"] else s["Bg"])
        up = s["A"] @ (s["Bu"].T if c["tb"] else s["Bu"])
    if s["bg"] is not None:
        gate, up = gate + s["bg"], up + s["bu"]
    y = _act(gate, c["act"]) * up
    return {"Y": y, "G": gate, "U": up} if c.get("pre") else {"Y": y}


def _plain_gated_grad(s, c):
    dy, gate, up = s["dY"], s["G"], s["U"]
    dg = dy * up if c["act"] == "none" else dy * up * _act_grad(gate, c["act"])
    du = dy * _act(gate, c["act"])
    bg, bu = (s["Bg"], s["Bu"]) if c["tb"] else (s["Bg"].T, s["Bu"].T)
    out = {"dA": dg @ bg + du @ bu}
    if c["tb"]:
        out |= {"dBg": dg.T @ s["A"], "dBu": du.T @ s["A"]}
    else:
        out |= {"dBg": s["A"].T @ dg, "dBu": s["A"].T @ du}
    return out | {"dbg": dg.sum(0), "dbu": du.sum(0)}


def _plain_layernorm(s, c):
    x = s["X"] if s["R"] is None else s["X"] + s["R"]
    h = x - x.mean(1, keepdim=True)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    if c["e4m3"]:
        scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
        out = {"Q": (y * (1.0 / scale)[:, None]).to(torch.float8_e4m3fn), "scale": scale}
    else:
        out = {"Y": y}
    return out if s["R"] is None else out | {"S": x}


def _plain_layernorm_grad(s, c):
    x, dy = s["X"], s["dY"]
    h = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    h = h * r
    g = dy * s["w"]
    dx = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if s["dS"] is not None:
        dx = dx + s["dS"]
    return {"dX": dx, "dw": (dy * h).sum(0), "db": dy.sum(0)}


def _plain_clip(s, c):
    # (long sums of squares: 64 bits)
    total = torch.stack([(x * x).sum(dtype=torch.float64) for x in s["x"]]).sum()
    norm = total.sqrt().float()
    factor = (c["max_norm"] / (norm + CLIP_EPS)).clamp_max(1.0)
    return {"norm": norm, "y": [x * factor for x in s["x"]]}


def _plain(s, c):
    if c["kind"] in ("gated", "gated_e4m3"):
        return _plain_gated(s, c)
    if c["kind"] == "gated_grad":
        return _plain_gated_grad(s, c)
    if c["kind"] == "layernorm":
        return _plain_layernorm(s, c)
    if c["kind"] == "layernorm_grad":
        return _plain_layernorm_grad(s, c)
    return _plain_clip(s, c)


# ---- the framework's calls -----------------------------------------------------------


def _own(s, c):
    import fp32_gemm_sgemm_amd as sg
    if c["kind"] == "gated":
        m, n = c["M"], c["N"]
        pre = (torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")) if c["pre"] else (None, None)
        y = sg.sgemm_gated(s["A"], s["Bg"], s["Bu"], bias_gate=s["bg"], bias_up=s["bu"], activation=c["act"],
                           pre_gate=pre[0], pre_up=pre[1], transb=c["tb"])
        return {"Y": y, "G": pre[0], "U": pre[1]} if c["pre"] else {"Y": y}
    if c["kind"] == "gated_grad":
        da, dbg, dbu, dbias_g, dbias_u = sg.sgemm_gated_backward(
            s["dY"], s["A"], s["Bg"], s["Bu"], pre_gate=s["G"], pre_up=s["U"], activation=c["act"], transb=c["tb"])
        return {"dA": da, "dBg": dbg, "dBu": dbu, "dbg": dbias_g, "dbu": dbias_u}
    if c["kind"] == "gated_e4m3":
        return {"Y": sg.gemm_e4m3_gated(s["A"], s["sa"], s["Bg"], s["sg"], s["Bu"], s["su"], bias_gate=s["bg"],
                                        bias_up=s["bu"], activation=c["act"])}
    if c["kind"] == "layernorm":
        if c["e4m3"]:
            q, scale, x = sg.layernorm_e4m3(s["X"], s["w"], s["b"], eps=EPS, residual=s["R"])
            out = {"Q": q, "scale": scale}
        else:
            y, x = sg.layernorm(s["X"], s["w"], s["b"], eps=EPS, residual=s["R"])
            out = {"Y": y}
        return out if s["R"] is None else out | {"S": x}
    if c["kind"] == "layernorm_grad":
        dx, dw, db = sg.layernorm_backward(s["dY"], s["X"], s["w"], eps=EPS, dsum=s["dS"])
        return {"dX": dx, "dw": dw, "db": db}
    norm = sg.clip_grad_norm(s["x"], c["max_norm"], eps=CLIP_EPS, out=s["out"])
    return {"norm": norm, "y": s["out"]}


def run(state):
    if own:
        return _own(state, state["case"])
    return _plain(state, state["case"])


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    c = case
    if c["kind"] in ("gated", "gated_grad", "gated_e4m3"):
        m, n, k = c["M"], c["N"], c["K"]
        if c["kind"] == "gated":
            return {"bytes": 4 * (m * k + 2 * k * n + m * n * (3 if c["pre"] else 1) + 2 * n * c["bias"]),
                    "flops": 4 * m * n * k}
        if c["kind"] == "gated_e4m3":
            return {"bytes": m * k + 2 * n * k + 4 * (m + 2 * n + 2 * n * c["bias"] + m * n),
                    "flops": 4 * m * n * k}
        return {"bytes": 4 * (3 * m * n + 2 * m * k + 4 * k * n + 2 * n), "flops": 8 * m * n * k}
    if c["kind"] == "clip":
        return {"bytes": 8 * _elements(c), "flops": 3 * _elements(c)}
    e = c["rows"] * c["D"]
    if c["kind"] == "layernorm":
        out = (e + 4 * c["rows"]) if c["e4m3"] else 4 * e
        return {"bytes": 4 * e * (3 if c["residual"] else 1) + 4 * c["D"] * (1 + c["bias"]) + out, "flops": 9 * e}
    return {"bytes": 4 * e * (4 if c["stream"] else 3) + 12 * c["D"], "flops": 14 * e}


# ---- the definitions in 64 bits ------------------------------------------------------


def _phi(z):
    """The normal distribution's probability below z."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _gelu_tanh_gate(z):
    return torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


_VALUE = {
    "none": lambda z: z,
    "relu": lambda z: z.clamp(min=0),
    "gelu": lambda z: z * _phi(z),
    "gelu_tanh": lambda z: z * _gelu_tanh_gate(z),
    "silu": lambda z: z * torch.sigmoid(z),
}


def _slope_gelu_tanh(z):
    p = _gelu_tanh_gate(z)
    return p + z * p * (1 - p) * 2.0 * math.sqrt(2.0 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


_SLOPE = {
    "none": torch.ones_like,
    "relu": lambda z: (z > 0).double(),
    "gelu": lambda z: _phi(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi),
    "gelu_tanh": _slope_gelu_tanh,
    "silu": lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z),
}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "clip":
        total = sum(torch.linalg.vector_norm(x.double()).square() for x in s["x"])
        norm = total.sqrt()
        factor = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0)
        return {"norm": norm, "y": [x.double() * factor for x in s["x"]]}
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if kind in ("gated", "gated_e4m3"):
        if kind == "gated":
            a, (bg, bu) = d["A"], ((d[b].T if case["tb"] else d[b]) for b in ("Bg", "Bu"))
        else:
            a = d["A"] * d["sa"][:, None]
            bg, bu = (d["Bg"] * d["sg"][:, None]).T, (d["Bu"] * d["su"][:, None]).T
        gate, up = torch.mm(a.contiguous(), bg.contiguous()), torch.mm(a.contiguous(), bu.contiguous())
        if "bg" in d:
            gate += d["bg"][None, :]
            up += d["bu"][None, :]
        y = _VALUE[case["act"]](gate) * up
        return {"Y": y, "G": gate, "U": up} if case.get("pre") else {"Y": y}
    if kind == "gated_grad":
        du = d["dY"] * _VALUE[case["act"]](d["G"])
        dg = d["dY"] * _SLOPE[case["act"]](d["G"]) * d["U"]
        wide = torch.cat([dg, du], dim=1)                         # (M, 2N)
        if case["tb"]:
            weights = torch.cat([d["Bg"], d["Bu"]], dim=0)        # (2N, K)
        else:
            weights = torch.cat([d["Bg"], d["Bu"]], dim=1).T.contiguous()
        dw = torch.mm(wide.T.contiguous(), d["A"].contiguous())   # (2N, K)
        n = case["N"]
        halves = (dw[:n], dw[n:]) if case["tb"] else (dw[:n].T, dw[n:].T)
        return {"dA": torch.mm(wide, weights), "dBg": halves[0], "dBu": halves[1],
                "dbg": torch.sum(dg, dim=0), "dbu": torch.sum(du, dim=0)}
    x = d["X"] + d["R"] if "R" in d else d["X"]
    n = x.shape[1]
    centred = x - (x.sum(1) / n)[:, None]
    inv = (centred.pow(2).sum(1) / n + EPS).pow(-0.5)[:, None]
    unit = centred * inv
    if kind == "layernorm_grad":
        up = d["dY"] * d["w"]
        dx = inv * (up - (up.sum(1) / n)[:, None] - unit * ((up * unit).sum(1) / n)[:, None])
        return {"dX": dx + d["dS"] if "dS" in d else dx, "dw": (d["dY"] * unit).sum(0), "db": d["dY"].sum(0)}
    y = unit * d["w"]
    if "b" in d:
        y = y + d["b"]
    if case["e4m3"]:
        scale = torch.clamp(torch.max(torch.abs(y), dim=1).values / E4M3_MAX, min=TINY)
        out = {"Q": (y / scale[:, None]).float().to(torch.float8_e4m3fn), "scale": scale}
    else:
        out = {"Y": y}
    return out | {"S": x} if "R" in d else out
