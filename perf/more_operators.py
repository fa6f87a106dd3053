"""What the operators around the experts' products are measured on: root-mean-square norm into e4m3, products of
8-bit operands with an epilogue, gated activations into e4m3, and products by expert of 16-bit operands.

A case names one operator and its sizes. ``prepare`` makes what a program holds before the call, ``run`` makes one
pass, ``exact`` gives the same outputs from the definitions in 64 bits (values in e4m3 before their rounding). With
``own`` false, ``run`` uses elementary torch operations only; with ``own`` true, the calls of this repository's package.

The operators (rows are tokens; a block is 128 consecutive values of a row, the last one shorter; e4m3 values are
q = e4m3(v / s) with s = max|block| / 448):

* norm: h = x + r, rounded to the type of x (h = x without r); a = 1 / sqrt(mean(h^2) + eps) of each row;
  y = h a w in blocks of e4m3. With "train" also, for gradients dy of y and dh of h, g = w dy and n = h a,
  dx = a (g - n mean(g n)) + dh (the gradient of x and of r), dw = sum over rows of dy n;
* epilogue: p = A B^T + bias and C = act(p) + residual for e4m3 A (m x k) and B (n x k) with scales; "backward":
  dp = act'(p) dc for a kept p, and the bias' gradient, the sum of act'(p) dc over the rows;
* gated: h = [g | u], z = act(g) u in blocks of e4m3; with "train" also dg = act'(g) u dz, du = act(g) dz;
* experts: rows [offsets[e], offsets[e + 1]) belong to expert e, rows from the last offset on to none. "forward":
  y = x W_e^T for W_e of n x k (zero for the last rows); "train": also dx = dy W_e and dW_e = dy^T x, in 32 bits.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
FP8 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 number
LEAST = 2.0 ** -64  # the least magnitude a block is scaled by, so that no scale is zero or subnormal
EPS = 1e-6


def listed():
    return [
        # a decoding step of eight sequences: the residual stream on its way into an 8-bit product; latency is all
        {"name": "norm_decode", "op": "norm", "rows": 8, "cols": 4096, "type": "bf16", "weight": "fp32",
         "residual": True, "train": False},
        # an odd prompt whose rows end inside a block and are not a whole number of loads
        {"name": "norm_ragged", "op": "norm", "rows": 3001, "cols": 2047, "type": "fp16", "weight": "same",
         "residual": True, "train": False},
        # a training batch, forward and backward
        {"name": "norm_train", "op": "norm", "rows": 8192, "cols": 4096, "type": "bf16", "weight": "fp32",
         "residual": True, "train": True},
        # a layer of a decoding step: reads its weights once
        {"name": "epilogue_decode", "op": "epilogue", "form": "forward", "scales": "blocks", "m": 8, "n": 4096,
         "k": 4096, "act": "silu", "bias": True, "residual": True, "keep": False, "type": "bf16"},
        # odd sizes with a 32-bit result that keeps its argument of the activation
        {"name": "epilogue_ragged", "op": "epilogue", "form": "forward", "scales": "rows", "m": 3001, "n": 2047,
         "k": 1537, "act": "gelu", "bias": True, "residual": True, "keep": True, "type": "fp32"},
        # a layer of a long prompt or a training batch
        {"name": "epilogue_train", "op": "epilogue", "form": "forward", "scales": "blocks", "m": 8192, "n": 8192,
         "k": 4096, "act": "gelu_tanh", "bias": True, "residual": False, "keep": True, "type": "bf16"},
        # its way back, as far as the products that follow
        {"name": "epilogue_backward", "op": "epilogue", "form": "backward", "scales": "blocks", "m": 8192, "n": 8192,
         "k": 4096, "act": "gelu_tanh", "bias": True, "residual": False, "keep": True, "type": "bf16"},
        # between the experts' two products in a decoding step
        {"name": "gated_decode", "op": "gated", "rows": 64, "cols": 2048, "act": "silu", "type": "bf16", "train": False},
        # the same for a training batch, with its backward pass
        {"name": "gated_train", "op": "gated", "rows": 16384, "cols": 2048, "act": "silu", "type": "bf16", "train": True},
        # experts in a decoding step: few rows each, the weights' bytes count
        {"name": "experts16_decode", "op": "experts", "form": "forward", "tokens": 16, "choices": 4, "experts": 32,
         "n": 2048, "k": 4096, "spare": 0, "type": "bf16"},
        # experts over a prompt
        {"name": "experts16_prompt", "op": "experts", "form": "forward", "tokens": 4096, "choices": 4, "experts": 32,
         "n": 2048, "k": 4096, "spare": 0, "type": "bf16"},
        # a training step of the experts: the product, the gradients of its rows and of its weights
        {"name": "experts16_train", "op": "experts", "form": "train", "tokens": 4096, "choices": 2, "experts": 8,
         "n": 2048, "k": 1024, "spare": 5, "type": "fp16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "epilogue", "gated", "experts"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 16, 4096), "type": rng.choice(["bf16", "fp16", "fp32"]),
                "weight": rng.choice(["fp32", "same"]), "residual": rng.random() < 0.7, "train": rng.random() < 0.5}
    if op == "epilogue":
        form = rng.choice(["forward", "forward", "backward"])
        return {"op": op, "form": form, "scales": rng.choice(["blocks", "rows"]), "m": _log(rng, 1, 8192),
                "n": _log(rng, 64, 8192), "k": _log(rng, 100, 4096),
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "keep": rng.random() < 0.5, "type": rng.choice(["bf16", "fp32", "fp16"])}
    if op == "gated":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 16, 4096),
                "act": rng.choice(["relu", "silu", "gelu", "gelu_tanh"]), "type": rng.choice(["bf16", "fp32", "fp16"]),
                "train": rng.random() < 0.5}
    experts = rng.choice([4, 8, 12, 16, 32])
    form = rng.choice(["forward", "train"])
    return {"op": op, "form": form, "tokens": _log(rng, 1, 4096), "choices": rng.randint(1, 4), "experts": experts,
            "n": _log(rng, 64, 2048), "k": _log(rng, 64, 2048 if form == "train" else 4096),
            "spare": rng.choice([0, 0, 1, 37]), "type": rng.choice(["bf16", "fp16"])}


# ---- inputs ------------------------------------------------------------------

def _normal(g, *shape, spread=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * spread


def _blocked(x):
    """x (..., n, k) with k filled up with zeros to whole blocks: (..., n, blocks, 128)."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 128)).unflatten(-1, (-1, 128))


def _scale_of(most):
    return most.clamp_min(LEAST) / torch.full_like(most, TOP)  # a quotient; by a number torch takes the reciprocal


def _row_quantised(x):
    """e4m3 values of x's blocks along its rows, and their scales."""
    b = _blocked(x)
    s = _scale_of(b.abs().amax(-1))
    return (b / s.unsqueeze(-1)).flatten(-2)[..., : x.shape[-1]].to(FP8), s


def _tile_quantised(x):
    """e4m3 values of x's 128 x 128 blocks, and their scales."""
    n, k = x.shape
    b = _blocked(torch.nn.functional.pad(x, (0, 0, 0, -n % 128))).unflatten(0, (-1, 128))
    s = _scale_of(b.abs().amax((1, 3)))
    return (b / s[:, None, :, None]).flatten(2).flatten(0, 1)[:n, :k].to(FP8), s


def _stored(q, s, by_block=True):
    """As the quantisers store them: rows of a stride that is a multiple of 16 bytes, the rows' scales block by block."""
    k = q.shape[-1]
    room = torch.zeros(q.shape[0], k + -k % 16, dtype=torch.uint8, device=q.device)
    room[:, :k] = q.view(torch.uint8)
    return room.view(FP8)[:, :k], s.t().contiguous().t() if by_block else s.contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[c["type"]]
    if c["op"] == "norm":
        rows, cols = c["rows"], c["cols"]
        wide = torch.exp(_normal(g, 1, cols, spread=0.7))  # some channels of a residual stream are larger
        c["x"] = _normal(g, rows, cols, spread=0.5).to(kind)
        c["r"] = (_normal(g, rows, cols, spread=2.0) * wide).to(kind) if c["residual"] else None
        c["w"] = (1.0 + _normal(g, cols, spread=0.2)).to(kind if c["weight"] == "same" else torch.float32)
        c["dy"] = _normal(g, rows, cols, spread=0.1).to(kind) if c["train"] else None
        c["dh"] = _normal(g, rows, cols, spread=0.1).to(kind) if c["train"] else None
    elif c["op"] == "epilogue":
        m, n, k = c["m"], c["n"], c["k"]
        c["bias_values"] = _normal(g, n, spread=0.3) if c["bias"] else None
        if c["form"] == "forward":
            c["a"], c["sa"] = _stored(*_row_quantised(_normal(g, m, k)))
            w = _normal(g, n, k, spread=k ** -0.5)
            c["b"], c["sb"] = _stored(*_row_quantised(w)) if c["scales"] == "rows" else _stored(*_tile_quantised(w), False)
            c["res"] = _normal(g, m, n).to(kind) if c["residual"] else None
        else:
            c["p"] = _normal(g, m, n, spread=1.1).to(kind)
            c["dc"] = _normal(g, m, n, spread=0.1).to(kind)
    elif c["op"] == "gated":
        c["h"] = _normal(g, c["rows"], 2 * c["cols"], spread=1.2).to(kind)
        c["dz"] = _normal(g, c["rows"], c["cols"], spread=0.1).to(kind) if c["train"] else None
    else:
        e, k, n = c["experts"], c["k"], c["n"]
        liked = _normal(g, c["tokens"], e) + _normal(g, e, spread=0.4)  # some experts are liked better than others
        ids = liked.sort(dim=-1, descending=True, stable=True).indices[:, : c["choices"]].flatten().sort().values
        c["offsets"] = torch.searchsorted(ids, torch.arange(e + 1, device=ids.device)).int()
        c["counts"] = c["offsets"].diff().tolist()
        rows = ids.numel() + c["spare"]
        c["x"] = _normal(g, rows, k).to(kind)
        c["w"] = _normal(g, e, n, k, spread=k ** -0.5).to(kind)
        c["dy"] = _normal(g, rows, n, spread=0.1).to(kind) if c["form"] == "train" else None
    return c


# ---- one pass ----------------------------------------------------------------

def run(c):
    return (_own if own else _plain)(c)


def _own(c):
    import dense_fp32_matrix_02_amd as sg

    if c["op"] == "norm":
        q, s, h, a = sg.rms_norm_fp8(c["x"], c["w"], residual=c["r"], eps=EPS)
        return [q, s, h, a] + (list(sg.rms_norm_backward(c["dy"], h, a, c["w"], dH=c["dh"])) if c["train"] else [])
    if c["op"] == "epilogue":
        if c["form"] == "forward":
            return sg.gemm_fp8_epilogue(c["a"], c["sa"], c["b"], c["sb"], bias=c["bias_values"], activation=c["act"],
                                        residual=c["res"], pre=c["keep"], dtype=TYPES[c["type"]])
        return sg.epilogue_backward(c["dc"], c["p"], activation=c["act"])
    if c["op"] == "gated":
        out = list(sg.gated_fp8(c["h"], activation=c["act"]))
        return out + [sg.gated_backward(c["dz"], c["h"], activation=c["act"])] if c["train"] else out
    y = sg.gemm_experts(c["x"], c["w"], c["offsets"])
    if c["form"] == "forward":
        return y
    return [y, sg.gemm_experts_dgrad(c["dy"], c["w"], c["offsets"]), sg.gemm_experts_wgrad(c["dy"], c["x"], c["offsets"])]


def _plain(c):
    return {"norm": _plain_norm, "epilogue": _plain_epilogue, "gated": _plain_gated, "experts": _plain_experts}[c["op"]](c)


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _act(p, name):
    """act(p) and act'(p)."""
    if name == "none":
        return p, torch.ones_like(p)
    if name == "relu":
        return torch.where(p > 0, p, 0.0), (p > 0).to(p.dtype)
    if name == "silu":
        s = _sigmoid(p)
        return p * s, s * (1 + p * (1 - s))
    if name == "gelu":
        half = 0.5 * (1 + torch.erf(p * math.sqrt(0.5)))
        return p * half, half + p * torch.exp(-0.5 * p * p) * (2 * math.pi) ** -0.5
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (p + b * p * p * p))
    return 0.5 * p * (1 + t), 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * a * (1 + 3 * b * p * p)


def _plain_norm(c):
    kind = TYPES[c["type"]]
    h = c["x"] if c["r"] is None else (c["x"].float() + c["r"].float()).to(kind)
    wide, w = h.float(), c["w"].float()
    a = 1 / torch.sqrt((wide * wide).mean(-1, keepdim=True) + EPS)
    n = wide * a
    out = [*_row_quantised(n * w), h, a.squeeze(-1)]
    if c["train"]:
        dy = c["dy"].float()
        g = w * dy
        dx = a * (g - n * (g * n).mean(-1, keepdim=True)) + c["dh"].float()
        out += [dx.to(kind), (dy * n).sum(0)]
    return out


def _values(q, s):
    """The 32-bit values of e4m3 rows with a scale for each block of a row, or for each 128 x 128 block."""
    s = s if s.shape[0] == q.shape[0] else s.repeat_interleave(128, 0)[: q.shape[0]]
    return (_blocked(q.float()) * s.unsqueeze(-1)).flatten(-2)[:, : q.shape[1]]


def _plain_epilogue(c):
    kind = TYPES[c["type"]]
    if c["form"] == "backward":
        dp = _act(c["p"].float(), c["act"])[1] * c["dc"].float()
        return [dp.to(kind), dp.sum(0)]
    p = _values(c["a"], c["sa"]) @ _values(c["b"], c["sb"]).t().contiguous()
    p = p if c["bias_values"] is None else p + c["bias_values"]
    out = _act(p, c["act"])[0]
    out = (out if c["res"] is None else out + c["res"].float()).to(kind)
    return (out, p.to(kind)) if c["keep"] else out


def _plain_gated(c):
    g, u = c["h"].float().chunk(2, dim=1)
    value, slope = _act(g, c["act"])
    out = list(_row_quantised(value * u))
    if c["train"]:
        dz = c["dz"].float()
        out.append(torch.cat([dz * u * slope, dz * value], 1).to(TYPES[c["type"]]))
    return out


def _plain_experts(c):
    kind, off = TYPES[c["type"]], c["offsets"].long()
    at = torch.arange(max(c["counts"]), device=off.device)
    there = at < off.diff().unsqueeze(1)  # which of the room of each expert is in use
    rows = torch.where(there, off[:-1, None] + at, 0)
    x, w = c["x"].float()[rows] * there.unsqueeze(-1), c["w"].float()

    def back(y):
        out = torch.zeros(c["x"].shape[0], y.shape[-1], device=y.device)
        out[: sum(c["counts"])] = y[there]
        return out.to(kind)

    y = back(torch.bmm(x, w.transpose(1, 2).contiguous()))
    if c["form"] == "forward":
        return y
    dy = c["dy"].float()[rows] * there.unsqueeze(-1)
    return [y, back(torch.bmm(dy, w)), torch.bmm(dy.transpose(1, 2).contiguous(), x)]


# ---- what a pass cannot do without ---------------------------------------------

def work(c):
    size = SIZE[c["type"]]
    if c["op"] == "norm":
        n, w = c["rows"] * c["cols"], c["cols"] * (4 if c["weight"] == "fp32" else size)
        b = n * (size * (3 if c["residual"] else 2) + 1) + 4 * c["rows"] * (1 + -(-c["cols"] // 128)) + w
        return {"bytes": b + c["train"] * (4 * n * size + 4 * c["rows"] + w + 4 * c["cols"]), "flops": n * (6 + 9 * c["train"])}
    if c["op"] == "epilogue":
        m, n, k = c["m"], c["n"], c["k"]
        if c["form"] == "backward":
            return {"bytes": 3 * m * n * size + 4 * n, "flops": 12 * m * n}
        rows = n if c["scales"] == "rows" else -(-n // 128)
        return {"bytes": (m + n) * k + 4 * -(-k // 128) * (m + rows) + m * n * size * (1 + c["residual"] + c["keep"]) +
                4 * n * c["bias"], "flops": 2 * m * n * k}
    if c["op"] == "gated":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 * size + 1) + 4 * c["rows"] * -(-c["cols"] // 128) + c["train"] * 5 * n * size,
                "flops": n * (8 + 12 * c["train"])}
    e, n, k, size = c["experts"], c["n"], c["k"], 2
    r, j = c["tokens"] * min(c["choices"], e), min(c["choices"], e)
    used = e * (1 - (1 - j / e) ** c["tokens"])  # experts with a row, on average
    b = int((r + c["spare"]) * n * size + r * k * size + used * n * k * size)
    if c["form"] == "train":  # dy and W give dx, dy and x give dW
        b += int((r + c["spare"]) * k * size + r * n * size + used * n * k * size) + (r * (n + k) * size + 4 * e * n * k)
    return {"bytes": b, "flops": 2 * r * n * k * (3 if c["form"] == "train" else 1)}


# ---- the definitions in 64 bits, written apart from the plain form ------------------

def exact(case, seed):
    c = prepare(case, seed)
    return {"norm": _exact_norm, "epilogue": _exact_epilogue, "gated": _exact_gated, "experts": _exact_experts}[c["op"]](c)


def _exact_quantised(v):
    """v over the scale of its block, before the rounding to e4m3, and the scales."""
    cols = torch.arange(v.shape[1], device=v.device) // 128
    most = torch.zeros(v.shape[0], int(cols[-1]) + 1, dtype=torch.float64, device=v.device)
    most.scatter_reduce_(1, cols.expand_as(v), v.abs(), "amax")
    scale = torch.clamp(most, min=LEAST) / TOP
    return [v / scale[:, cols], scale]


def _exact_norm(c):
    total = c["x"].double() if c["r"] is None else c["x"].double() + c["r"].double()
    h, w = total.to(c["x"].dtype).double(), c["w"].double()
    norm = torch.rsqrt(h.pow(2).sum(1) / h.shape[1] + EPS)
    out = [*_exact_quantised(torch.einsum("rc,r,c->rc", h, norm, w)), total, norm]
    if c["train"]:
        # y_j = w_j h_j norm and d norm / d h_i = -norm^3 h_i / cols
        dy = c["dy"].double()
        along = (dy * w * h).sum(1)
        dx = torch.einsum("rc,c,r->rc", dy, w, norm) - h * (along * norm ** 3 / h.shape[1]).unsqueeze(1)
        out += [dx + c["dh"].double(), norm @ (dy * h)]
    return out


def _exact_act(p, name):
    """The activation and, by its own derivation, its slope."""
    p = p.detach().requires_grad_(True)
    f = {"none": lambda x: x * 1.0, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
         "gelu": torch.nn.functional.gelu, "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[name]
    with torch.enable_grad():
        y = f(p)
        slope, = torch.autograd.grad(y.sum(), p)
    return y.detach(), slope


def _exact_values(q, s):
    at = torch.arange(q.shape[0], device=q.device) // (1 if s.shape[0] == q.shape[0] else 128)
    return q.float().double() * s.double()[at][:, torch.arange(q.shape[1], device=q.device) // 128]


def _exact_epilogue(c):
    if c["form"] == "backward":
        dp = c["dc"].double() * _exact_act(c["p"].double(), c["act"])[1]
        return [dp, torch.ones(1, dp.shape[0], dtype=torch.float64, device=dp.device).mm(dp)[0]]
    p = torch.mm(_exact_values(c["a"], c["sa"]), _exact_values(c["b"], c["sb"]).t().contiguous())
    if c["bias_values"] is not None:
        p += c["bias_values"].double()
    y = _exact_act(p, c["act"])[0]
    if c["res"] is not None:
        y += c["res"].double()
    return (y, p) if c["keep"] else y


def _exact_gated(c):
    h = c["h"].double()
    n = c["cols"]
    value, slope = _exact_act(h[:, :n].contiguous(), c["act"])
    out = _exact_quantised(value * h[:, n:])
    if c["train"]:
        dz = c["dz"].double()
        out.append(torch.hstack([slope * h[:, n:] * dz, value * dz]))
    return out


def _exact_experts(c):
    off, x = c["offsets"].tolist(), c["x"].double()
    y = torch.zeros(x.shape[0], c["n"], dtype=torch.float64, device=x.device)
    dx, dw = torch.zeros_like(x), []
    for e in range(c["experts"]):
        at, w = slice(off[e], off[e + 1]), c["w"][e].double()
        y[at] = x[at] @ w.t().contiguous()
        if c["form"] == "train":
            dy = c["dy"][at].double()
            dx[at] = dy @ w
            dw.append(dy.t().contiguous() @ x[at])
    return [y, dx, torch.stack(dw)] if c["form"] == "train" else y
