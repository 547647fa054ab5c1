"""Cases for the row-wise operators of a voxel block: RMS norm, linear and gated feed-forward.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the
package's entry points.  ``exact`` gives the same outputs from the operators'
definitions in 64 bits.

A case's ``op`` is one of
  norm           y = (x + residual) / rms * w, and the sum; with ``eight`` y as e4m3 with a scale per row
  norm_backward  gradients of the norm's input and weight
  linear         act(x W + b) + residual; with ``eight`` e4m3 operands with scales
  linear_backward  gradients of x, W and b
  gated          act(x Wg) * (x Wu); with ``eight`` e4m3 operands with scales
  gated_backward gradients of x, Wg and Wu
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
# the most one drawn case may cost: the largest listed ones (gated_large, norm_large_8bit)
MAX_FLOPS = 1.0e12
MAX_BYTES = 0.9e9


def listed():
    return [
        # one new row of the residual stream, normalised into 8 bits for an 8-bit product
        {"name": "norm_token_8bit", "op": "norm", "rows": 1, "c": 2048, "eight": True},
        # the outdoor scan's voxels at the convolution's width: norm after a layer's residual
        {"name": "norm_outdoor", "op": "norm", "rows": 32371, "c": 128, "eight": False},
        # a long batch of wide rows into 8 bits: the largest stream
        {"name": "norm_large_8bit", "op": "norm", "rows": 16381, "c": 8192, "eight": True},
        # training, an odd width and a ragged row count, gradient arriving on the residual as well
        {"name": "norm_backward_ragged", "op": "norm_backward", "rows": 20011, "c": 1000},
        # one row through a square projection with bias and residual: the weight is the traffic
        {"name": "linear_token", "op": "linear", "rows": 1, "c": 4096, "h": 4096, "act": "none", "bias": True,
         "residual": True, "eight": False},
        # the block's down-projection over the outdoor scan: thin and bound by memory
        {"name": "linear_outdoor", "op": "linear", "rows": 32371, "c": 512, "h": 128, "act": "none", "bias": True,
         "residual": True, "eight": False},
        # an 8-bit projection with an activation, bound by the tensor cores
        {"name": "linear_large_8bit", "op": "linear", "rows": 8192, "c": 4096, "h": 4096, "act": "gelu", "bias": True,
         "residual": False, "eight": True},
        # training a pointwise layer of the deep stage (its voxels and widths)
        {"name": "linear_backward_deep", "op": "linear_backward", "rows": 15052, "c": 512, "h": 512, "act": "silu",
         "bias": True},
        # a handful of rows through a wide feed-forward part: the two weights are the traffic
        {"name": "gated_tokens", "op": "gated", "rows": 7, "c": 2048, "h": 6000, "act": "silu", "eight": False},
        # the block's up-projections over the outdoor scan
        {"name": "gated_outdoor", "op": "gated", "rows": 32371, "c": 128, "h": 512, "act": "silu", "eight": False},
        # long batch, wide model: bound by the tensor cores
        {"name": "gated_large", "op": "gated", "rows": 7777, "c": 4096, "h": 8192, "act": "silu", "eight": False},
        # training the feed-forward part
        {"name": "gated_backward", "op": "gated_backward", "rows": 16384, "c": 1024, "h": 4096, "act": "silu"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "norm_backward", "linear", "linear", "linear_backward", "gated", "gated",
                         "gated_backward"])
        case = {"op": op, "rows": _spread(rng, 1, 131072)}
        if op in ("norm", "norm_backward"):
            case["c"] = _spread(rng, 16, 8192)
            # most networks' widths are whole vectors; the odd ones stay in
            if rng.random() < 0.7:
                case["c"] = (case["c"] + 7) // 8 * 8
            if op == "norm":
                case["eight"] = rng.random() < 0.5
        else:
            eight = op in ("linear", "gated") and rng.random() < 0.4
            if op in ("linear", "gated"):
                case["eight"] = eight
            step = 16 if eight else 8 if rng.random() < 0.85 else 1
            case["c"], case["h"] = (-(-_spread(rng, 16, 8192) // step) * step for _ in range(2))
            # gradients through the smooth activations (ReLU's gradient jumps where z is within rounding of 0)
            case["act"] = rng.choice(["silu", "gelu", "gelu_tanh"]
                                     + (["none"] if op.startswith("linear") else [])
                                     + (["relu"] if not op.endswith("backward") else []))
            if op.startswith("linear"):
                case["bias"] = rng.random() < 0.6
            if op == "linear":
                case["residual"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES:
            return case


def work(case):
    n, c = case["rows"], case["c"]
    op = case["op"]
    if op == "norm":
        # x and the residual in, the sum and y out
        return {"bytes": 6 * n * c + (n * c + 4 * n if case["eight"] else 2 * n * c) + 4 * c, "flops": 6 * n * c}
    if op == "norm_backward":
        return {"bytes": 8 * n * c + 8 * c, "flops": 12 * n * c}
    h = case["h"]
    size = 1 if case.get("eight") else 2
    if op == "linear":
        b = size * (n * c + c * h) + 2 * n * h * (2 if case["residual"] else 1) + (4 * h if case["bias"] else 0)
        return {"bytes": b + (4 * (n + h) if case["eight"] else 0), "flops": 2 * n * c * h}
    if op == "linear_backward":
        again = 0 if case["act"] == "none" else 2 * n * c * h
        return {"bytes": 2 * (2 * n * c + 2 * c * h + n * h) + (8 * h if case["bias"] else 0),
                "flops": 4 * n * c * h + again}
    if op == "gated":
        return {"bytes": size * (n * c + 2 * c * h) + 2 * n * h + (4 * (n + 2 * h) if case["eight"] else 0),
                "flops": 4 * n * c * h}
    return {"bytes": 2 * (2 * n * c + 4 * c * h + n * h), "flops": 12 * n * c * h}


def _rows_to_e4m3(v):
    """e4m3 rows of v with a 32-bit scale each."""
    scale = v.abs().amax(1) / E4M3_MAX
    return (v / scale.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    n, c, op = case["rows"], case["c"], case["op"]
    state = {"case": case}
    if op in ("norm", "norm_backward"):
        state["w"] = 1 + normal(c, std=0.2)
        # a residual stream: rows of different size, a few channels that stand out
        wide = torch.where(torch.rand(c, generator=gen, device="cuda") < 0.02, 8.0, 1.0)
        stream = normal(n, c) * wide * torch.exp(normal(n, 1, std=0.5))
        if op == "norm":
            state["x"], state["residual"] = normal(n, c).bfloat16(), stream.bfloat16()
        else:
            state["x"] = stream.bfloat16()
            state["dy"], state["dres"] = normal(n, c, std=1e-2).bfloat16(), normal(n, c, std=1e-2).bfloat16()
        return state
    h = case["h"]
    names = ["w"] if op.startswith("linear") else ["w_gate", "w_up"]
    if case.get("eight"):
        state["x"], state["x_scale"] = _rows_to_e4m3(normal(n, c))
        for k in names:   # [h, c]: the layout of quantised weights
            state[k], state[k + "_scale"] = _rows_to_e4m3(normal(h, c, std=c ** -0.5))
    else:
        state["x"] = normal(n, c).bfloat16()
        for k in names:
            state[k] = normal(c, h, std=c ** -0.5).bfloat16()
    if case.get("bias"):
        state["b"] = normal(h, std=0.1)
    if case.get("residual"):
        state["residual"] = normal(n, h).bfloat16()
    if op.endswith("backward"):
        state["dy"] = normal(n, h, std=1e-2).bfloat16()
    return state


# ---- plain forms -------------------------------------------------------------
def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _operand(s, name):
    """An operand in 32 bits; 8-bit ones as the values they stand for."""
    v = s[name].float()
    return v * s[name + "_scale"][:, None] if name + "_scale" in s else v


def _weight(s, name):
    """A weight in 32 bits as [c, h]."""
    w = _operand(s, name)
    return w.t() if name + "_scale" in s else w


def _plain(s):
    case = s["case"]
    op, x = case["op"], _operand(s, "x")
    if op == "norm":
        t = x + s["residual"].float()
        y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["w"]
        if not case["eight"]:
            return {"y": y.bfloat16(), "sum": t.bfloat16()}
        scale = y.abs().amax(1) / E4M3_MAX
        q = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y))
        return {"q": q.to(torch.float8_e4m3fn), "scale": scale, "sum": t.bfloat16()}
    if op == "norm_backward":
        dy = s["dy"].float()
        r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        g = dy * s["w"]
        dx = r * (g - x * r * r * (g * x).mean(1, keepdim=True)) + s["dres"].float()
        return {"dx": dx.bfloat16(), "dw": (dy * x * r).sum(0)}
    if op == "linear":
        z = x @ _weight(s, "w")
        if "b" in s:
            z = z + s["b"]
        y = _act(case["act"], z)
        if "residual" in s:
            y = y + s["residual"].float()
        return {"y": y.bfloat16()}
    if op == "linear_backward":
        w, dz = _weight(s, "w"), s["dy"].float()
        if case["act"] != "none":
            z = x @ w
            if "b" in s:
                z = z + s["b"]
            dz = dz * _act_grad(case["act"], z)
        out = {"dx": (dz @ w.t()).bfloat16(), "dw": (x.t() @ dz).bfloat16()}
        if "b" in s:
            out["db"] = dz.sum(0)
        return out
    wg, wu = _weight(s, "w_gate"), _weight(s, "w_up")
    g, u = x @ wg, x @ wu
    if op == "gated":
        return {"h": (_act(case["act"], g) * u).bfloat16()}
    dh = s["dy"].float()
    dg, du = dh * u * _act_grad(case["act"], g), dh * _act(case["act"], g)
    return {"dx": (dg @ wg.t() + du @ wu.t()).bfloat16(), "dw_gate": (x.t() @ dg).bfloat16(),
            "dw_up": (x.t() @ du).bfloat16()}


# ---- the package's operators -------------------------------------------------
def _own(s):
    import submanifold_sparse_convolution_gb300 as sc

    case = s["case"]
    op, x = case["op"], s["x"]
    if op == "norm":
        out = sc.rms_norm(x, s["w"], residual=s["residual"], eps=EPS, quantize=case["eight"])
        return dict(zip(("q", "scale", "sum") if case["eight"] else ("y", "sum"), out))
    if op == "norm_backward":
        dx, dw = sc.rms_norm_backward(s["dy"], x, s["w"], dres=s["dres"], eps=EPS)
        return {"dx": dx, "dw": dw}
    if op == "linear":
        return {"y": sc.linear(x, s["w"], bias=s.get("b"), activation=case["act"], residual=s.get("residual"),
                               x_scale=s.get("x_scale"), w_scale=s.get("w_scale"))}
    if op == "linear_backward":
        dx, dw, db = sc.linear_backward(s["dy"], x, s["w"], bias=s.get("b"), activation=case["act"])
        return {"dx": dx, "dw": dw} | ({} if db is None else {"db": db})
    if op == "gated":
        return {"h": sc.gated_ffn(x, s["w_gate"], s["w_up"], activation=case["act"], x_scale=s.get("x_scale"),
                                  gate_scale=s.get("w_gate_scale"), up_scale=s.get("w_up_scale"))}
    dx, dwg, dwu = sc.gated_ffn_backward(s["dy"], x, s["w_gate"], s["w_up"], activation=case["act"])
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definitions in 64 bits ----------------------------------------------
def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(8 / math.pi)   # 0.5 (1 + tanh(v / 2)) is the logistic function of v
    s = torch.sigmoid(a * z * (1 + 0.044715 * z * z))
    return z * s, s + z * s * (1 - s) * a * (1 + 0.134145 * z * z)


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    for k in ("x", "w", "w_gate", "w_up"):
        if k + "_scale" in d:
            d[k] = torch.einsum("ij,i->ij", d[k], d[k + "_scale"])
            if k != "x":
                d[k] = d[k].T
    op, x = case["op"], d["x"]
    if op == "norm":
        t = d["residual"] + x
        y = t / torch.sqrt(torch.linalg.vector_norm(t, dim=1, keepdim=True) ** 2 / case["c"] + EPS) * d["w"]
        if not case["eight"]:
            return {"y": y, "sum": t}
        scale = torch.linalg.vector_norm(y, float("inf"), dim=1) / 448
        return {"q": y / scale.clamp_min(1e-300)[:, None], "scale": scale, "sum": t}
    if op == "norm_backward":
        rms = torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / case["c"] + EPS)
        unit = x / rms
        g = d["dy"] * d["w"]
        along = torch.einsum("ij,ij->i", g, unit)[:, None] / case["c"]
        return {"dx": (g - unit * along) / rms + d["dres"], "dw": torch.einsum("ij,ij->j", d["dy"], unit)}
    if op == "linear":
        z = torch.einsum("nc,ch->nh", x, d["w"]) + d.get("b", 0.0)
        return {"y": _exact_act(case["act"], z)[0] + d.get("residual", 0.0)}
    if op == "linear_backward":
        dz = d["dy"]
        if case["act"] != "none":
            dz = dz * _exact_act(case["act"], torch.einsum("nc,ch->nh", x, d["w"]) + d.get("b", 0.0))[1]
        out = {"dx": torch.einsum("nh,ch->nc", dz, d["w"]), "dw": torch.einsum("nc,nh->ch", x, dz)}
        return out | ({"db": torch.einsum("nh->h", dz)} if "b" in d else {})
    g, u = torch.einsum("nc,ch->nh", x, d["w_gate"]), torch.einsum("nc,ch->nh", x, d["w_up"])
    a, slope = _exact_act(case["act"], g)
    if op == "gated":
        return {"h": a * u}
    dg, du = d["dy"] * slope * u, d["dy"] * a
    return {"dx": torch.einsum("nh,ch->nc", dg, d["w_gate"]) + torch.einsum("nh,ch->nc", du, d["w_up"]),
            "dw_gate": torch.einsum("nc,nh->ch", x, dg), "dw_up": torch.einsum("nc,nh->ch", x, du)}
