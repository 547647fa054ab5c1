"""Cases for group norm, rows sorted by expert, and e4m3 products with a scale for each block of 128.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, sums over rows in 64, rounded where an operator's output is) or,
where ``own`` is true, through the package's entry points.  ``exact`` gives the
same outputs from the operators' definitions in 64 bits.

A case's ``op`` is one of
  norm           act(group norm of the rows of each scan), and the statistics where ``stats``
  norm_backward  gradients of its input, weight and bias
  experts        rows sorted by expert, gathered, and brought back with their weights
  experts_backward  gradients of the gathering and of the weighted sum
  blocks         act(x W + b) + residual of e4m3 operands with block scales
  gated_blocks   act(x Wg) * (x Wu) of the same
  experts_ffn    the experts' gated feed-forward on sorted rows, in 8 bits from the rows to the down-projection's sums

Rows of no scan and of no expert are zeros; -1 is no expert.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
BLOCK = 128
# the most one drawn case may cost: the largest listed ones (experts_ffn_batch, norm_large)
MAX_FLOPS = 6e11
MAX_BYTES = 1.0e9


def listed():
    return [
        # one small scan in one pass: latency
        {"name": "norm_small_scan", "op": "norm", "rows": 3000, "c": 64, "groups": 8, "scans": 1, "act": "relu",
         "fp32": False, "stats": False, "behind": 0},
        # the outdoor scan at the convolution's width
        {"name": "norm_outdoor", "op": "norm", "rows": 32371, "c": 128, "groups": 32, "scans": 1, "act": "silu",
         "fp32": False, "stats": False, "behind": 0},
        # a batch of ragged scans in 32 bits with its statistics for training, an odd group, a padded tail
        {"name": "norm_scans_32bit", "op": "norm", "rows": 200003, "c": 60, "groups": 12, "scans": 7, "act": "gelu",
         "fp32": True, "stats": True, "behind": 1021},
        # a large batch of scans: twice the L2 cache
        {"name": "norm_large", "op": "norm", "rows": 600000, "c": 256, "groups": 32, "scans": 24, "act": "silu",
         "fp32": False, "stats": False, "behind": 0},
        # training at the deep stage's voxels and width
        {"name": "norm_backward_deep", "op": "norm_backward", "rows": 15052, "c": 512, "groups": 32, "scans": 2,
         "act": "silu", "fp32": False, "behind": 0},
        # one row to its eight experts and back
        {"name": "experts_token", "op": "experts", "tokens": 1, "k": 8, "experts": 128, "c": 2048, "fp32": False,
         "dropped": False},
        # a batch of rows to four experts each, some of them over an expert's capacity and dropped
        {"name": "experts_batch", "op": "experts", "tokens": 16381, "k": 4, "experts": 64, "c": 1024, "fp32": False,
         "dropped": True},
        # training: the gradients of both directions
        {"name": "experts_backward", "op": "experts_backward", "tokens": 8190, "k": 6, "experts": 64, "c": 2048,
         "fp32": False, "dropped": False},
        # one row through a square projection with bias and residual: the weight is the traffic
        {"name": "blocks_token", "op": "blocks", "rows": 1, "c": 4096, "h": 4096, "act": "none", "bias": True,
         "residual": True},
        # an 8-bit projection with an activation, bound by the tensor cores
        {"name": "blocks_large", "op": "blocks", "rows": 8192, "c": 4096, "h": 4096, "act": "gelu", "bias": True,
         "residual": False},
        # a few rows through their experts: the experts' weights are the traffic
        {"name": "experts_ffn_few", "op": "experts_ffn", "tokens": 16, "k": 4, "experts": 32, "c": 2048, "h": 1408,
         "act": "silu"},
        # a batch of rows through their experts
        {"name": "experts_ffn_batch", "op": "experts_ffn", "tokens": 8189, "k": 4, "experts": 32, "c": 2048, "h": 1408,
         "act": "silu"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "norm_backward", "experts", "experts_backward", "blocks", "blocks",
                         "gated_blocks", "experts_ffn", "experts_ffn"])
        smooth = ["silu", "gelu", "gelu_tanh"]
        case = {"op": op}
        if op in ("norm", "norm_backward"):
            case["rows"] = _spread(rng, 1, 600000)
            case["groups"] = rng.choice([1, 2, 4, 8, 8, 16, 32, 32, 48])
            # mostly channels in whole vectors; the odd ones stay in
            case["c"] = case["groups"] * _spread(rng, 1, 2048 // case["groups"])
            if rng.random() < 0.6:
                case["c"] = -(-case["c"] // (8 * case["groups"])) * 8 * case["groups"]
            case["scans"] = rng.choice([1, 1, 2]) if rng.random() < 0.5 else _spread(rng, 1, min(case["rows"], 2048))
            # gradients through the smooth activations (ReLU's gradient jumps where z is within rounding of 0)
            case["act"] = rng.choice(smooth + ["none"] + (["relu"] if op == "norm" else []))
            case["fp32"] = rng.random() < 0.3
            if op == "norm":
                case["stats"] = rng.random() < 0.3
            case["behind"] = rng.choice([0, 0, 0, case["rows"] // 9])
        elif op in ("experts", "experts_backward"):
            case["tokens"] = _spread(rng, 1, 65536)
            case["k"] = rng.choice([1, 2, 2, 4, 6, 8])
            case["experts"] = _spread(rng, case["k"], 256)
            case["c"] = _spread(rng, 16, 4096)
            if rng.random() < 0.8:
                case["c"] = -(-case["c"] // 8) * 8
            case["fp32"] = rng.random() < 0.2
            case["dropped"] = rng.random() < 0.3
        elif op in ("blocks", "gated_blocks"):
            case["rows"] = _spread(rng, 1, 65536)
            case["c"] = -(-_spread(rng, 64, 8192) // 16) * 16
            step = 8 if rng.random() < 0.8 else 1
            case["h"] = -(-_spread(rng, 16, 8192) // step) * step
            case["act"] = rng.choice(smooth + (["none", "none", "relu"] if op == "blocks" else ["relu"]))
            if op == "blocks":
                case["bias"], case["residual"] = rng.random() < 0.5, rng.random() < 0.5
        else:
            case["tokens"] = _spread(rng, 1, 16384)
            case["k"] = rng.choice([1, 2, 4, 4, 8])
            case["experts"] = _spread(rng, max(4, case["k"]), 128)
            case["c"] = -(-_spread(rng, 128, 4096) // 16) * 16
            case["h"] = -(-_spread(rng, 128, 4096) // 16) * 16
            case["act"] = rng.choice(smooth)
            if 3 * case["experts"] * case["c"] * case["h"] > 5e8:
                continue
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES:
            return case


def _blocks(v):
    return -(-v // BLOCK)


def work(case):
    op, c = case["op"], case["c"]
    size = 4 if case.get("fp32") else 2
    if op == "norm":
        n = case["rows"]
        return {"bytes": 2 * size * n * c + 8 * c + (8 * case["scans"] * case["groups"] if case["stats"] else 0),
                "flops": 10 * n * c}
    if op == "norm_backward":
        n = case["rows"]
        return {"bytes": 3 * size * n * c + 16 * c + 8 * case["scans"] * case["groups"], "flops": 20 * n * c}
    if op in ("experts", "experts_backward"):
        t, k = case["tokens"], case["k"]
        if op == "experts":
            # indices, places and weights; x in, the sorted rows out; the experts' rows in, their sums out
            return {"bytes": 24 * t * k + size * c * (2 * t + 2 * t * k), "flops": 2 * t * k * c}
        # the sums' gradient and the experts' rows in, their gradient out; the gathered rows' gradient in, x's out
        return {"bytes": 12 * t * k + size * c * (2 * t + 3 * t * k), "flops": 5 * t * k * c}
    h = case["h"]
    if op in ("blocks", "gated_blocks"):
        n, weights = case["rows"], 2 if op == "gated_blocks" else 1
        b = n * c + weights * c * h + 4 * n * _blocks(c) + 4 * weights * _blocks(c) * _blocks(h) + 2 * n * h
        b += (4 * h if case.get("bias") else 0) + (2 * n * h if case.get("residual") else 0)
        return {"bytes": b, "flops": 2 * weights * n * c * h}
    # x in, the sum out, and the weights of the experts that some row goes to
    t, k = case["tokens"], case["k"]
    reached = min(case["experts"], t * k)
    return {"bytes": 4 * t * c + 8 * t * k + reached * (3 * c * h + 12 * _blocks(c) * _blocks(h)), "flops": 6 * t * k * c * h}


def _rows_in_blocks(v):
    """e4m3 rows of v [n, c] and fp32 scales [blocks, n], one for each 128 values of a row."""
    n, c = v.shape
    b = torch.nn.functional.pad(v.float(), (0, _blocks(c) * BLOCK - c)).view(n, -1, BLOCK)
    most = b.abs().amax(2)
    # (by a tensor: a division by a number becomes a product with its inverse, and bf16
    # values often lie halfway between two e4m3 ones, where the scale's last bit decides)
    scale = most / torch.full_like(most, E4M3_MAX)
    q = torch.where(scale[:, :, None] > 0, b / scale[:, :, None], torch.zeros_like(b))
    return q.reshape(n, -1)[:, :c].to(torch.float8_e4m3fn).contiguous(), scale.t().contiguous()


def _weight_in_blocks(w):
    """e4m3 of w [e, h, c] and fp32 scales [e, h blocks, c blocks], one for each 128 x 128 values."""
    e, h, c = w.shape
    b = torch.nn.functional.pad(w, (0, _blocks(c) * BLOCK - c, 0, _blocks(h) * BLOCK - h))
    b = b.view(e, _blocks(h), BLOCK, _blocks(c), BLOCK)
    scale = b.abs().amax((2, 4)) / E4M3_MAX
    q = (b / scale.clamp_min(1e-30)[:, :, None, :, None]).reshape(e, _blocks(h) * BLOCK, -1)
    return q[:, :h, :c].to(torch.float8_e4m3fn).contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    op, c = case["op"], case["c"]
    dtype = torch.float32 if case.get("fp32") else torch.bfloat16
    state = {"case": case}
    if op in ("norm", "norm_backward"):
        n, live = case["rows"], case["rows"] - case["behind"]
        # features after a convolution: channels of their own mean and size, rows of different size
        x = normal(n, c) * torch.exp(normal(n, 1, std=0.3)) * torch.exp(normal(c, std=0.5)) + normal(c, std=0.7)
        state["x"] = x.to(dtype)
        state["w"], state["b"] = 1 + normal(c, std=0.2), normal(c, std=0.2)
        # ragged scans; of many short ones some are empty
        cuts = (uniform(case["scans"] - 1) * (live + 1)).int().clamp_max(live).sort()[0]
        ends = torch.tensor([0, live], dtype=torch.int32, device="cuda")
        state["offsets"] = torch.cat((ends[:1], cuts, ends[1:]))
        if op == "norm_backward":
            state["dy"] = normal(n, c, std=1e-2).to(dtype)
            state["stats"] = _statistics(state)
        return state
    if op in ("blocks", "gated_blocks"):
        n, h = case["rows"], case["h"]
        state["x"], state["x_scale"] = _rows_in_blocks(normal(n, c) * torch.exp(normal(n, 1, std=0.5)))
        for k in ["w"] if op == "blocks" else ["w_gate", "w_up"]:
            q, scale = _weight_in_blocks(normal(1, h, c, std=c ** -0.5))
            state[k], state[k + "_scale"] = q[0], scale[0]
        if case.get("bias"):
            state["b"] = normal(h, std=0.1)
        if case.get("residual"):
            state["residual"] = normal(n, h).bfloat16()
        return state
    t, k, e = case["tokens"], case["k"], case["experts"]
    # a router's choice: some experts are preferred, no expert twice in a row
    score = normal(t, e) + normal(e, std=0.5)
    top, chosen = score.topk(k, dim=1)
    state["experts"], state["weights"] = chosen.int(), torch.softmax(top, 1)
    if case.get("dropped"):
        state["experts"] = torch.where(uniform(t, k) < 0.05, -1, state["experts"])
    if op == "experts_ffn":
        h = case["h"]
        state["x"] = normal(t, c).bfloat16()
        for name, shape in (("w_gate", (e, h, c)), ("w_up", (e, h, c)), ("w_down", (e, c, h))):
            state[name], state[name + "_scale"] = _weight_in_blocks(normal(*shape, std=shape[2] ** -0.5))
        # room for one expert's rows in the plain form's padded batch
        state["most"] = int(torch.bincount(chosen.reshape(-1), minlength=e).max())
        return state
    state["x"] = normal(t, c).to(dtype)
    state["y"] = normal(t * k, c).to(dtype)   # what the experts gave
    if op == "experts_backward":
        state["dout"], state["dy"] = normal(t, c, std=1e-2).to(dtype), normal(t * k, c, std=1e-2).to(dtype)
        # what the forward pass left: where each row went
        state["placed"] = _sorted(state["experts"], e)
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
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _sums(v, offsets):
    """Sums of the rows of each scan, in 64 bits."""
    total = torch.nn.functional.pad(v.double().cumsum(0), (0, 0, 1, 0))
    at = offsets.long()
    return total[at[1:]] - total[at[:-1]]


def _scan_of_rows(s):
    """The scan of each row (the last one's for the rows behind it), and whether it has one."""
    row = torch.arange(s["x"].shape[0], device="cuda", dtype=torch.int32)
    scan = torch.searchsorted(s["offsets"][1:], row, right=True)
    return scan.clamp_max(s["case"]["scans"] - 1), (row < s["offsets"][-1])[:, None]


def _statistics(s):
    """fp32 [scans, groups, 2]: mean and 1 / sqrt(variance + eps)."""
    n, c, g = s["x"].shape[0], s["case"]["c"], s["case"]["groups"]
    x, (scan, live) = s["x"].float(), _scan_of_rows(s)
    count = (s["offsets"][1:] - s["offsets"][:-1]).clamp_min(1)[:, None] * float(c // g)
    mean = _sums(x.view(n, g, -1).sum(2), s["offsets"]) / count
    d = x.view(n, g, -1) - mean.float()[scan][:, :, None]
    var = _sums((d * d).sum(2) * live, s["offsets"]) / count
    return torch.stack((mean.float(), torch.rsqrt(var.float() + EPS)), 2)


def _normalised(s, stats):
    n, c, g = s["x"].shape[0], s["case"]["c"], s["case"]["groups"]
    scan, live = _scan_of_rows(s)
    of_row = stats[scan]
    x = s["x"].float().view(n, g, -1)
    return ((x - of_row[:, :, :1]) * of_row[:, :, 1:]).view(n, c), of_row[:, :, 1], scan, live


def _sorted(experts, e):
    """offsets [e + 1], the pair of each sorted row (-1 behind the last) and the row of each pair (-1: none)."""
    flat = experts.reshape(-1)
    hit = flat[:, None] == torch.arange(e, device="cuda", dtype=torch.int32)
    order = hit.int().cumsum(0, dtype=torch.int32)
    offsets = torch.nn.functional.pad(order[-1].cumsum(0, dtype=torch.int32), (1, 0))
    rank = (order * hit).sum(1, dtype=torch.int32) - 1
    slots = torch.where(flat >= 0, offsets[flat.clamp_min(0).long()] + rank, -1)
    pairs = torch.full_like(flat, -1)
    place = torch.where(slots >= 0, slots, flat.numel()).long()
    pair = torch.arange(flat.numel(), device="cuda", dtype=torch.int32)
    pairs = torch.nn.functional.pad(pairs, (0, 1)).scatter(0, place, pair)[:-1]
    return offsets, pairs, slots.view(experts.shape)


def _gathered(x, pairs, k):
    rows = x[(pairs.clamp_min(0) // k).long()]
    return torch.where(pairs[:, None] >= 0, rows, torch.zeros_like(rows))


def _brought_back(y, slots, weights=None):
    """sum_j weights_j y[slots_j] in 32 bits."""
    part = y[slots.clamp_min(0).long()].float()
    if weights is not None:
        part = part * weights[:, :, None]
    return torch.where(slots[:, :, None] >= 0, part, torch.zeros_like(part)).sum(1)


def _row_values(q, scale):
    return q.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _weight_values(q, scale):
    """[.., c, h] of a weight [.., h, c]."""
    full = scale.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)
    return (q.float() * full[..., :q.shape[-2], :q.shape[-1]]).transpose(-1, -2)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        stats = _statistics(s)
        unit, _, _, live = _normalised(s, stats)
        y = _act(case["act"], unit * s["w"] + s["b"])
        out = {"y": torch.where(live, y, torch.zeros_like(y)).to(s["x"].dtype)}
        return out | ({"stats": stats} if case["stats"] else {})
    if op == "norm_backward":
        n, c, g = case["rows"], case["c"], case["groups"]
        unit, scale, scan, live = _normalised(s, s["stats"])
        dz = s["dy"].float() * _act_grad(case["act"], unit * s["w"] + s["b"])
        dz = torch.where(live, dz, torch.zeros_like(dz))
        dw = torch.where(live, dz * unit, torch.zeros_like(dz))
        p = dz * s["w"]
        count = (s["offsets"][1:] - s["offsets"][:-1]).clamp_min(1)[:, None] * float(c // g)
        mean_p, mean_pu = ((_sums(v.view(n, g, -1).sum(2), s["offsets"]) / count).float()[scan][:, :, None]
                           for v in (p, dw * s["w"]))
        dx = scale[:, :, None] * (p.view(n, g, -1) - mean_p - unit.view(n, g, -1) * mean_pu)
        dx = torch.where(live, dx.view(n, c), torch.zeros_like(dz))
        return {"dx": dx.to(s["x"].dtype), "dw": dw.double().sum(0).float(), "db": dz.double().sum(0).float()}
    if op == "experts":
        offsets, pairs, slots = _sorted(s["experts"], case["experts"])
        return {"offsets": offsets, "pairs": pairs, "slots": slots, "rows": _gathered(s["x"], pairs, case["k"]),
                "sum": _brought_back(s["y"], slots, s["weights"]).to(s["x"].dtype)}
    if op == "experts_backward":
        _, pairs, slots = s["placed"]
        dout = _gathered(s["dout"], pairs, case["k"]).float()
        weight = torch.where(pairs >= 0, s["weights"].reshape(-1)[pairs.clamp_min(0).long()], 0.0)
        along = (dout * s["y"].float()).sum(1)[slots.clamp_min(0).long()]
        return {"dy": (dout * weight[:, None]).to(s["y"].dtype), "dweights": torch.where(slots >= 0, along, 0.0),
                "dx": _brought_back(s["dy"], slots).to(s["x"].dtype)}
    if op == "blocks":
        z = _row_values(s["x"], s["x_scale"]) @ _weight_values(s["w"], s["w_scale"])
        if "b" in s:
            z = z + s["b"]
        y = _act(case["act"], z)
        if "residual" in s:
            y = y + s["residual"].float()
        return {"y": y.bfloat16()}
    if op == "gated_blocks":
        x = _row_values(s["x"], s["x_scale"])
        g, u = (x @ _weight_values(s[k], s[k + "_scale"]) for k in ("w_gate", "w_up"))
        return {"h": (_act(case["act"], g) * u).bfloat16()}
    offsets, pairs, slots = _sorted(s["experts"], case["experts"])
    expert = s["experts"].reshape(-1)[pairs.long()].long()   # (none is dropped here)
    place = torch.arange(pairs.numel(), device="cuda") - offsets[expert]

    def product(rows, name):
        """Sorted rows times their experts' weights, as one padded batch."""
        batch = rows.new_zeros(case["experts"], s["most"], rows.shape[1])
        batch[expert, place] = rows
        return torch.bmm(batch, _weight_values(s[name], s[name + "_scale"]))[expert, place]

    rows = _row_values(*_rows_in_blocks(_gathered(s["x"], pairs, case["k"])))
    h = _act(case["act"], product(rows, "w_gate")) * product(rows, "w_up")
    y = product(_row_values(*_rows_in_blocks(h)), "w_down").bfloat16()
    return {"sum": (s["x"].float() + _brought_back(y, slots, s["weights"])).bfloat16()}


# ---- the package's operators -------------------------------------------------
def _own(s):
    import submanifold_sparse_convolution_gb300 as sc

    case = s["case"]
    op = case["op"]
    if op == "norm":
        out = sc.group_norm(s["x"], s["w"], s["b"], case["groups"], offsets=s["offsets"], activation=case["act"], eps=EPS,
                            stats=case["stats"])
        return {"y": out[0], "stats": out[1]} if case["stats"] else {"y": out}
    if op == "norm_backward":
        dx, dw, db = sc.group_norm_backward(s["dy"], s["x"], s["w"], s["b"], case["groups"], s["stats"],
                                            offsets=s["offsets"], activation=case["act"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "experts":
        plan = sc.expert_plan(s["experts"], case["experts"])
        return {"offsets": plan.offsets, "pairs": plan.pairs, "slots": plan.slots, "rows": sc.expert_gather(s["x"], plan),
                "sum": sc.expert_combine(s["y"], plan, s["weights"])}
    if op == "experts_backward":
        plan = sc.ExpertPlan(*s["placed"])
        dy, dweights = sc.expert_combine_backward(s["dout"], s["y"], plan, s["weights"])
        return {"dy": dy, "dweights": dweights, "dx": sc.expert_gather_backward(s["dy"], plan)}
    if op == "blocks":
        return {"y": sc.linear_blocks(s["x"], s["w"], s["x_scale"], s["w_scale"], bias=s.get("b"), activation=case["act"],
                                      residual=s.get("residual"))}
    if op == "gated_blocks":
        return {"h": sc.gated_ffn_blocks(s["x"], s["w_gate"], s["w_up"], s["x_scale"], s["w_gate_scale"], s["w_up_scale"],
                                         activation=case["act"])}
    plan = sc.expert_plan(s["experts"], case["experts"])
    q, scale = sc.expert_gather(s["x"], plan, quantize=True)
    q, scale = sc.gated_ffn_blocks(q, s["w_gate"], s["w_up"], scale, s["w_gate_scale"], s["w_up_scale"],
                                   offsets=plan.offsets, activation=case["act"], quantize=True)
    y = sc.linear_blocks(q, s["w_down"], scale, s["w_down_scale"], offsets=plan.offsets)
    return {"sum": sc.expert_combine(y, plan, s["weights"], residual=s["x"])}


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


def _exact_norm(s):
    """Scan by scan; the backward pass from the statistics it is given."""
    case = s["case"]
    g, w, b = case["groups"], s["w"].double(), s["b"].double()
    at = s["offsets"].tolist()
    back = case["op"] == "norm_backward"
    first = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    stats = torch.zeros(case["scans"], g, 2, dtype=torch.float64, device="cuda")
    stats[:, :, 1] = EPS ** -0.5
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    for i, (lo, hi) in enumerate(zip(at, at[1:])):
        if lo == hi:
            continue
        v = s["x"][lo:hi].double().unflatten(1, (g, -1))
        if back:
            mean, r = s["stats"][i].double().unbind(1)
        else:
            var, mean = torch.var_mean(v, dim=(0, 2), correction=0)
            r = 1 / torch.sqrt(var + EPS)
            stats[i] = torch.stack((mean, r), 1)
        unit = torch.einsum("ngd,g->ngd", v - mean[None, :, None], r).flatten(1)
        a, slope = _exact_act(case["act"], unit * w + b)
        if not back:
            first[lo:hi] = a
            continue
        dz = s["dy"][lo:hi].double() * slope
        dw += torch.einsum("nc,nc->c", dz, unit)
        db += torch.einsum("nc->c", dz)
        p, u = (dz * w).unflatten(1, (g, -1)), unit.unflatten(1, (g, -1))
        m = float(p[:, 0].numel())
        along = torch.einsum("ngd,ngd->g", p, u) / m
        dx = p - torch.einsum("ngd->g", p)[None, :, None] / m - u * along[None, :, None]
        first[lo:hi] = torch.einsum("ngd,g->ngd", dx, r).flatten(1)
    if back:
        return {"dx": first, "dw": dw, "db": db}
    return {"y": first} | ({"stats": stats} if case["stats"] else {})


def _exact_rows(q, scale):
    v = q.double()
    for i in range(scale.shape[0]):
        v[:, i * BLOCK:(i + 1) * BLOCK] *= scale[i].double()[:, None]
    return v


def _exact_weight(q, scale):
    h, c = q.shape
    index = [torch.arange(m, device="cuda") // BLOCK for m in (h, c)]
    return q.double() * scale.double()[index[0]][:, index[1]]


def _exact_in_blocks(v):
    """The values that v's e4m3 blocks stand for: scales are held in 32 bits."""
    out = torch.zeros_like(v)
    for i in range(0, v.shape[1], BLOCK):
        part = v[:, i:i + BLOCK]
        scale = (torch.linalg.vector_norm(part, float("inf"), dim=1) / E4M3_MAX).float().double()[:, None]
        q = (part / scale.clamp_min(1e-300)).clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)
        out[:, i:i + BLOCK] = q.double() * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        return _exact_norm(s)
    if op in ("blocks", "gated_blocks"):
        x = _exact_rows(s["x"], s["x_scale"])
        if op == "gated_blocks":
            g, u = (torch.einsum("nc,hc->nh", x, _exact_weight(s[k], s[k + "_scale"])) for k in ("w_gate", "w_up"))
            return {"h": _exact_act(case["act"], g)[0] * u}
        z = torch.einsum("nc,hc->nh", x, _exact_weight(s["w"], s["w_scale"]))
        if "b" in s:
            z = z + s["b"].double()
        return {"y": _exact_act(case["act"], z)[0] + (s["residual"].double() if "residual" in s else 0.0)}
    t, k, e = case["tokens"], case["k"], case["experts"]
    flat = s["experts"].flatten().long()
    key = torch.where(flat < 0, e, flat)
    order = torch.sort(key, stable=True)[1]
    live = int((flat >= 0).sum())
    order = order[:live]
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(e + 1, device="cuda"))
    slots = torch.full((t * k,), -1, dtype=torch.int64, device="cuda")
    slots[order] = torch.arange(live, device="cuda")
    token, weights = order // k, s["weights"].double().flatten()

    def add_up(rows):
        """The live sorted rows added to their tokens, one choice after the other."""
        out = torch.zeros(t, rows.shape[1], dtype=torch.float64, device="cuda")
        for j in range(k):
            sel = (order % k == j).nonzero()[:, 0]
            out[token[sel]] += rows[sel]
        return out

    if op == "experts":
        rows = torch.zeros(t * k, case["c"], dtype=torch.float64, device="cuda")
        rows[:live] = s["x"].double()[token]
        return {"offsets": offsets.int(), "pairs": torch.nn.functional.pad(order, (0, t * k - live), value=-1).int(),
                "slots": slots.view(t, k).int(), "rows": rows,
                "sum": add_up(s["y"][:live].double() * weights[order][:, None])}
    if op == "experts_backward":
        dout, dy = s["dout"].double()[token], torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        dy[:live] = dout * weights[order][:, None]
        dweights = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        dweights[order] = torch.einsum("nc,nc->n", dout, s["y"][:live].double())
        return {"dy": dy, "dweights": dweights.view(t, k), "dx": add_up(s["dy"][:live].double())}
    x = _exact_in_blocks(s["x"].double())
    y = torch.zeros(t * k, case["c"], dtype=torch.float64, device="cuda")
    at = offsets.tolist()
    for i in range(e):
        lo, hi = at[i], at[i + 1]
        if lo == hi:
            continue
        g, u, down = (_exact_weight(s[n][i], s[n + "_scale"][i]) for n in ("w_gate", "w_up", "w_down"))
        rows = x[token[lo:hi]]
        h = _exact_act(case["act"], rows @ g.T)[0] * (rows @ u.T)
        y[lo:hi] = _exact_in_blocks(h) @ down.T
    return {"sum": s["x"].double() + add_up(y * weights[order][:, None])}
