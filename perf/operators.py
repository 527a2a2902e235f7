"""The microscaled 4-bit operators and the router's balance loss, as cases to be timed.

Four operators, measured in three kinds of case:

- ``storage``: rows are quantised to MXFP4 (blocks of 32 values along the row, e2m1 codes, one
  power-of-two scale a block) and read back, so that a pass returns the values the codes stand for;
- ``experts``: the product of routed rows with MXFP4 expert weights, in the two places where an MoE
  layer has it (gate/up with SwiGLU, down with the routing weights) and for one dense matrix;
- ``balance``: the router's balance and z losses with the per-expert counts, forward and backward.

``run`` computes them with elementary torch operations, or with the library's calls where ``own``
is true.
"""
import math

import torch

own = False

BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the eight e2m1 codes
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def storage_case(rows, cols, kind):
    return {"op": "storage", "rows": rows, "cols": cols, "in": kind}


def experts_case(tokens, experts, top_k, n, k, x, y, place, skew):
    """place: "gateup" (rows gathered by token, SwiGLU, n = gate and up rows), "down" (rows in expert
    order, routing weights, one output row an assignment) or "dense" (one expert, every row)."""
    return {"op": "experts", "tokens": tokens, "experts": experts, "top_k": top_k, "n": n, "k": k, "x": x, "y": y,
            "place": place, "skew": skew}


def balance_case(tokens, experts, top_k, kind, padded):
    return {"op": "balance", "tokens": tokens, "experts": experts, "top_k": top_k, "in": kind, "padded": padded}


def listed():
    cases = {
        # Eight decoded tokens' activations on their way into a 4-bit product: launch latency.
        "storage 8 tokens": storage_case(8, 2048, "bf16"),
        # A whole stack of 256 gate matrices converted when a checkpoint is loaded.
        "storage weight stack": storage_case(256 * 512, 2048, "bf16"),
        # One decoded token through its eight experts' gate and up matrices: weights read once.
        "gateup 1 token": experts_case(1, 256, 8, 1024, 2048, "bf16", "bf16", "gateup", False),
        # The down product of eight tokens decoded together, weighted, as float rows to be summed.
        "down 8 tokens": experts_case(8, 256, 8, 2048, 512, "bf16", "f32", "down", False),
        # A short prompt, near-uniform routing: 16 rows an expert on average, every expert active.
        "gateup 512 tokens": experts_case(512, 256, 8, 1024, 2048, "bf16", "bf16", "gateup", False),
        # A long prompt with skewed routing (0 to thousands of rows an expert), 4-bit on both sides,
        # the intermediate quantised for the down product in the same call.
        "gateup 4096 tokens 4-bit": experts_case(4096, 256, 8, 1024, 2048, "mx4", "mx4", "gateup", True),
        # The down product that follows it.
        "down 4096 tokens 4-bit": experts_case(4096, 256, 8, 2048, 512, "mx4", "bf16", "down", True),
        # A ragged prompt through one dense matrix with bf16 activations.
        "dense 2085 rows": experts_case(2085, 1, 1, 4096, 2048, "bf16", "bf16", "dense", False),
        # The layer's largest widths, 4-bit on both sides: bound by the matrix units.
        "dense 4096 rows wide 4-bit": experts_case(4096, 1, 1, 8192, 8192, "mx4", "bf16", "dense", False),
        # A small layer's router in a small batch: launch latency.
        "balance 64 tokens": balance_case(64, 16, 2, "f32", False),
        # One padded training batch of the full-size router.
        "balance 4096 tokens": balance_case(4096, 256, 8, "f32", True),
        # The largest router over a large packed batch in bf16.
        "balance 65536 tokens": balance_case(65536, 512, 16, "bf16", True),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["storage", "experts", "experts", "experts", "balance"])
    if op == "storage":
        cols = BLOCK * _log(rng, 1, 256)
        rows = _log(rng, 1, min(1 << 20, 256 * 512 * 2048 // cols))
        return storage_case(rows, cols, rng.choice(["bf16", "f32"]))
    if op == "balance":
        experts = _log(rng, 2, 512)
        return balance_case(_log(rng, 1, 65536), experts, rng.randint(1, min(16, experts)), rng.choice(["bf16", "f32"]),
                            rng.random() < 0.5)
    place = rng.choice(["gateup", "down", "dense"])
    x, y = rng.choice(["bf16", "mx4"]), rng.choice(["f32", "bf16"])
    if place == "dense":
        return experts_case(_log(rng, 1, 4096), 1, 1, _log(rng, 32, 8192), BLOCK * _log(rng, 1, 256), x, y, place, False)
    experts = _log(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    hidden, inter = BLOCK * _log(rng, 2, 64), BLOCK * _log(rng, 1, 16)
    tokens = _log(rng, 1, 4096)
    skew = rng.random() < 0.5
    if place == "gateup":
        return experts_case(tokens, experts, top_k, 2 * inter, hidden, x, rng.choice([y, "mx4"]), place, skew)
    # The output width is free: an odd one now and then.
    return experts_case(tokens, experts, top_k, hidden - rng.choice([0, 0, 1, 24]), inter, x, y, place, skew)


# ---- inputs ------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "storage":
        # Rows of different magnitude, as activations and weight rows have.
        x = randn(case["rows"], case["cols"])
        x *= torch.exp(randn(case["rows"], 1))
        return {"case": case, "x": x.to(TYPES[case["in"]])}

    T, E, k = case["tokens"], case["experts"], case["top_k"]
    if case["op"] == "balance":
        logits = (1.5 * randn(T, E) + randn(E)).to(TYPES[case["in"]])
        ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
        valid = None
        if case["padded"]:
            valid = (torch.rand(T, generator=g, device="cuda") < 0.85).to(torch.uint8)
        return {"case": case, "logits": logits, "ids": ids, "valid": valid, "coefs": (0.01, 0.001),
                "grad": torch.full((1,), 1.0, device="cuda") + 0.25 * randn(1)}

    n, K = case["n"], case["k"]
    logits = randn(T, E)
    if case["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1
        logits -= 1.1 * torch.log(rank)
    top = torch.topk(logits, k, dim=1)
    flat = top.indices.flatten()
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    w_codes, w_scales = to_mx4(randn(E * n, K).mul_(0.02))
    state = {"case": case, "w_codes": w_codes.view(E, n, K // 2), "w_scales": w_scales.view(E, n, K // BLOCK),
             "offsets": offsets, "assign": order.to(torch.int32), "weights": torch.softmax(top.values, 1).flatten(),
             "x_scales": None}
    x = randn(T * k if case["place"] == "down" else T, K)
    if case["x"] == "mx4":
        state["x"], state["x_scales"] = to_mx4(x)
    else:
        state["x"] = x.to(torch.bfloat16)
    return state


# ---- the plain form ----------------------------------------------------------------------------


def to_mx4(v):
    """[R, C] numbers -> codes [R, C/2] (the even column in the low nibble) and scale bytes [R, C/32].

    The scale is 2^(floor(log2 amax) - 2), at least 2^-127; a code is the nearest e2m1 value, ties to
    the even one, magnitudes above 6 held at 6."""
    v = v.float().view(v.shape[0], -1, BLOCK)
    power = torch.frexp(v.abs().amax(2)).exponent - 3  # frexp's mantissa is in [0.5, 1)
    power = torch.where(v.abs().amax(2) > 0, power, -127).clamp(min=-127)
    m = torch.ldexp(v.abs(), -power[..., None])
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(v.shape[0], -1)
    return code[:, ::2] | (code[:, 1::2] << 4), (power + 127).to(torch.uint8)


def from_mx4(codes, scales):
    """The values of to_mx4's codes and scales, any leading dimensions."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).long()
    values = table[both].view(*scales.shape, BLOCK)
    return torch.ldexp(values, (scales.to(torch.int32) - 127)[..., None]).flatten(-2)


def plain_experts(s):
    c = s["case"]
    offsets, assign, k = s["offsets"].long(), s["assign"].long(), c["top_k"]
    E, rows = c["experts"], s["assign"].numel()
    x = s["x"].float() if s["x_scales"] is None else from_mx4(s["x"], s["x_scales"])
    if c["place"] == "gateup":
        x = x[assign // k]
    expert = torch.searchsorted(offsets[1:], torch.arange(rows, device=x.device), right=True)
    if rows <= E:  # few rows: each with its own expert's matrix
        z = torch.bmm(from_mx4(s["w_codes"][expert], s["w_scales"][expert]), x[:, :, None])[:, :, 0]
    else:  # every expert's rows side by side, up to the largest number that one may have
        slot = torch.arange(rows, device=x.device) - offsets[expert]
        wide = x.new_zeros(E, c["tokens"], c["k"])
        wide[expert, slot] = x
        z = torch.bmm(wide, from_mx4(s["w_codes"], s["w_scales"]).transpose(1, 2).contiguous())[expert, slot]
    if c["place"] == "gateup":
        gate, up = z.chunk(2, 1)
        z = gate / (1 + torch.exp(-gate)) * up
    if c["place"] == "down":
        out = torch.empty_like(z)
        out[assign] = z * s["weights"][assign][:, None]
        z = out
    if c["y"] == "mx4":
        return from_mx4(*to_mx4(z)).to(torch.bfloat16)
    return z.to(TYPES[c["y"]])


def plain_balance(s):
    c = s["case"]
    E, k = c["experts"], c["top_k"]
    balance_coef, z_coef = s["coefs"]
    logits = s["logits"].float()
    valid = torch.ones(len(logits), device=logits.device) if s["valid"] is None else s["valid"].float()
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = (top + torch.log(total))[:, 0]
    # The sums over tokens are long: taken in 64 bits.
    n = valid.double().sum().clamp(min=1)
    chosen = torch.zeros(E, dtype=torch.int32, device=logits.device)
    chosen.index_add_(0, s["ids"].flatten().long(), valid.to(torch.int32).repeat_interleave(k))
    mean_prob = (p * valid[:, None]).double().sum(0) / n
    share = chosen.double() / (n * k)
    balance = E * (share * mean_prob).sum()
    z = (lse.double().square() * valid).sum() / n
    losses = torch.stack((balance_coef * balance + z_coef * z, balance, z)).float()
    f = share.float()
    slope = balance_coef * E * (f - (p * f).sum(1, keepdim=True)) + 2 * z_coef * lse[:, None]
    dlogits = p * slope * (valid[:, None] * s["grad"] / n.float())
    return {"losses": losses, "counts": chosen, "mean_prob": mean_prob.float(), "dlogits": dlogits.to(s["logits"].dtype)}


# ---- the library's calls -----------------------------------------------------------------------


def own_storage(s):
    import bit_quantized_moe_router_amd as moe

    x = s["x"]
    rows, cols = x.shape
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, cols // BLOCK, dtype=torch.uint8, device=x.device)
    y = torch.empty_like(x)
    moe.moe_mx4_quantize(x, codes, scales)
    moe.moe_mx4_dequantize(codes, scales, y)
    return y


def own_experts(s):
    import bit_quantized_moe_router_amd as moe

    c, x = s["case"], s["x"]
    kinds = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "mx4": moe.MOE_MX4}
    gateup, down = c["place"] == "gateup", c["place"] == "down"
    desc = moe.make_mx4_desc(c["experts"], c["n"], c["k"], kinds[c["x"]], kinds[c["y"]], swiglu=int(gateup))
    rows, width = s["assign"].numel(), c["n"] // 2 if gateup else c["n"]
    y_scales = None
    if c["y"] == "mx4":
        y = torch.empty(rows, width // 2, dtype=torch.uint8, device=x.device)
        y_scales = torch.empty(rows, width // BLOCK, dtype=torch.uint8, device=x.device)
    else:
        y = torch.empty(rows, width, dtype=TYPES[c["y"]], device=x.device)
    moe.moe_mx4_experts(desc, s["w_codes"], s["w_scales"], x, s["x_scales"], s["offsets"], rows, y, y_scales,
                        src_rows=s["assign"] if gateup else None, src_div=c["top_k"] if gateup else 1,
                        dst_rows=s["assign"] if down else None, row_scale=s["weights"] if down else None)
    if y_scales is None:
        return y
    values = torch.empty(rows, width, dtype=torch.bfloat16, device=x.device)
    moe.moe_mx4_dequantize(y, y_scales, values)
    return values


def own_balance(s):
    import bit_quantized_moe_router_amd as moe

    logits, ids, valid = s["logits"], s["ids"], s["valid"]
    T, E = logits.shape
    dev = logits.device
    losses, mean_prob = torch.empty(3, device=dev), torch.empty(E, device=dev)
    counts, n_valid = (torch.empty(m, dtype=torch.int32, device=dev) for m in (E, 1))
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device=dev)
    dlogits = torch.empty_like(logits)
    moe.moe_balance_loss_forward(logits, ids, valid, *s["coefs"], losses, counts, mean_prob, n_valid, ws)
    moe.moe_balance_loss_backward(logits, ids.shape[1], valid, *s["coefs"], counts, n_valid, s["grad"], dlogits)
    return {"losses": losses, "counts": counts, "mean_prob": mean_prob, "dlogits": dlogits}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"storage": own_storage, "experts": own_experts, "balance": own_balance}[op](state)
    if op == "storage":
        return from_mx4(*to_mx4(state["x"])).to(state["x"].dtype)
    return plain_experts(state) if op == "experts" else plain_balance(state)


# ---- what a pass cannot do without -------------------------------------------------------------


def active_experts(tokens, experts, top_k, skew):
    """Experts that get a row, in one draw of prepare()'s routing."""
    g = torch.Generator().manual_seed(0)
    logits = torch.randn(tokens, experts, generator=g)
    if skew:
        logits -= 1.1 * torch.log(torch.arange(experts) + 1.0)
    return torch.topk(logits, top_k, dim=1).indices.unique().numel()


def work(case):
    if case["op"] == "storage":
        values = case["rows"] * case["cols"]
        size = {"f32": 4, "bf16": 2}[case["in"]]
        # x in, codes and scales out and in again, the values out.
        return {"bytes": values * (2 * size + 2 * 17 / 32), "flops": 4 * values}
    if case["op"] == "balance":
        cells = case["tokens"] * case["experts"]
        size = {"f32": 4, "bf16": 2}[case["in"]]
        # Forward and backward each read the logits; the backward writes their gradient.
        return {"bytes": 3 * cells * size + 4 * case["tokens"] * case["top_k"] + 16 * case["experts"], "flops": 16 * cells}
    T, E, k, n, K = (case[name] for name in ("tokens", "experts", "top_k", "n", "k"))
    rows = T * k
    active = active_experts(T, E, k, case["skew"])
    row = {"bf16": 2, "mx4": 17 / 32, "f32": 4}
    x_rows = rows if case["place"] == "down" else T
    width = n // 2 if case["place"] == "gateup" else n
    moved = active * n * K * row["mx4"] + x_rows * K * row[case["x"]] + rows * width * row[case["y"]] + 8 * rows
    if case["y"] == "mx4":  # read back as values
        moved += rows * width * (row["mx4"] + 2)
    return {"bytes": moved, "flops": 2 * rows * n * K}


# ---- the definition in 64 bits -----------------------------------------------------------------


def exact_grid(v):
    """float64 [..., 32] -> the e2m1 value nearest to each under its block's scale, times that scale."""
    amax = v.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(amax.clamp(min=2.0 ** -126))) - 2).clamp(min=-127))
    # log2 may round up to a whole number just below a power of two.
    scale = torch.where((amax < 4 * scale) & (scale > 2.0 ** -127), scale / 2, scale)
    m = v.abs() / scale
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return torch.copysign((torch.round(m / step) * step).clamp(max=6.0), v) * scale


def exact_values(codes, scales):
    low, high = codes.to(torch.int64) & 15, codes.to(torch.int64) >> 4
    q = torch.stack((low, high), -1).flatten(-2)
    exponent, mantissa = (q >> 1) & 3, (q & 1).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(exponent.double() - 1))
    value = torch.where(q > 7, -size, size)
    return value * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "storage":
        parts = [exact_grid(p.double().view(len(p), -1, BLOCK)).flatten(1) for p in s["x"].split(1 << 14)]
        return torch.cat(parts)
    if case["op"] == "balance":
        logits, valid = s["logits"].double(), s["valid"]
        keep = torch.ones(len(logits), dtype=torch.bool, device="cuda") if valid is None else valid.bool()
        n = max(1, int(keep.sum()))
        a, b = s["coefs"]
        log_p = torch.log_softmax(logits, 1)
        p, lse = torch.exp(log_p), torch.logsumexp(logits, 1)
        counts = torch.bincount(s["ids"][keep].flatten().long(), minlength=case["experts"])
        f = counts.double() / (n * case["top_k"])
        mean_prob = p[keep].sum(0) / n
        balance, z = case["experts"] * f @ mean_prob, lse[keep].square().sum() / n
        dot = p @ f
        d = (a * case["experts"] / n) * p * (f - dot[:, None]) + (2 * b / n) * lse[:, None] * p
        d = torch.where(keep[:, None], d, 0) * s["grad"].double()
        return {"losses": torch.stack((a * balance + b * z, balance, z)), "counts": counts.to(torch.int32),
                "mean_prob": mean_prob, "dlogits": d}
    ends, assign = s["offsets"].tolist(), s["assign"].long()
    width = case["n"] // 2 if case["place"] == "gateup" else case["n"]
    x = s["x"].double() if s["x_scales"] is None else exact_values(s["x"], s["x_scales"])
    y = torch.empty(len(assign), width, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        at = torch.arange(ends[e], ends[e + 1], device="cuda")
        if not len(at):
            continue
        w = exact_values(s["w_codes"][e], s["w_scales"][e])
        if case["place"] == "gateup":
            z = x[assign[at] // case["top_k"]] @ w.T
            y[at] = z[:, :width] * torch.sigmoid(z[:, :width]) * z[:, width:]
        elif case["place"] == "down":
            y[assign[at]] = (x[at] @ w.T) * s["weights"][assign[at], None].double()
        else:
            y[at] = x[at] @ w.T
    return exact_grid(y.view(len(y), -1, BLOCK)).flatten(1) if case["y"] == "mx4" else y
