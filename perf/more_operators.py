"""Routing from scores, the combination of routed rows and low-rank adapters, as cases to be timed.

Three operators, each forward alone or forward and backward (``train``):

- ``select``: a router's logits to experts and weights (softmax or sigmoid scores, a bias for the
  choice, groups, renormalised weights), with the assignments sorted by expert; the logits' gradient;
- ``combine``: the weighted sum of every token's routed rows; the rows' and the weights' gradients;
- ``adapters``: low-rank adapters beside a projection, of many requests or one for each expert; the
  gradients of the input and of both factors.

``run`` computes them with elementary torch operations, or with the library's calls where ``own``
is true.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "bf16": 2}


def select_case(tokens, experts, top_k, scores, groups, bias, renorm, kind, padded, train):
    """groups: (groups, groups kept, scores summed in a group), (1, 1, 1) for none."""
    return {"op": "select", "tokens": tokens, "experts": experts, "top_k": top_k, "scores": scores, "groups": groups[0],
            "kept": groups[1], "best": groups[2], "bias": bias, "renorm": renorm, "in": kind, "padded": padded,
            "train": train}


def combine_case(tokens, top_k, width, kind, out, base, dropped, train):
    return {"op": "combine", "tokens": tokens, "top_k": top_k, "width": width, "in": kind, "out": out, "base": base,
            "dropped": dropped, "train": train}


def adapters_case(tokens, adapters, top_k, rank, n_in, n_out, out, place, train):
    """place: "decode" (every token a request of its own), "prompts" (requests of many tokens) or
    "experts" (top_k adapters a token, rows gathered by token)."""
    return {"op": "adapters", "tokens": tokens, "adapters": adapters, "top_k": top_k, "rank": rank, "n_in": n_in,
            "n_out": n_out, "out": out, "place": place, "train": train}


def listed():
    cases = {
        # One decoded token's router of 256 experts in 8 groups: launch latency.
        "select 1 token": select_case(1, 256, 8, "sigmoid", (8, 4, 2), True, True, "f32", False, False),
        # A ragged prompt in bf16 through a router with softmax weights as they are.
        "select 2085 tokens": select_case(2085, 100, 6, "softmax", (1, 1, 1), False, False, "bf16", False, False),
        # One padded training batch of the full-size router, forward and backward.
        "select 4096 tokens training": select_case(4096, 256, 8, "softmax", (1, 1, 1), False, True, "f32", True, True),
        # The largest router over a large packed batch.
        "select 65536 tokens training": select_case(65536, 512, 16, "sigmoid", (8, 4, 2), True, True, "bf16", True, True),
        # One decoded token's eight rows of the down product beside the shared expert's.
        "combine 1 token": combine_case(1, 8, 2048, "f32", "f32", True, False, False),
        # A long prompt's rows in bf16, as the next layer takes them.
        "combine 4096 tokens": combine_case(4096, 8, 2048, "bf16", "bf16", True, False, False),
        # A training batch with padding tokens and an odd width.
        "combine 2085 tokens training": combine_case(2085, 6, 1999, "bf16", "f32", False, True, True),
        # One decoded token with its request's adapter out of a store of 64.
        "adapters 1 token": adapters_case(1, 64, 1, 16, 2048, 4096, "bf16", "decode", False),
        # A batch of decoded tokens, each its own request.
        "adapters 64 tokens": adapters_case(64, 64, 1, 32, 4096, 4096, "bf16", "decode", False),
        # Prompts of several requests side by side.
        "adapters 4096 tokens": adapters_case(4096, 8, 1, 16, 4096, 4096, "bf16", "prompts", False),
        # Three adapters trained together on a ragged batch, with an output width of no even multiple.
        "adapters 2085 tokens training": adapters_case(2085, 3, 1, 64, 2048, 1000, "f32", "prompts", True),
        # An adapter for each of 256 experts' gate and up matrices, trained on a batch of routed rows.
        "adapters of 256 experts training": adapters_case(4096, 256, 8, 16, 2048, 1024, "bf16", "experts", True),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "combine", "adapters", "adapters"])
    train = rng.random() < 0.5
    kind = rng.choice(["bf16", "f32"])
    tokens = _log(rng, 1, 65536)
    if op == "select":
        experts = _log(rng, 2, 512)
        groups = (1, 1, 1)
        if rng.random() < 0.5:
            # At least four experts a group, so that a choice among groups is one of sums, not of single ties.
            runs = [g for g in (2, 3, 4, 8, 16) if experts % g == 0 and experts // g >= 4]
            if runs:
                n = rng.choice(runs)
                groups = (n, rng.randint(1, n - 1), rng.choice([1, 2]))
        top_k = rng.randint(1, min(16, experts // groups[0] * groups[1]))
        scores = rng.choice(["softmax", "sigmoid"])
        bias = rng.random() < 0.5 or (scores == "sigmoid" and groups[0] > 1)
        return select_case(tokens, experts, top_k, scores, groups, bias, rng.random() < 0.6, kind, rng.random() < 0.5, train)
    if op == "combine":
        width, top_k = _log(rng, 16, 8192), rng.randint(1, 16)
        tokens = _log(rng, 1, max(1, min(65536, 4096 * 8 * 2048 // (width * top_k))))
        return combine_case(tokens, top_k, width, kind, rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                            rng.random() < 0.5, train)
    place = rng.choice(["decode", "prompts", "experts"])
    rank = rng.choice([4, 8, 16, 16, 32, 64, 12, 128])
    n_in, n_out = (_log(rng, 64, 4096) for _ in range(2))
    if rng.random() < 0.7:  # widths are mostly multiples of 64
        n_in, n_out = (64 * max(1, n // 64) for n in (n_in, n_out))
    if place == "decode":
        return adapters_case(_log(rng, 1, 256), _log(rng, 1, 64), 1, rank, n_in, n_out, kind, place, False)
    if place == "prompts":
        return adapters_case(_log(rng, 16, 4096), _log(rng, 1, 16), 1, rank, n_in, n_out, kind, place, train)
    adapters = _log(rng, 4, 64)
    return adapters_case(_log(rng, 16, 2048), adapters, rng.randint(1, min(8, adapters)), min(rank, 32), n_in, n_out, kind,
                         place, train)


# ---- inputs ------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def buffer(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    T, i32 = case["tokens"], torch.int32
    s = {"case": case}
    if case["op"] == "select":
        E, k = case["experts"], case["top_k"]
        s["logits"] = (1.5 * randn(T, E) + 0.5 * randn(E)).to(TYPES[case["in"]])
        s["bias"] = 0.1 * randn(E) if case["bias"] else None
        s["valid"] = (rand(T) < 0.85).to(torch.uint8) if case["padded"] else None
        s["scale"] = 2.5 if case["scores"] == "sigmoid" else 1.0
        s["ids"], s["weights"] = buffer(T, k, dtype=i32), buffer(T, k)
        s["counts"], s["offsets"] = buffer(E, dtype=i32), buffer(E + 1, dtype=i32)
        # Places of a padding token's assignments stay as they are.
        s["order"] = torch.full((T * k,), -1, dtype=i32, device="cuda")
        if case["train"]:
            s["dweights"], s["dlogits"] = randn(T, k), torch.empty_like(s["logits"])
            # The balance loss's gradient, to which this one is added, in bf16 only, to have both forms.
            s["other"] = (1e-3 * randn(T, E)).to(s["logits"].dtype) if case["in"] == "bf16" else None
        return s

    if case["op"] == "combine":
        k, H = case["top_k"], case["width"]
        s["rows"] = randn(T * k, H).to(TYPES[case["in"]])
        s["weights"] = torch.softmax(randn(T, k), 1)
        s["ids"] = torch.randint(0, 256, (T, k), generator=g, device="cuda", dtype=i32)
        if case["dropped"]:  # padding tokens have no expert
            s["ids"][rand(T) < 0.15] = -1
        out = TYPES[case["out"]]
        s["base"] = randn(T, H).to(out) if case["base"] else None
        s["y"] = buffer(T, H, dtype=out)
        if case["train"]:
            s["dy"] = randn(T, H).to(out)
            s["drows"], s["dweights"] = torch.empty_like(s["rows"]), buffer(T, k)
        return s

    n, k, r, K, N = (case[name] for name in ("adapters", "top_k", "rank", "n_in", "n_out"))
    out = TYPES[case["out"]]
    if case["place"] == "decode":  # some requests have no adapter (but not the only one)
        ids = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=i32)
        ids[1:][rand(T)[1:] < 0.1] = -1
    elif case["place"] == "prompts":
        cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda")).values
        which = torch.randperm(n, generator=g, device="cuda")
        ids = which[torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)].to(i32)
    else:
        logits = randn(T, n) + 0.5 * randn(n)
        ids = torch.topk(logits, k, dim=1).indices.flatten().to(i32)
    rows = T * k
    s["ids"] = ids
    s["most"] = int(torch.bincount(ids[ids >= 0].long(), minlength=n).amax())
    s["a"], s["b"] = (randn(n, r, K) / math.sqrt(K)).to(torch.bfloat16), (0.1 * randn(n, N, r)).to(torch.bfloat16)
    s["scales"] = 0.5 + rand(n)
    s["x"] = randn(T, K).to(torch.bfloat16)
    s["base"] = randn(rows, N).to(out)
    s["y"] = s["base"].clone()
    s["counts"], s["offsets"] = buffer(n, dtype=i32), buffer(n + 1, dtype=i32)
    s["order"] = torch.full((rows,), -1, dtype=i32, device="cuda")
    if case["train"]:
        s["dy"] = randn(rows, N).to(out)
        s["h"], s["dx"] = buffer(rows, r), buffer(rows, K, dtype=torch.bfloat16)
        s["da"], s["db"] = buffer(n, r, K), buffer(n, N, r)
    return s


# ---- the plain form ----------------------------------------------------------------------------


def sorted_by_id(ids, n):
    """Counts, offsets and the places of ids 0 .. n - 1 in their order (others: -1 behind the last)."""
    flat = ids.flatten().long()
    known = flat >= 0
    key = torch.where(known, flat, n)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(n + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(n + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(counts[:n], 0)
    order = torch.where(torch.arange(len(flat), device=ids.device) < offsets[n], order, -1)
    return counts[:n].to(torch.int32), offsets.to(torch.int32), order.to(torch.int32)


def largest(v, k):
    """Values and places of the k largest of each row, equal ones towards the lower place."""
    v, at = torch.sort(v, dim=1, descending=True, stable=True)
    return v[:, :k], at[:, :k]


def plain_select(s):
    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    # The choice is one between values that may be close, or equal: taken in 64 bits.
    l = s["logits"].double()
    if c["scores"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-l))
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        per = E // c["groups"]
        group = largest(choice.view(T * c["groups"], per), c["best"])[0].sum(1).view(T, c["groups"])
        kept = torch.zeros_like(group, dtype=torch.bool)
        kept.scatter_(1, largest(group, c["kept"])[1], True)
        choice = torch.where(kept.repeat_interleave(per, 1), choice, -math.inf)
    ids = largest(choice, k)[1]
    chosen = score.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if c["renorm"] else 1.0
    weights = s["scale"] * chosen / total
    on = None
    if s["valid"] is not None:
        on = s["valid"].bool()[:, None]
        ids, weights = torch.where(on, ids, -1), torch.where(on, weights, 0)
    counts, offsets, order = sorted_by_id(ids, E)
    out = {"ids": ids.to(torch.int32), "weights": weights.float(), "counts": counts, "offsets": offsets, "order": order}
    if c["train"]:
        # w = scale s / total: dl = (ds/dl)^T dw/ds, with ds/dl diag(s) - s s^T or diag(s (1 - s)).
        dw = s["dweights"].double()
        if c["renorm"]:
            dw = dw - (dw * weights).sum(1, keepdim=True) / s["scale"]
        dscore = torch.zeros_like(score).scatter_(1, ids.clamp(min=0), s["scale"] * dw / total)
        if c["scores"] == "softmax":
            dl = score * (dscore - (dscore * score).sum(1, keepdim=True))
        else:
            dl = dscore * score * (1 - score)
        if on is not None:
            dl = torch.where(on, dl, 0)
        if s["other"] is not None:
            dl = dl + s["other"].double()
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def plain_combine(s):
    c = s["case"]
    T, k, H = c["tokens"], c["top_k"], c["width"]
    rows = s["rows"].float().view(T, k, H)
    w = torch.where(s["ids"] >= 0, s["weights"], 0)
    y = (rows * w[:, :, None]).sum(1)
    if s["base"] is not None:
        y = y + s["base"].float()
    out = {"y": y.to(TYPES[c["out"]])}
    if c["train"]:
        dy = s["dy"].float()[:, None, :]
        out["drows"] = (w[:, :, None] * dy).view(T * k, H).to(s["rows"].dtype)
        out["dweights"] = torch.where(s["ids"] >= 0, (rows * dy).sum(2), 0)
    return out


def plain_adapters(s):
    c = s["case"]
    n, k, rows = c["adapters"], c["top_k"], c["tokens"] * c["top_k"]
    _, offsets, order = sorted_by_id(s["ids"], n)
    at = torch.arange(rows, device=order.device)
    at = at[at < offsets[n]] if c["place"] == "decode" else at  # the others have an adapter for every row
    row = order.long()[at]
    which = s["ids"].long()[row]
    x, scale = s["x"][row // k].float(), s["scales"][which]
    if not c["train"] and len(at) <= 2 * n:  # few rows: each with its own adapter
        h = torch.bmm(s["a"][which].float(), x[:, :, None])
        d = torch.bmm(s["b"][which].float(), h)[:, :, 0]
    else:  # every adapter's rows side by side, up to the largest number that one has
        slot = at - offsets.long()[which]
        a, b = s["a"].float(), s["b"].float()
        wide = x.new_zeros(n, s["most"], c["n_in"])
        wide[which, slot] = x
        h = torch.bmm(wide, a.transpose(1, 2).contiguous())
        d = torch.bmm(h, b.transpose(1, 2).contiguous())[which, slot]
    y = s["base"].to(torch.float32, copy=True)
    y[row] += scale[:, None] * d
    out = {"y": y.to(TYPES[c["out"]])}
    if c["train"]:
        wide_dy = x.new_zeros(n, s["most"], c["n_out"])
        wide_dy[which, slot] = scale[:, None] * s["dy"][row].float()
        dh = torch.bmm(wide_dy, b)
        dx = x.new_empty(rows, c["n_in"])
        dx[row] = torch.bmm(dh, a)[which, slot]
        out["dx"] = dx.to(torch.bfloat16)
        out["da"] = torch.bmm(dh.transpose(1, 2).contiguous(), wide)
        out["db"] = torch.bmm(wide_dy.transpose(1, 2).contiguous(), h)
    return out


# ---- the library's calls -----------------------------------------------------------------------


def own_select(s):
    import bit_quantized_moe_router_amd as moe

    c = s["case"]
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    if "desc" not in s:  # what a program makes once
        s["desc"] = moe.make_select_desc(E, k, moe.MOE_SOFTMAX if c["scores"] == "softmax" else moe.MOE_SIGMOID, c["groups"],
                                         c["kept"], c["best"], renormalise=int(c["renorm"]), scale=s["scale"])
        s["ws"] = torch.empty(moe.moe_select_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")
    out = {name: s[name] for name in ("ids", "weights", "counts", "offsets", "order")}
    moe.moe_select_forward(s["desc"], s["logits"], s["bias"], s["valid"], *out.values(), s["ws"])
    if c["train"]:
        moe.moe_select_backward(s["desc"], s["logits"], s["ids"], s["weights"], s["dweights"], s["other"], s["dlogits"])
        out["dlogits"] = s["dlogits"]
    return out


def own_combine(s):
    import bit_quantized_moe_router_amd as moe

    moe.moe_combine_forward(s["rows"], s["ids"], s["weights"], s["base"], s["y"])
    if not s["case"]["train"]:
        return {"y": s["y"]}
    moe.moe_combine_backward(s["dy"], s["rows"], s["ids"], s["weights"], s["drows"], s["dweights"])
    return {name: s[name] for name in ("y", "drows", "dweights")}


def own_adapters(s):
    import bit_quantized_moe_router_amd as moe

    c = s["case"]
    n, k, rows = c["adapters"], c["top_k"], c["tokens"] * c["top_k"]
    if "desc" not in s:  # what a program makes once
        s["desc"] = moe.make_adapter_desc(n, c["rank"], c["n_in"], c["n_out"],
                                          moe.MOE_F32 if c["out"] == "f32" else moe.MOE_BF16)
        s["sort_ws"] = torch.empty(moe.moe_sort_workspace_bytes(rows, n), dtype=torch.uint8, device="cuda")
        if c["train"]:
            s["ws"] = torch.empty(moe.moe_adapters_workspace_bytes(s["desc"], rows), dtype=torch.uint8, device="cuda")
    moe.moe_sort_assignments(s["ids"], n, s["counts"], s["offsets"], s["order"], s["sort_ws"])
    places = dict(src_rows=s["order"], src_div=k, dst_rows=s["order"])
    moe.moe_adapters_forward(s["desc"], s["a"], s["b"], s["scales"], s["x"], s["offsets"], rows, s["base"], s["y"],
                             s.get("h"), **places)
    if not c["train"]:
        return {"y": s["y"]}
    moe.moe_adapters_backward(s["desc"], s["a"], s["b"], s["scales"], s["x"], s["h"], s["dy"], s["offsets"], rows, None,
                              s["dx"], s["da"], s["db"], s["ws"], **places)
    return {name: s[name] for name in ("y", "dx", "da", "db")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"select": own_select, "combine": own_combine, "adapters": own_adapters}[op](state)
    return {"select": plain_select, "combine": plain_combine, "adapters": plain_adapters}[op](state)


# ---- what a pass cannot do without -------------------------------------------------------------


def work(case):
    T, k = case["tokens"], case["top_k"]
    if case["op"] == "select":
        cells, size = T * case["experts"], SIZES[case["in"]]
        moved = cells * size + 12 * T * k + 12 * case["experts"]
        if case["train"]:
            # Ids, weights and their gradient in again, the logits' gradient out, and the one it is added to in.
            moved += 12 * T * k + cells * size * (2 if case["in"] == "bf16" else 1)
            if not case["renorm"] and case["scores"] == "softmax":
                moved += cells * size  # the probabilities again
        return {"bytes": moved, "flops": (8 + 2 * k) * cells}
    if case["op"] == "combine":
        H, size, out = case["width"], SIZES[case["in"]], SIZES[case["out"]]
        moved = T * H * (k * size + out * (2 if case["base"] else 1)) + 8 * T * k
        flops = 2 * T * k * H
        if case["train"]:  # the rows and dy in, the rows' gradient out
            moved += T * H * (2 * k * size + out) + 12 * T * k
            flops *= 2.5
        return {"bytes": moved, "flops": flops}
    n, r, K, N = (case[name] for name in ("adapters", "rank", "n_in", "n_out"))
    rows, out = T * k, SIZES[case["out"]]
    used = n if case["place"] != "decode" else min(n, round(n * (1 - (1 - 1 / n) ** T)))
    factors = used * r * (K + N) * 2
    moved = factors + T * K * 2 + 2 * rows * N * out + 12 * rows
    flops = 2 * rows * r * (K + N)
    if case["train"]:
        # dy, x and the factors in; dx, dA and dB out.
        moved += factors + rows * N * out + T * K * 2 + rows * K * 2 + n * r * (K + N) * 4 + rows * r * 8
        flops *= 3
    return {"bytes": moved, "flops": flops}


# ---- the definition in 64 bits -----------------------------------------------------------------


def exact_select(case, s):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    l = s["logits"].double()
    p = torch.softmax(l, 1) if case["scores"] == "softmax" else torch.sigmoid(l)
    c = p.clone() if s["bias"] is None else p + s["bias"].double()
    per = E // case["groups"]
    if case["groups"] > 1:
        g = c.view(T, case["groups"], per)
        g = g.amax(2) if case["best"] == 1 else torch.topk(g, 2, dim=2).values.sum(2)
        # A group stays if fewer than `kept` others are better, or as good and further left.
        left = torch.ones(case["groups"], case["groups"], dtype=torch.bool, device="cuda").triu(1)
        better = (g[:, :, None] > g[:, None, :]) | ((g[:, :, None] == g[:, None, :]) & left)
        stays = better.sum(1) < case["kept"]
        c.view(T, case["groups"], per).masked_fill_(~stays[:, :, None], -math.inf)
    place = torch.arange(E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int64, device="cuda")
    for j in range(k):
        top = c.amax(1, keepdim=True)
        ids[:, j] = torch.where(c == top, place, E).amin(1)
        c.scatter_(1, ids[:, j:j + 1], -math.inf)
    # Weights and gradient by the softmax's or the sigmoid's own derivative.
    p_j = p.gather(1, ids)
    f = s["scale"] / (p_j.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(p_j[:, :1]))
    keep = torch.ones(T, 1, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"].bool()[:, None]
    weights = torch.where(keep, f * p_j, 0)
    ids = torch.where(keep, ids, -1)
    flat = ids.flatten()
    counts = torch.bincount(flat + 1, minlength=E + 1)[1:]
    ends = torch.cumsum(counts, 0)
    order = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    known = torch.nonzero(flat >= 0)[:, 0]
    order[:len(known)] = known[torch.sort(flat[known], stable=True).indices]
    out = {"ids": ids.to(torch.int32), "weights": weights, "counts": counts.to(torch.int32),
           "offsets": torch.cat((ends.new_zeros(1), ends)).to(torch.int32), "order": order.to(torch.int32)}
    if case["train"]:
        up = s["dweights"].double()
        dp = f * (up - (up * f * p_j).sum(1, keepdim=True) / s["scale"]) if case["renorm"] else f * up
        at = ids.clamp(min=0)
        if case["scores"] == "softmax":
            d = -p * (dp * p_j).sum(1, keepdim=True)
            d.scatter_add_(1, at, dp * p_j)
        else:
            d = torch.zeros_like(p).scatter_add_(1, at, dp * p_j * torch.sigmoid(-l.gather(1, at)))
        d = torch.where(keep, d, 0)
        out["dlogits"] = d if s["other"] is None else d + s["other"].double()
    return out


def exact_combine(case, s):
    T, k, H = case["tokens"], case["top_k"], case["width"]
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda") if s["base"] is None else s["base"].double()
    out = {"y": y}
    if case["train"]:
        out["drows"] = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        out["dweights"] = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["ids"][:, j] >= 0)[:, 0]
        w, r = s["weights"][t, j, None].double(), s["rows"][t * k + j].double()
        y[t] += w * r
        if case["train"]:
            dy = s["dy"][t].double()
            out["drows"][t * k + j] = w * dy
            out["dweights"][t, j] = (dy * r).sum(1)
    return out


def exact_adapters(case, s):
    k, train = case["top_k"], case["train"]
    y = s["base"].double()
    if train:
        dx = torch.zeros(len(y), case["n_in"], dtype=torch.float64, device="cuda")
        da, db = torch.zeros_like(s["da"], dtype=torch.float64), torch.zeros_like(s["db"], dtype=torch.float64)
    for e in range(case["adapters"]):
        row = torch.nonzero(s["ids"] == e)[:, 0]
        if not len(row):
            continue
        a, b, x = s["a"][e].double(), s["b"][e].double() * s["scales"][e].double(), s["x"][row // k].double()
        y[row] += (x @ a.T) @ b.T
        if train:
            dy = s["dy"][row].double()
            dh = dy @ b
            dx[row] = dh @ a
            da[e] = dh.T @ x
            db[e] = (dy.T @ (x @ a.T)) * s["scales"][e].double()
    return {"y": y, "dx": dx, "da": da, "db": db} if train else {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"select": exact_select, "combine": exact_combine, "adapters": exact_adapters}[case["op"]](case, s)
