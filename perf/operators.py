"""The mixture-of-experts and fused-epilogue operators on compressed weights, as cases that can be measured.

An expert's MLP matrices are stored losslessly compressed (direct-palette form), so a product reads about 1.52 bytes per
weight.  The operators: the router (softmax, top-k, grouping by expert), the gate and up products of each expert's tokens
with SwiGLU, the product grouped by expert, the weighted combination of the experts' outputs, and the product with bias,
activation and residual in its epilogue.
"""
import math

import torch

own = False

#: Bytes of a weight in the direct-palette form: a 12304-byte record per 128 x 64 tile, and 128 bytes for each of the about
#: 1.1% of 64-element rows that hold an exponent outside the palette (one weight in 10^4 is a scaled outlier).
WEIGHT_BYTES = 12304 / 8192 + 2 * 0.011

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def _route(tokens, experts, top_k, dtype="float32", renormalize=True, masked=0):
    return dict(op="route", tokens=tokens, experts=experts, top_k=top_k, dtype=dtype, renormalize=renormalize, masked=masked)


def _swiglu(tokens, experts, top_k, rows, cols):
    return dict(op="swiglu", tokens=tokens, experts=experts, top_k=top_k, rows=rows, cols=cols)


def _grouped(tokens, experts, top_k, rows, cols, bias=False, activation="none"):
    """Down products: the input has one row per slot.  With a bias and an activation: the first layer of a plain MLP."""
    return dict(op="grouped", tokens=tokens, experts=experts, top_k=top_k, rows=rows, cols=cols, bias=bias, activation=activation)


def _epilogue(tokens, rows, cols, bias, activation, residual):
    return dict(op="epilogue", tokens=tokens, rows=rows, cols=cols, bias=bias, activation=activation, residual=residual)


def _combine(tokens, experts, top_k, cols, residual):
    return dict(op="combine", tokens=tokens, experts=experts, top_k=top_k, cols=cols, residual=residual)


def listed():
    cases = [
        # one token of a decode step through a router of 8 experts: latency
        ("route_token", _route(1, 8, 2)),
        # a long prompt through a router of 64 fine-grained experts, BF16 logits, 100 padded rows
        ("route_prompt", _route(8192, 64, 8, "bfloat16", True, 100)),
        # one token, two experts with the framework's block sizes: 0.36 GB of weights stream once
        ("swiglu_token", _swiglu(1, 8, 2, 14336, 4096)),
        # a decode batch of 32: every expert has a few tokens
        ("swiglu_decode", _swiglu(32, 8, 2, 14336, 4096)),
        # a prompt of 2048 tokens: about 512 rows per expert, bound by the tensor cores
        ("swiglu_prompt", _swiglu(2048, 8, 2, 14336, 4096)),
        # many small experts at an odd batch: 64 matrices of 2048 x 1024, about 4 rows each
        ("grouped_fine", _grouped(33, 64, 8, 2048, 1024)),
        # the first layer of a plain MLP per expert, with bias and GELU
        ("grouped_bias_gelu", _grouped(100, 8, 2, 4096, 1024, True, "gelu")),
        # the down products of a prompt of 2048 tokens
        ("grouped_prompt", _grouped(2048, 8, 2, 4096, 14336)),
        # an attention output projection for one token, bias and residual
        ("epilogue_token", _epilogue(1, 4096, 4096, True, "none", True)),
        # the first layer of a plain MLP for an odd batch
        ("epilogue_gelu", _epilogue(77, 14336, 4096, True, "gelu_tanh", False)),
        # one row of each of two experts' outputs
        ("combine_token", _combine(1, 8, 2, 4096, True)),
        # a prompt's tokens from 8 experts each
        ("combine_prompt", _combine(4096, 64, 8, 2048, True)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "swiglu", "grouped", "grouped", "epilogue", "epilogue", "combine"])
    if op == "route":
        experts = _log(rng, 2, 256)
        tokens = _log(rng, 1, 8192 if experts <= 64 else 2048)
        return _route(tokens, experts, rng.randint(1, min(8, experts)), rng.choice(["float32", "bfloat16"]),
                      rng.random() < 0.5, rng.randint(0, tokens - 1) // 4)
    if op == "epilogue":
        return _epilogue(_log(rng, 1, 2048), _log(rng, 64, 8192), 64 * _log(rng, 1, 112), rng.random() < 0.5,
                         rng.choice(ACTIVATIONS), rng.random() < 0.5)
    experts = _log(rng, 2, 48)
    top_k = rng.randint(1, min(4, experts))
    if op == "combine":
        return _combine(_log(rng, 1, 4096), experts, top_k, _log(rng, 64, 8192), rng.random() < 0.5)
    # few experts are large, many are small; any number of rows, columns in 64s
    most = 8192 if experts <= 8 else 2048
    rows, cols = _log(rng, 100, most), 64 * _log(rng, 1, most // 64)
    tokens = _log(rng, 1, 1024)
    if op == "swiglu":
        return _swiglu(tokens, experts, top_k, rows, cols)
    return _grouped(tokens, experts, top_k, rows, cols, rng.random() < 0.5, rng.choice(ACTIVATIONS))


def _active(c):
    """Experts that are expected to have a token."""
    return c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["tokens"])


def work(case):
    c, t = case, case["tokens"]
    n = t * c.get("top_k", 1)
    if c["op"] == "route":
        return {"bytes": t * c["experts"] * (4 if c["dtype"] == "float32" else 2) + n * 16 + 4 * (c["experts"] + 1),
                "flops": 4 * t * c["experts"]}
    if c["op"] == "combine":
        return {"bytes": n * (c["cols"] * 4 + 8) + t * c["cols"] * 2 * (2 if c["residual"] else 1), "flops": 2 * n * c["cols"]}
    weights = c["rows"] * c["cols"]
    if c["op"] == "epilogue":
        return {"bytes": weights * WEIGHT_BYTES + 2 * t * (c["cols"] + c["rows"] * (2 if c["residual"] else 1)) + 2 * c["rows"] * c["bias"],
                "flops": 2 * t * weights}
    if c["op"] == "swiglu":
        return {"bytes": 2 * _active(c) * weights * WEIGHT_BYTES + 2 * t * c["cols"] + 2 * n * c["rows"] + 4 * n, "flops": 4 * n * weights}
    return {"bytes": _active(c) * weights * WEIGHT_BYTES + 2 * n * (c["cols"] + c["rows"]) + 2 * _active(c) * c["rows"] * c["bias"],
            "flops": 2 * n * weights}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _weights(g, n, rows, cols):
    """[n, rows, cols] BF16: N(0, 0.02), one weight in 10^4 scaled by 100 (these force verbatim rows)."""
    w = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    for e in range(n):
        v = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
        out = torch.rand(rows, cols, generator=g, device="cuda") < 1e-4
        w[e] = torch.where(out, v * 100, v)
    return w


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _logits(g, tokens, experts):
    """Some experts are liked more than others, as in a trained router."""
    return torch.randn(tokens, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")


def _group(logits, top_k):
    """What the router hands to the products: slots grouped by expert, in token order."""
    tokens, experts = logits.shape
    weights, chosen = torch.topk(torch.softmax(logits, 1), top_k, dim=1)
    flat = chosen.reshape(-1)
    order = torch.argsort(flat, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(flat, minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    return dict(offsets=offsets.int(), rows=(order // top_k).int(), slots=slots.view(tokens, top_k).int(),
                weights=(weights / weights.sum(1, keepdim=True)).contiguous(), most=int(counts.max()))


def _experts(uw, w):
    """The handle that a user's program makes of its weights at load time."""
    ws = uw.Workspace(256)
    return uw.Experts([uw.DeviceMatrix.encode_on_device(w[e]).prepare_direct_palette(ws, keep_idx4=False) for e in range(len(w))])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    t, op = c["tokens"], c["op"]
    if op == "route":
        logits = _logits(g, t, c["experts"])
        if c["masked"]:  # padded rows take no expert
            logits[t - c["masked"]:] = -math.inf
        s["logits"] = logits.to(getattr(torch, c["dtype"]))
        if own:
            from mlp_huffman_coded_b200 import uw
            s["route"] = uw.Route(t, c["experts"], c["top_k"])
            s["route"].rows.zero_()
            s["ws"] = uw.Workspace(uw.route_workspace_bytes(t, c["experts"], c["top_k"]))
        return s
    if op == "epilogue":
        s["w"] = _weights(g, 1, c["rows"], c["cols"])[0]
        s["x"] = _bf16(g, t, c["cols"])
        s["bias"] = _bf16(g, c["rows"]) if c["bias"] else None
        s["residual"] = _bf16(g, t, c["rows"]) if c["residual"] else None
        if own:
            from mlp_huffman_coded_b200 import uw
            s["dm"] = uw.DeviceMatrix.encode_on_device(s["w"]).prepare_direct_palette(uw.Workspace(256), keep_idx4=False)
            s["ws"] = uw.Workspace(uw.epilogue_workspace_bytes(s["dm"], t))
            s["y"] = torch.empty(t, c["rows"], dtype=torch.bfloat16, device="cuda")
        return s
    s.update(_group(_logits(g, t, c["experts"]), c["top_k"]))
    n = t * c["top_k"]
    if op == "combine":
        s["parts"] = torch.randn(n, c["cols"], generator=g, device="cuda")
        s["residual"] = _bf16(g, t, c["cols"]) if c["residual"] else None
        if own:
            s["y"] = torch.empty(t, c["cols"], dtype=torch.bfloat16, device="cuda")
        return s
    s["w"] = _weights(g, c["experts"], c["rows"], c["cols"])
    if op == "swiglu":
        s["w_up"] = _weights(g, c["experts"], c["rows"], c["cols"])
        s["x"] = _bf16(g, t, c["cols"])
    else:
        s["x"] = _bf16(g, n, c["cols"])
        s["bias"] = _bf16(g, c["experts"], c["rows"]) if c["bias"] else None
    if own:
        from mlp_huffman_coded_b200 import uw
        s["experts"] = _experts(uw, s["w"])
        if op == "swiglu":
            s["experts_up"] = _experts(uw, s["w_up"])
        s["ws"] = uw.Workspace(uw.grouped_workspace_bytes(s["experts"], n, swiglu=op == "swiglu"))
        s["y"] = torch.empty(n, c["rows"], dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def _activate(v, name):
    if name == "relu":
        return v * (v > 0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def _plain_route(logits, top_k, renormalize):
    v = logits.float()
    tokens, experts = v.shape
    v = torch.where(torch.isnan(v), -math.inf, v).clamp(max=torch.finfo(torch.float32).max)
    top = v.max(1, keepdim=True).values
    p = torch.where(v > -math.inf, torch.exp(v - top.clamp(min=-torch.finfo(torch.float32).max)), 0)
    order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top_k]
    taken = torch.gather(v, 1, order) > -math.inf
    w = torch.where(taken, torch.gather(p, 1, order), 0)
    whole = (w if renormalize else p).sum(1, keepdim=True)
    w = torch.where(whole > 0, w / whole, 0)
    flat = torch.where(taken, order, experts).reshape(-1)
    by_expert = torch.sort(flat, stable=True)
    place = torch.empty_like(flat)
    place[by_expert.indices] = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.searchsorted(by_expert.values, torch.arange(experts + 1, device=flat.device))
    rows = torch.where(by_expert.values < experts, by_expert.indices // top_k, 0)
    return dict(weights=w, experts=torch.where(taken, order, -1).int(), rows=rows.int(), offsets=offsets.int(),
                slots=torch.where(taken, place.view(tokens, top_k), -1).int())


def _by_expert(s, x, rows):
    """x's rows as [experts, most, cols], and where each slot is in that."""
    o = s["offsets"].long()
    n = s["slots"].numel()
    at = (o[:-1, None] + torch.arange(s["most"], device=o.device)).clamp(max=n - 1)
    slot = torch.arange(n, device=o.device)
    expert = torch.searchsorted(o[1:], slot, right=True)
    return x[at if rows is None else rows.long()[at]].float(), expert, slot - o[expert]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from mlp_huffman_coded_b200 import uw
        if op == "route":
            r = s["route"]
            uw.moe_route(s["logits"], r, s["ws"], renormalize=c["renormalize"])
            return dict(weights=r.weights, experts=r.experts, rows=r.rows, offsets=r.offsets, slots=r.slots)
        if op == "swiglu":
            uw.gemm_grouped_swiglu(s["experts"], s["experts_up"], s["x"], s["offsets"], s["y"], s["ws"], rows=s["rows"])
        elif op == "grouped":
            uw.gemm_grouped(s["experts"], s["x"], s["offsets"], s["y"], s["ws"], bias=s["bias"], activation=c["activation"])
        elif op == "combine":
            uw.moe_combine(s["parts"], s["slots"], s["weights"], s["y"], residual=s["residual"])
        else:
            uw.gemm_epilogue(s["dm"], s["x"], s["y"], s["ws"], bias=s["bias"], activation=c["activation"], residual=s["residual"])
        return s["y"]
    if op == "route":
        return _plain_route(s["logits"], c["top_k"], c["renormalize"])
    if op == "swiglu":
        x, expert, place = _by_expert(s, s["x"], s["rows"])
        gate = torch.matmul(x, s["w"].float().transpose(1, 2))
        up = torch.matmul(x, s["w_up"].float().transpose(1, 2))
        return (gate * torch.sigmoid(gate) * up)[expert, place].bfloat16()
    if op == "grouped":
        x, expert, place = _by_expert(s, s["x"], None)
        v = torch.matmul(x, s["w"].float().transpose(1, 2))
        v = v if s["bias"] is None else v + s["bias"].float()[:, None]
        return _activate(v, c["activation"])[expert, place].bfloat16()
    if op == "combine":
        v = (s["weights"][:, :, None] * s["parts"][s["slots"].long()]).sum(1)
        return (v if s["residual"] is None else v + s["residual"].float()).bfloat16()
    v = torch.matmul(s["x"].float(), s["w"].float().t())
    v = _activate(v if s["bias"] is None else v + s["bias"].float(), c["activation"])
    return (v if s["residual"] is None else v + s["residual"].float()).bfloat16()


# ---------------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------------------------------

def _exact_activation(v, name):
    if name == "none":
        return v
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return v * torch.special.ndtr(v)
    return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def _exact_route(logits, top_k, renormalize):
    """Token by token, on the host."""
    rows_of = [[] for _ in range(logits.shape[1])]
    weights, chosen = [], []
    for t, l in enumerate(logits.double().cpu().tolist()):
        best = sorted((-v, e) for e, v in enumerate(l) if v > -math.inf)[:top_k]
        p = {e: math.exp(v + best[0][0]) for e, v in enumerate(l) if v > -math.inf}
        total = sum(p[e] for _, e in best) if renormalize else sum(p.values())
        chosen.append([e for _, e in best])
        weights.append([p[e] / total for _, e in best] + [0.0] * (top_k - len(best)))
        for j, e in enumerate(chosen[-1]):
            rows_of[e].append((t, j))
    offsets, rows, slots = [0], [], [[-1] * top_k for _ in weights]
    for group in rows_of:
        for t, j in group:
            slots[t][j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    rows += [0] * (len(weights) * top_k - len(rows))
    chosen = [e + [-1] * (top_k - len(e)) for e in chosen]
    whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(weights=torch.tensor(weights, dtype=torch.float64), experts=whole(chosen), rows=whole(rows), offsets=whole(offsets),
                slots=whole(slots))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s["logits"], case["top_k"], case["renormalize"])
    if op == "combine":
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        for j in range(case["top_k"]):
            y += s["weights"][:, j:j + 1].double() * s["parts"].index_select(0, s["slots"][:, j]).double()
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "epilogue":
        v = torch.nn.functional.linear(s["x"].double(), s["w"].double(), None if s["bias"] is None else s["bias"].double())
        v = _exact_activation(v, case["activation"])
        return v if s["residual"] is None else v + s["residual"].double()
    parts = []
    bounds = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):  # expert by expert
        x = s["x"].double()
        x = x[s["rows"][a:b].long()] if op == "swiglu" else x[a:b]
        v = x @ s["w"][e].double().T
        if op == "swiglu":
            v = v / (1 + torch.exp(-v)) * (x @ s["w_up"][e].double().T)
        else:
            v = _exact_activation(v if s["bias"] is None else v + s["bias"][e].double(), case["activation"])
        parts.append(v)
    return torch.cat(parts)
