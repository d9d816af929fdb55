"""The operators of a mixture-of-experts layer over block-scaled operands: what is measured, and their plain forms.

  route     router scores -> the k experts of each token, their weights, and the expert-sorted order of the (token, expert)
            pairs; with the router's gradient for training
  dispatch  copies each token's row to its experts' places in that order, plain or quantised on the way to the codes and scales
            that the block-scaled product reads
  combine   adds the experts' result rows back per token, weighted, onto a residual; with its gradients for training
  linear    the grouped block-scaled product with bias, activation and residual in its epilogue; with the epilogue's gradients

A case is one pass through one of them. The sizes are this repository's MoE workload (65536 expert rows of 7168, 256 experts,
2048 wide) and weight (14336 x 4096) next to generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

CODE_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of a decoding step: latency counts
        dict(name="route-decode", op="route", tokens=1, experts=256, k=8, dtype="fp32", score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renorm=True, scale=2.5, masked=0.0, train=False),
        # a long prompt batch, balanced by a bias, experts in groups
        dict(name="route-prefill", op="route", tokens=65536, experts=256, k=8, dtype="bf16", score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_score="top2", renorm=True, scale=2.5, masked=0.0, train=False),
        # a training batch with padding: softmax over all experts, weights as they are, forward and the logits' gradient
        dict(name="route-train", op="route", tokens=16381, experts=64, k=6, dtype="fp32", score="softmax", bias=False, groups=1,
             topk_groups=1, group_score="max", renorm=False, scale=1.0, masked=0.1, train=True),
        # a decoding step of a few requests into the E2M1 operand
        dict(name="dispatch-decode", op="dispatch", tokens=4, experts=256, k=8, cols=7168, dtype="bf16", format="e2m1", mode="page"),
        # a prompt batch into the E2M1 operand: 65536 expert rows of 7168
        dict(name="dispatch-prefill", op="dispatch", tokens=8192, experts=256, k=8, cols=7168, dtype="bf16", format="e2m1", mode="page"),
        # fp32 activations into the E4M3 operand, a width that ends inside a scale atom
        dict(name="dispatch-e4m3", op="dispatch", tokens=4099, experts=60, k=3, cols=4128, dtype="fp32", format="e4m3", mode="floor"),
        # a prompt batch back onto its residual stream
        dict(name="combine-prefill", op="combine", tokens=8192, experts=256, k=8, cols=7168, dtype="bf16", residual=True, train=False),
        # the gradients of a training batch: of the experts' rows and of the router's weights
        dict(name="combine-train", op="combine", tokens=4099, experts=64, k=6, cols=4096, dtype="bf16", residual=False, train=True),
        # the first expert product of one decoded token: eight experts of one row each
        dict(name="linear-decode", op="linear", rows=8, experts=64, n=4096, k=7168, format="e2m1", out="bf16", bias=False,
             act="swiglu", residual=False, preact=False, train=False),
        # the first expert product of a prompt batch: 65536 rows over 64 experts, gate and up side by side
        dict(name="linear-prefill", op="linear", rows=65536, experts=64, n=4096, k=7168, format="e2m1", out="bf16", bias=False,
             act="swiglu", residual=False, preact=False, train=False),
        # a dense layer of the E4M3 path with everything in the epilogue, fp32 results, pre-activation kept for the backward pass
        dict(name="linear-dense", op="linear", rows=2049, experts=1, n=14336, k=4096, format="e4m3", out="fp32", bias=True,
             act="gelu", residual=True, preact=True, train=False),
        # the epilogue's gradients over the experts of a training batch
        dict(name="linear-train", op="linear", rows=16384, experts=64, n=4096, k=0, format="e2m1", out="bf16", bias=True,
             act="swiglu", residual=False, preact=True, train=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("route", "route", "dispatch", "combine", "linear", "linear"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * max(2, _log(rng, 8, 512) // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(12, topk_groups * (experts // groups)))
        train = rng.random() < 0.4
        return dict(op=op, tokens=_log(rng, 1, 65536 * 256 // max(256, experts)), experts=experts, k=k,
                    dtype=rng.choice(("bf16", "fp32")), score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.6,
                    groups=groups, topk_groups=topk_groups, group_score=rng.choice(("top2", "max")), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.2)), train=train)
    if op in ("dispatch", "combine"):
        experts = _log(rng, 4, 256)
        k = rng.randint(1, min(8, experts))
        case = dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, k=k, cols=_log(rng, 64, 7168), dtype=rng.choice(("bf16", "bf16", "fp32")))
        if case["dtype"] == "fp32":
            case["tokens"] = max(1, case["tokens"] // 2)
        if op == "dispatch":
            case["format"] = rng.choice(("e2m1", "e2m1", "e4m3", "values"))
            case["mode"] = "floor" if case["format"] == "e4m3" else rng.choice(("page", "floor"))
            if rng.random() < 0.7:  # operands of the product are whole blocks wide; other widths are allowed
                case["cols"] = max(64, case["cols"] // 64 * 64)
        else:
            case["residual"] = rng.random() < 0.5
            case["train"] = rng.random() < 0.4
        return case
    fmt = rng.choice(("e2m1", "e2m1", "e4m3"))
    unit = 64 if fmt == "e2m1" else 32
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "swiglu"))
    k, n = max(unit, _log(rng, 128, 7168) // unit * unit), _log(rng, 32, 8192)
    n += n % 2 if act == "swiglu" else 0
    train = rng.random() < 0.25
    return dict(op=op, rows=_log(rng, 1, 16384), experts=rng.choice((1, 2, 7, 16, 48)), n=n, k=0 if train else k, format=fmt,
                out=rng.choice(("bf16", "bf16", "fp32")), bias=rng.random() < 0.5, act=act, residual=rng.random() < 0.4,
                preact=train or rng.random() < 0.3, train=train)


# ---------------------------------------------------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _plan(experts, count):
    """The expert-sorted order of a [tokens, k] table of experts (-1: none): each pair's row, each row's pair, rows per expert."""
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, count, flat)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(flat < 0, -1, rows)
    counts = torch.zeros(count, dtype=torch.int64, device=flat.device)
    counts.index_add_(0, key.clamp(max=count - 1), (flat >= 0).long())
    slots = torch.where(torch.arange(flat.numel(), device=flat.device) < counts.sum(), order, -1)
    return rows.view(experts.shape).int(), slots.int(), counts


def _expert_sizes(g, rows, experts):
    """Rows per expert: a skewed load, some experts without a row; few rows go to as many experts."""
    if rows <= experts:
        return (torch.randperm(experts, generator=g, device="cuda") < rows).long()
    share = torch.rand(experts, generator=g, device="cuda") ** 4 + 1e-9
    picks = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(picks, minlength=experts)


def _codes(g, rows, k, fmt):
    if fmt == "e2m1":  # two codes a byte, every code as often
        return torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    return _normal(g, rows, k, std=80.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scale_bytes(rows, k):
    return 512 * (-(-rows // 128)) * (-(-k // 128))


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = dict(case)
    if op == "route":
        t, e = case["tokens"], case["experts"]
        s["logits"] = _normal(g, t, e, std=1.5, dtype=DTYPES[case["dtype"]])
        s["bias_values"] = _normal(g, e, std=0.05) if case["bias"] else None
        s["token_mask"] = torch.rand(t, generator=g, device="cuda") >= case["masked"] if case["masked"] else None
        s["grad"] = _normal(g, t, case["k"])
        return s
    if op in ("dispatch", "combine"):
        t, k, cols, dt = case["tokens"], case["k"], case["cols"], DTYPES[case["dtype"]]
        load = torch.rand(case["experts"], generator=g, device="cuda") ** 2 + 1e-3
        s["chosen"] = torch.multinomial(load.expand(t, -1), k, generator=g).int()
        s["rows"], s["slots"], s["counts"] = _plan(s["chosen"], case["experts"])
        s["weights"] = torch.rand(t, k, generator=g, device="cuda") * 0.5
        if op == "dispatch":  # activations: normal values, a few wide channels
            s["x"] = _normal(g, t, cols)
            s["x"][:, torch.randint(0, cols, (1 + cols // 200,), generator=g, device="cuda")] *= 50.0
            s["x"] = s["x"].to(dt)
        else:
            s["y"] = _normal(g, t * k, cols, dtype=dt)
            s["res"] = _normal(g, t, cols, dtype=dt) if case["residual"] else None
            s["grad"] = _normal(g, t, cols, dtype=dt) if case["train"] else None
        return s
    m, n, k, e, fmt, dt = case["rows"], case["n"], case["k"], case["experts"], case["format"], DTYPES[case["out"]]
    s["counts"] = _expert_sizes(g, m, e)
    s["sizes"] = s["counts"].tolist()
    width = n // 2 if case["act"] == "swiglu" else n
    if case["train"]:
        s["z"] = _normal(g, m, n, std=1.5, dtype=dt)
        s["grad"] = _normal(g, m, width, dtype=dt)
        return s
    s["a"] = _codes(g, m, k, fmt)
    s["b"] = _codes(g, e * n, k, fmt).view(e, n, -1)
    # block scales around the size that gives pre-activations of about one
    rms = 2.9 if fmt == "e2m1" else 80.0
    mid = 127 - round(math.log2(rms * rms * math.sqrt(k)))
    s["a_scales"] = torch.randint(126, 129, (_scale_bytes(m, k),), generator=g, device="cuda", dtype=torch.uint8)
    s["b_scales"] = torch.randint(mid - 1, mid + 2, (e, _scale_bytes(n, k)), generator=g, device="cuda", dtype=torch.uint8)
    s["bias_values"] = _normal(g, e, n) if case["bias"] else None
    s["res"] = _normal(g, m, width, dtype=dt) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------------- plain forms


def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    top = logits.max(1, keepdim=True).values
    p = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    return p / p.sum(1, keepdim=True).clamp(min=1e-300 if p.dtype == torch.float64 else 1e-37)


def _select(s):
    """The chosen experts [tokens, k], best key first (ties: the lower expert); -1 where there is none. Keys in 64 bits."""
    t, e, groups, k = s["tokens"], s["experts"], s["groups"], s["k"]
    x = s["logits"].double()
    bad = (torch.isnan(x) | (x == math.inf)).any(1)
    key = _scores(x, s["score"])
    closed = x == -math.inf
    if s["bias_values"] is not None:
        key = key + s["bias_values"].double()
        closed = closed | ~torch.isfinite(s["bias_values"])
    key = torch.where(closed, -math.inf, key)
    if groups > 1:
        by = key.view(t, groups, e // groups)
        best = by.sort(2, descending=True).values
        if s["group_score"] == "top2":
            second = best[:, :, 1] if e // groups > 1 else torch.full_like(best[:, :, 0], -math.inf)
            rank = best[:, :, 0] + torch.where(second == -math.inf, 0.0, second)
        else:
            rank = best[:, :, 0]
        order = rank.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros(t, groups, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order, True)
        key = torch.where(keep[:, :, None], by, -math.inf).view(t, e)
    best = key.sort(dim=1, descending=True, stable=True)
    chosen = torch.where(best.values[:, :k] == -math.inf, -1, best.indices[:, :k])
    chosen = torch.where(bad[:, None], torch.arange(k, device=x.device), chosen)
    if s["token_mask"] is not None:
        chosen = torch.where(s["token_mask"][:, None], chosen, -1)
        bad = bad & s["token_mask"]
    return chosen, bad


def _route(s):
    chosen, bad = _select(s)
    some = chosen >= 0
    at = chosen.clamp(min=0)
    scores = _scores(s["logits"].float(), s["score"])
    picked = torch.where(some, scores.gather(1, at), 0.0)
    total = picked.sum(1, keepdim=True)
    weights = s["scale"] * (picked / torch.where(total == 0, 1.0, total) if s["renorm"] else picked)
    weights = torch.where(bad[:, None], math.nan, weights)
    rows, slots, counts = _plan(chosen, s["experts"])
    out = dict(weights=weights, experts=chosen.int(), rows=rows, slots=slots, counts=counts)
    if s["train"]:
        grad = torch.where(some, s["grad"], 0.0) * s["scale"]
        if s["renorm"]:
            share = picked / torch.where(total == 0, 1.0, total)
            grad = (grad - (grad * share).sum(1, keepdim=True)) / torch.where(total == 0, 1.0, total)
        by_score = torch.zeros_like(scores).scatter_add_(1, at, torch.where(some, grad, 0.0))
        if s["score"] == "sigmoid":
            by_logit = by_score * scores * (1.0 - scores)
        else:
            by_logit = scores * (by_score - (by_score * scores).sum(1, keepdim=True))
        out["grad_logits"] = by_logit.to(s["logits"].dtype)
    return out


def _power(k):
    """2^k as fp32, built from the exponent's bits in 64."""
    return ((k.long() + 1023) << 52).view(torch.float64).float()


def _block_exponents(amax, mode, fmt):
    if fmt == "e4m3":
        return torch.frexp(amax).exponent - 1 - 8
    if mode == "floor":
        return torch.frexp(amax).exponent - 1 - 2
    raw = (amax / 6.0).clamp(min=2.0 ** -30)
    return torch.log2(raw.double()).round().int()  # 64 bits next to a border


def _quantise(x, fmt, mode):
    """Codes [rows, bytes] and E8M0 bytes [rows, blocks] of blocks of 32 along the rows."""
    t, cols = x.shape
    blocks = -(-cols // 32)
    v = torch.zeros(t, blocks * 32, device=x.device)
    v[:, :cols] = x.float()
    v = v.view(t, blocks, 32)
    amax = v.abs().amax(2)
    k = torch.where(amax == 0, -30 if mode == "page" else -127, _block_exponents(amax, mode, fmt).clamp(min=-127))
    y = (v * _power(-k)[:, :, None]).view(t, -1)[:, :cols]
    scales = (k + 127).to(torch.uint8)
    if fmt == "e4m3":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scales
    borders = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=x.device)
    nibble = torch.bucketize(y.abs(), borders, right=True).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    if cols % 2:
        nibble = torch.cat([nibble, nibble.new_zeros(t, 1)], 1)
    return nibble[:, 0::2] + 16 * nibble[:, 1::2], scales


def _to_atoms(scales):
    """A [rows, blocks] scale matrix as atoms of 128 rows x 4 blocks, 512 bytes each; zeros behind its edges."""
    rows, blocks = scales.shape
    r, c = -(-rows // 128), -(-blocks // 4)
    full = scales.new_zeros(r * 128, c * 4)
    full[:rows, :blocks] = scales
    return full.view(r, 4, 32, c, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _from_atoms(flat, rows, k):
    r, c = -(-rows // 128), -(-k // 128)
    full = flat.view(r, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, c * 4)
    return full[:rows, :k // 32]


def _dispatch(s):
    token = s["slots"].long() // s["k"]
    if s["format"] == "values":
        return dict(values=s["x"][token])
    codes, scales = _quantise(s["x"], s["format"], s["mode"])
    return _operand(codes[token], _to_atoms(scales[token]), s["format"])


def _operand(codes, scales, fmt):
    # E4M3 codes and E8M0 scales as the types whose values they are; two E2M1 codes share a byte, which no type spells out
    return dict(codes=codes.view(torch.float8_e4m3fn) if fmt == "e4m3" else codes, scales=scales.view(torch.float8_e8m0fnu))


def _combine(s):
    t, k, cols = s["tokens"], s["k"], s["cols"]
    picked = s["y"][s["rows"].long().view(-1)].float().view(t, k, cols)
    if s["train"]:
        grad = s["grad"].float()
        by_row = torch.empty(t * k, cols, device=grad.device)
        by_row[s["rows"].long().view(-1)] = (s["weights"][:, :, None] * grad[:, None, :]).view(t * k, cols)
        return dict(grad_y=by_row.to(s["y"].dtype), grad_weights=(picked * grad[:, None, :]).sum(2))
    out = (picked * s["weights"][:, :, None]).sum(1)
    return dict(out=(out if s["res"] is None else out + s["res"].float()).to(s["y"].dtype))


def _decode(codes, fmt):
    if fmt == "e4m3":
        return codes.view(torch.float8_e4m3fn).float()
    magnitude = torch.tensor(CODE_MAGNITUDES, device=codes.device)
    table = torch.cat([magnitude, -magnitude])
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)  # byte -> its two values
    return pairs[codes.int()].view(codes.shape[0], -1)


def _dequantise(codes, scales, rows, k, fmt):
    exponent = _from_atoms(scales, rows, k).int() - 127
    return (_decode(codes, fmt).view(rows, k // 32, 32) * _power(exponent)[:, :, None]).view(rows, k)


def _activate(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "swiglu":  # gate and up columns side by side
        gate, up = z[:, 0::2], z[:, 1::2]
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return torch.ones_like(z)


def _linear(s):
    n, k, fmt, act, dt = s["n"], s["k"], s["format"], s["act"], DTYPES[s["out"]]
    a = _dequantise(s["a"], s["a_scales"], s["rows"], k, fmt)
    z = torch.empty(s["rows"], n, device=a.device)
    first = 0
    for e, size in enumerate(s["sizes"]):  # an expert's rows with its own weight
        if size:
            z[first:first + size] = a[first:first + size] @ _dequantise(s["b"][e], s["b_scales"][e], n, k, fmt).T
            if s["bias_values"] is not None:
                z[first:first + size] += s["bias_values"][e]
        first += size
    y = _activate(z, act)
    if s["res"] is not None:
        y = y + s["res"].float()
    out = dict(y=y.to(dt))
    if s["preact"]:
        out["preact"] = z.to(dt)
    return out


def _linear_train(s):
    z, grad = s["z"].float(), s["grad"].float()
    if s["act"] == "swiglu":
        by = torch.empty_like(z)
        by[:, 0::2] = grad * z[:, 1::2] * _slope(z[:, 0::2], "silu")
        by[:, 1::2] = grad * _activate(z[:, 0::2], "silu")
    else:
        by = grad * _slope(z, s["act"])
    parts = [p.sum(0) for p in torch.split(by, s["sizes"])]
    return dict(grad_preact=by.to(s["z"].dtype), grad_bias=torch.stack(parts))


def run(s):
    op = s["op"]
    if own:
        from mxfp4_block_fake_b200 import ops

        if op == "route":
            r = ops.mxfp4_moe_route(s["logits"], s["k"], score=s["score"], bias=s["bias_values"], num_groups=s["groups"],
                                    topk_groups=s["topk_groups"], group_score=s["group_score"], renormalize=s["renorm"],
                                    scale=s["scale"], token_mask=s["token_mask"])
            out = dict(weights=r.weights, experts=r.experts, rows=r.rows, slots=r.slots, counts=r.counts)
            if s["train"]:
                out["grad_logits"] = ops.mxfp4_moe_route_bwd(s["grad"], s["logits"], r.experts, score=s["score"],
                                                             renormalize=s["renorm"], scale=s["scale"])
            return out
        if op == "dispatch":
            if s["format"] == "values":
                return dict(values=ops.mxfp4_moe_dispatch(s["x"], s["rows"]).values)
            r = ops.mxfp4_moe_dispatch(s["x"], s["rows"], emit_values=False, emit_codes=True, elem_format=s["format"],
                                       scale_mode=s["mode"])
            return _operand(r.codes, r.scales, s["format"])
        if op == "combine":
            if s["train"]:
                gy, gw = ops.mxfp4_moe_combine_bwd(s["grad"], s["y"], s["rows"], s["weights"])
                return dict(grad_y=gy, grad_weights=gw)
            return dict(out=ops.mxfp4_moe_combine(s["y"], s["rows"], s["weights"], residual=s["res"]))
        if s["train"]:
            gz, gb = ops.mxfp4_grouped_linear_bwd(s["grad"], s["z"], s["counts"], group_list_type=1, activation=s["act"],
                                                  check=False)
            return dict(grad_preact=gz, grad_bias=gb)
        r = ops.mxfp4_grouped_linear(s["a"], s["a_scales"], s["b"], s["b_scales"], s["counts"], k=s["k"], group_list_type=1,
                                     elem_format=s["format"], bias=s["bias_values"], activation=s["act"], residual=s["res"],
                                     out_dtype=DTYPES[s["out"]], emit_preact=s["preact"], check=False)
        return dict(y=r.y, preact=r.preact) if s["preact"] else dict(y=r.y)
    if op == "route":
        return _route(s)
    if op == "dispatch":
        return _dispatch(s)
    if op == "combine":
        return _combine(s)
    return _linear_train(s) if s["train"] else _linear(s)


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        # logits in; weight, expert, row and slot of each pair and the rows per expert out; the gradient takes the logits again
        moved = t * e * size + t * k * 16 + e * 12
        moved += t * e * size + t * k * 4 if case["train"] else 0
        return {"bytes": moved, "flops": 8 * t * e * (2 if case["train"] else 1)}
    if op in ("dispatch", "combine"):
        t, k, cols = case["tokens"], case["k"], case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "dispatch":
            row = {"values": cols * size, "e2m1": -(-cols // 2) + -(-cols // 32), "e4m3": cols + -(-cols // 32)}[case["format"]]
            return {"bytes": t * cols * size + t * k * (row + 4), "flops": 4 * t * cols}
        moved = t * k * cols * size + t * k * 8 + t * cols * size
        if case["train"]:
            return {"bytes": moved + t * k * cols * size + t * k * 4, "flops": 3 * t * k * cols}
        return {"bytes": moved + (t * cols * size if case["residual"] else 0), "flops": 2 * t * k * cols}
    m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    size = 2 if case["out"] == "bf16" else 4
    width = n // 2 if case["act"] == "swiglu" else n
    if case["train"]:
        return {"bytes": m * (2 * n + width) * size + e * n * 4, "flops": 12 * m * n}
    each = (0.5 if case["format"] == "e2m1" else 1.0) + 1 / 32
    used = min(m, e)  # experts that can have a row
    moved = (m + used * n) * k * each + m * width * size * (2 if case["residual"] else 1)
    moved += used * n * 4 if case["bias"] else 0
    moved += m * n * size if case["preact"] else 0
    return {"bytes": int(moved), "flops": 2 * m * n * k + 10 * m * n}


# ------------------------------------------------------------------------------- the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine, "linear": _exact_linear}[case["op"]](s)


def _exact_route(s):
    x = s["logits"].to(torch.float64)
    score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
    key = score if s["bias_values"] is None else score + s["bias_values"].to(torch.float64)
    t, e = x.shape
    per = e // s["groups"]
    if s["groups"] > 1:
        two = key.view(t, s["groups"], per).topk(min(2, per), 2).values
        rank = two.sum(2) if s["group_score"] == "top2" else two[:, :, 0]
        # a group stays when fewer than topk_groups others are before it: greater, or equal with a lower number
        lower = torch.ones(s["groups"], s["groups"], device=x.device).tril(-1).bool()
        before = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & lower)
        key = key.masked_fill((before.sum(2) >= s["topk_groups"]).repeat_interleave(per, 1), -math.inf)
    chosen = torch.argsort(-key, dim=1, stable=True)[:, :s["k"]]
    live = torch.ones(t, 1, dtype=torch.float64, device=x.device) if s["token_mask"] is None else s["token_mask"].double()[:, None]
    share = torch.take_along_dim(score, chosen, 1)
    norm = share.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(live)
    out = dict(weights=live * s["scale"] * share / norm, experts=None, rows=None, slots=None, counts=None)
    if s["train"]:
        grad = live * s["scale"] * s["grad"].double() / norm
        if s["renorm"]:
            grad = grad - (grad * share / norm).sum(1, keepdim=True)
        if s["score"] == "sigmoid":
            out["grad_logits"] = torch.zeros_like(score).scatter_(1, chosen, grad * share * torch.sigmoid(-torch.take_along_dim(x, chosen, 1)))
        else:
            out["grad_logits"] = -score * (grad * share).sum(1, keepdim=True)
            out["grad_logits"].scatter_add_(1, chosen, grad * share)
    return out


def _exact_dispatch(s):
    """Codes by the nearest value of the format, scales from the definition; E2M1 codes share bytes and have no value of their own."""
    token = s["slots"].long().div(s["k"], rounding_mode="floor")
    if s["format"] == "values":
        return dict(values=s["x"].double()[token])
    x = s["x"].double()
    t, cols = x.shape
    pad = -cols % 32
    top = torch.nn.functional.pad(x, (0, pad)).abs().reshape(t, -1, 32).max(2).values
    drop = {"e4m3": 8, "e2m1": 2}[s["format"]]
    if s["mode"] == "floor":
        near = torch.log2(top.clamp(min=2.0 ** -140)).round()
        k = (near - (torch.exp2(near) > top).double()).clamp(min=-127.0 + drop) - drop
    else:
        k = torch.log2((top.float() / 6.0).double().clamp(min=2.0 ** -30)).round()
    scale = torch.exp2(k)
    rows, blocks = t * s["k"], k.shape[1]
    flat = torch.zeros(-(-rows // 128) * 128, -(-blocks // 4) * 4, dtype=torch.float64, device=x.device) + 2.0 ** -127
    flat[:rows, :blocks] = scale[token]
    r, c = torch.meshgrid(torch.arange(flat.shape[0], device=x.device), torch.arange(flat.shape[1], device=x.device), indexing="ij")
    atom = (r // 128) * (flat.shape[1] // 4) + c // 4
    place = 512 * atom + 16 * (r % 32) + 4 * (r % 128 // 32) + c % 4
    scales = torch.empty(flat.numel(), dtype=torch.float64, device=x.device)
    scales[place.reshape(-1)] = flat.reshape(-1)
    codes = None
    if s["format"] == "e4m3":
        y = x / scale.repeat_interleave(32, 1)[:, :cols]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
        codes = (torch.round(y / step) * step).clamp(-448.0, 448.0)[token]
    return dict(codes=codes, scales=scales)


def _exact_combine(s):
    t, k, cols = s["tokens"], s["k"], s["cols"]
    w, rows = s["weights"].double(), s["rows"].long()
    if s["train"]:
        grad = s["grad"].double()
        slot = s["slots"].long()
        grad_y = w.reshape(-1)[slot][:, None] * grad[slot // k]
        return dict(grad_y=grad_y, grad_weights=torch.stack([(s["y"][rows[:, j]].double() * grad).sum(1) for j in range(k)], 1))
    out = torch.zeros(t, cols, dtype=torch.float64, device=w.device) if s["res"] is None else s["res"].double()
    for j in range(k):
        out = out + w[:, j, None] * s["y"][rows[:, j]].double()
    return dict(out=out)


def _exact_values(codes, scales, rows, k, fmt):
    """Values from the codes' bit fields, scales from their places in the atoms."""
    if fmt == "e2m1":
        c = torch.stack([codes & 15, codes >> 4], 2).reshape(rows, k).long()
        sign, e, m, bits, low = c >> 3, (c >> 1) & 3, c & 1, 1, 0
    else:
        c = codes.long()
        sign, e, m, bits, low = c >> 7, (c >> 3) & 15, c & 7, 3, -6
    lead = (e > 0).double()
    value = (lead + m.double() / 2 ** bits) * torch.exp2((e - (1 if low == 0 else 7)).clamp(min=low).double())
    value = torch.where(sign == 1, -value, value)
    r = torch.arange(rows, device=codes.device)[:, None]
    b = torch.arange(k // 32, device=codes.device)[None, :]
    place = 512 * ((r // 128) * (-(-k // 128)) + b // 4) + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    return value * torch.exp2(scales[place].double() - 127.0).repeat_interleave(32, 1)


def _exact_linear(s):
    act = s["act"]
    if s["train"]:
        with torch.enable_grad():
            z = s["z"].double().requires_grad_(True)
            (grad_z,) = torch.autograd.grad(_exact_activate(z, act), z, s["grad"].double())
        ends = torch.cumsum(s["counts"], 0).tolist()
        starts = [0] + ends[:-1]
        return dict(grad_preact=grad_z, grad_bias=torch.stack([grad_z[p:q].sum(0) for p, q in zip(starts, ends)]))
    m, n, k, fmt = s["rows"], s["n"], s["k"], s["format"]
    a = _exact_values(s["a"], s["a_scales"], m, k, fmt)
    z = torch.zeros(m, n, dtype=torch.float64, device=a.device)
    ends = torch.cumsum(s["counts"], 0).tolist()
    for e, end in enumerate(ends):
        at = slice(ends[e - 1] if e else 0, end)
        if at.start < at.stop:
            z[at] = torch.mm(a[at], _exact_values(s["b"][e], s["b_scales"][e], n, k, fmt).t())
            if s["bias_values"] is not None:
                z[at] += s["bias_values"][e].double()
    y = _exact_activate(z, act)
    out = dict(y=y if s["res"] is None else y + s["res"].double())
    if s["preact"]:
        out["preact"] = z
    return out


def _exact_activate(z, act):
    f = torch.nn.functional
    if act == "swiglu":
        pair = z.view(z.shape[0], -1, 2)
        return f.silu(pair[:, :, 0]) * pair[:, :, 1]
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
            "silu": f.silu}[act](z)
