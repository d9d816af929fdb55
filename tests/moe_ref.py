"""Plain 64-bit forms of the mixture-of-experts operators, for their tests
(include/mxfp4.h): written token by token from the definitions."""
from __future__ import annotations

import math

import torch


def score_row(x: list[float], score: str) -> list[float]:
    if score == "sigmoid":
        return [1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v) for v in x]
    m = max(x)
    if m == -math.inf:
        return [0.0] * len(x)
    e = [math.exp(v - m) for v in x]
    s = math.fsum(e)
    return [v / s for v in e]


def route(logits, k, score="softmax", bias=None, num_groups=1, topk_groups=None, group_score="top2", renormalize=True,
          scale=1.0, token_mask=None):
    """(weights [t][k], experts [t][k]) as lists."""
    weights, experts = [], []
    b = None if bias is None else bias.double().tolist()
    for t, x in enumerate(logits.double().tolist()):
        n = len(x)
        if token_mask is not None and not bool(token_mask[t]):
            weights.append([0.0] * k)
            experts.append([-1] * k)
            continue
        if any(math.isnan(v) or v == math.inf for v in x):
            weights.append([math.nan] * k)
            experts.append(list(range(k)))
            continue
        s = score_row(x, score)
        key = {}
        for e in range(n):
            if x[e] == -math.inf or (b is not None and not math.isfinite(b[e])):
                continue
            key[e] = s[e] + (0.0 if b is None else b[e])
        if num_groups > 1:
            per = n // num_groups
            rank = {}
            for g in range(num_groups):
                inside = sorted((key[e] for e in range(g * per, (g + 1) * per) if e in key), reverse=True)
                if inside:
                    rank[g] = inside[0] + (inside[1] if group_score == "top2" and len(inside) > 1 else 0.0)
            keep = sorted(rank, key=lambda g: (-rank[g], g))[: (topk_groups or num_groups)]
            key = {e: v for e, v in key.items() if e // per in keep}
        chosen = sorted(key, key=lambda e: (-key[e], e))[:k]
        total = math.fsum(s[e] for e in chosen) if renormalize else 1.0
        w = [scale * s[e] / total for e in chosen]
        weights.append(w + [0.0] * (k - len(w)))
        experts.append(chosen + [-1] * (k - len(chosen)))
    return weights, experts


def plan(experts, count):
    """(rows, slots, counts) of a table of experts."""
    k = len(experts[0]) if experts else 0
    pairs = sorted((e, t, j) for t, row in enumerate(experts) for j, e in enumerate(row) if e >= 0)
    rows = [[-1] * k for _ in experts]
    slots = [-1] * (len(experts) * k)
    counts = [0] * count
    for r, (e, t, j) in enumerate(pairs):
        rows[t][j] = r
        slots[r] = t * k + j
        counts[e] += 1
    return rows, slots, counts


def route_weights(x: torch.Tensor, experts: torch.Tensor, score, renormalize, scale):
    """The chosen experts' weights as a differentiable function of the logits (64 bits)."""
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    some = experts >= 0
    w = torch.where(some, torch.take_along_dim(s, experts.long().clamp(min=0), 1), 0.0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return scale * w


def activation(z: torch.Tensor, act: str) -> torch.Tensor:
    f = torch.nn.functional
    if act == "swiglu":
        return f.silu(z[:, 0::2]) * z[:, 1::2]
    return {"none": lambda v: v, "relu": torch.relu, "gelu": f.gelu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"), "silu": f.silu}[act](z)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def decode(codes: torch.Tensor, scales: torch.Tensor, rows: int, k: int, fmt: str) -> torch.Tensor:
    """Operand codes [rows, bytes] and MMA-layout scales -> float64 [rows, k]."""
    if fmt == "e2m1":
        table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
        v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], 2).reshape(rows, -1)[:, :k]
    else:
        v = codes.view(torch.float8_e4m3fn).double()[:, :k]
    nblk = -(-k // 32)
    r = torch.arange(rows)[:, None]
    b = torch.arange(nblk)[None, :]
    at = 512 * ((r // 128) * (-(-nblk // 4)) + b // 4) + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    s = torch.exp2(scales.reshape(-1)[at].double() - 127.0)
    return v * s.repeat_interleave(32, 1)[:, :k]
