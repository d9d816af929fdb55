"""GPU checks of the mixture-of-experts operators against their definitions in
64 bits (tests/moe_ref.py) and against the oracle's quantiser.

Tolerances count roundings of half a step: fp32 2^-24, bf16 2^-8 relative to
the value. The bounds are written beside each check.
"""
from __future__ import annotations

import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as O
from mxfp4_block_fake_b200 import MXFP4ArgumentError, ops
from tests import moe_ref as R
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(*shape, seed=0, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen(seed)) * std).to(dtype)


def close(got, want, bound, what=""):
    got, want = got.detach().double().cpu(), want.double()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand_as(want)
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    err = torch.where(torch.isnan(want), 0.0, (got - want).abs())
    worst = (err / (bound + 1e-300)).max() if err.numel() else torch.tensor(0.0)
    assert bool((err <= bound + 1e-300).all()), f"{what}: error / bound {float(worst):.3g}"


# ---------------------------------------------------------------------------- routing

def check_route(x, k, token_mask=None, bias=None, **kw):
    """x: CPU logits. Experts and the order exactly, weights within the fp32
    evaluation: a score is an exponential of x - m (or x), whose rounding
    moves it by |x - m| 2^-24 relative, at most 2 ulp of expf, a sum of at
    most E terms in a tree of E/32 + 5 additions, and three more operations."""
    dev = "cuda"
    r = ops.mxfp4_moe_route(x.to(dev), k, token_mask=None if token_mask is None else token_mask.to(dev),
                            bias=None if bias is None else bias.to(dev), **kw)
    weights, experts = R.route(x, k, token_mask=token_mask, bias=bias, **kw)
    e = x.shape[1]
    rows, slots, counts = R.plan(experts, e)
    t = x.shape[0]
    assert r.experts.cpu().tolist() == experts
    assert r.rows.cpu().tolist() == rows and r.slots.cpu().tolist() == slots and r.counts.cpu().tolist() == counts
    w = torch.tensor(weights, dtype=torch.float64).view(t, k)
    spread = x.double().nan_to_num(0.0, 0.0, 0.0).abs().max().item() * 2 if x.numel() else 0.0
    close(r.weights, w, (spread + 2 * 4 + e / 32 + 5 + 8) * U32 * w.nan_to_num(0.0).abs(), "weights")
    return r


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 256, 8), (3, 7, 7), (64, 60, 4), (65, 33, 2), (200, 1024, 32), (333, 64, 6)])
def test_route(dtype, score, renormalize, tokens, experts, k):
    x = rnd(tokens, experts, seed=tokens, std=1.5, dtype=DT[dtype])
    check_route(x, k, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("group_score", ["top2", "max"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,topk_groups,k", [(256, 8, 4, 8), (60, 4, 2, 5), (32, 32, 3, 3), (96, 3, 1, 7), (264, 8, 8, 8),
                                                          (1024, 2, 1, 4), (160, 5, 3, 6)])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_groups(group_score, score, experts, groups, topk_groups, k, with_bias):
    x = rnd(130, experts, seed=experts, std=1.5)
    bias = rnd(experts, seed=5, std=0.05) if with_bias else None
    check_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=topk_groups, group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_special_rows(score, groups, with_bias):
    """Ties, closed experts, rows without any, NaN and +inf, masked rows that hold them."""
    e, k = 40, 6
    x = rnd(100, e, seed=3, dtype=torch.bfloat16).float()
    x[0] = 0.0                       # all equal: the lowest experts
    x[1] = -torch.inf                # nothing is open
    x[2, :37] = -torch.inf           # three open experts
    x[3, 11] = torch.nan
    x[4, 39] = torch.inf
    x[5] = -120.0                    # scores that underflow in fp32 next to 1
    x[5, 7] = -119.0
    x[6, ::2] = x[6, 1::2]           # pairs of equals
    x[7] = 3.0e38
    x[8] = -3.0e38 if score == "softmax" else -80.0
    x[9] = torch.nan
    x[10, 1:] = -torch.inf
    x[11] = 1.0e-42                  # subnormals
    mask = torch.ones(100, dtype=torch.bool)
    mask[9] = mask[20:25] = mask[99] = False
    bias = None
    if with_bias:
        bias = rnd(e, seed=4, std=0.02)
        bias[3], bias[5], bias[30] = torch.nan, torch.inf, -torch.inf
    for renormalize in (True, False):
        check_route(x, k, token_mask=mask, score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2),
                    renormalize=renormalize)


def test_route_near_ties_are_decided_in_64_bits():
    """Keys s + b that fp32 cannot tell apart: b is set so that neighbours' keys
    differ by 1e-9 (fp32 steps near 0.5 are 6e-8)."""
    e, k = 64, 8
    x = rnd(256, e, seed=9, std=0.5)
    # the same logits in every token, in a different order of the experts
    base = x[0].double()
    s = torch.sigmoid(base)
    order = torch.randperm(e, generator=gen(1))
    want = torch.empty(e, dtype=torch.float64)
    want[order] = 0.6 + 1e-9 * torch.arange(e, dtype=torch.float64)
    bias = (want - s).float()        # fp32: the keys now differ by its rounding, about 1e-9 to 1e-8
    x[:] = x[0]
    x[1::2] += rnd(128, e, seed=10, std=1e-7)
    check_route(x, k, score="sigmoid", bias=bias)
    check_route(x, k, score="sigmoid", bias=bias, num_groups=8, topk_groups=3)
    check_route(x, k, score="softmax", bias=(0.6 - torch.softmax(base, 0) + 1e-9 * order.double()).float(), num_groups=4, topk_groups=2)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias_kind", ["none", "zero", "small", "some"])
@pytest.mark.parametrize("experts,groups,topk_groups,k", [(256, 1, 1, 8), (256, 8, 4, 8), (60, 4, 3, 6), (1000, 10, 4, 12), (512, 32, 5, 9), (64, 1, 1, 32)])
def test_route_choice_of_many_tokens(dtype, score, bias_kind, experts, groups, topk_groups, k):
    """The choice against 64-bit keys sorted stably, over enough tokens that
    neighbouring keys come close to one another (and, in bf16, coincide)."""
    t = 6000
    x = rnd(t, experts, seed=21, std=1.0, dtype=DT[dtype]).cuda()
    bias = {"none": None, "zero": torch.zeros(experts), "small": rnd(experts, seed=22, std=1e-3),
            "some": (torch.arange(experts) % 3 == 0).float() * 0.01}[bias_kind]
    v = x.double()
    key = torch.sigmoid(v) if score == "sigmoid" else torch.softmax(v, 1)
    if bias is not None:
        bias = bias.cuda()
        key = key + bias.double()
    if groups > 1:
        by = key.view(t, groups, -1)
        rank = by.topk(2, 2).values.sum(2)
        keep = torch.zeros(t, groups, dtype=torch.bool, device="cuda").scatter_(1, rank.sort(dim=1, descending=True, stable=True).indices[:, :topk_groups], True)
        key = torch.where(keep[:, :, None], by, -torch.inf).view(t, experts)
    want = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    r = ops.mxfp4_moe_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=topk_groups)
    # softmax in 64 bits may round two different logits' keys to one only where they are 2^-52 apart: none here
    assert torch.equal(r.experts.long(), want)


def test_route_shared_memory_near_its_default_limit():
    """Calls whose shared memory is just below the size that a kernel may have
    without asking for more, each the first of its kernel in a new process."""
    code = """
import torch
from mxfp4_block_fake_b200 import ops
for dtype in (torch.float32, torch.bfloat16):
    for score in ("softmax", "sigmoid"):
        for experts, k in [(640, 24)] + [(e, k) for e in range(600, 700, 3) for k in (1, 16, 31)]:
            x = torch.randn(70, experts, generator=torch.Generator().manual_seed(experts)).to(dtype).cuda()
            want = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
            assert torch.equal(ops.mxfp4_moe_route(x, k, score=score).experts.long(), want), (dtype, score, experts, k)
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.parametrize("tokens", [0, 1, 64, 65, 2048, 2049, 5000])
def test_route_order_of_many_tokens(tokens):
    """The expert-sorted order against a stable sort (experts from the call)."""
    e, k = 48, 4
    x = rnd(tokens, e, seed=2, std=2.0).cuda()
    mask = (torch.rand(tokens, generator=gen(7)) > 0.3).cuda()
    r = ops.mxfp4_moe_route(x, k, token_mask=mask)
    flat = r.experts.reshape(-1).long()
    total = int((flat >= 0).sum())
    key = torch.where(flat < 0, e, flat)
    order = torch.sort(key, stable=True).indices[:total]
    assert torch.equal(r.slots[:total].long(), order) and bool((r.slots[total:] == -1).all())
    rows = torch.full_like(flat, -1)
    rows[order] = torch.arange(total, device="cuda")
    assert torch.equal(r.rows.reshape(-1).long(), rows)
    assert torch.equal(r.counts, torch.bincount(key, minlength=e + 1)[:e])
    assert torch.equal(torch.sort(r.experts[mask], 1).values, torch.sort(torch.topk(x[mask], k, 1).indices.int(), 1).values)


def test_route_strided_logits_and_repeatability():
    big = rnd(130, 90, seed=8, dtype=torch.bfloat16).cuda()
    x = big[:, 3:63]
    a = ops.mxfp4_moe_route(x, 5)
    b = ops.mxfp4_moe_route(x.contiguous(), 5)
    c = ops.mxfp4_moe_route(big.t().contiguous().t()[:, 3:63], 5)
    for f in ("weights", "experts", "rows", "slots", "counts"):
        assert torch.equal(getattr(a, f), getattr(b, f)) and torch.equal(getattr(a, f), getattr(c, f))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (5, 7, 7), (70, 256, 8), (33, 1000, 32)])
def test_route_backward(dtype, score, renormalize, tokens, experts, k):
    """Against autograd of the formula in 64 bits. With c = scale and G = max
    |g| a gradient is a sum of at most k + 1 products of scores (<= 1) and c g;
    every factor carries the weights' relative error."""
    x = rnd(tokens, experts, seed=11, std=1.5, dtype=DT[dtype])
    g = rnd(tokens, k, seed=12)
    chosen = torch.topk(x.double(), k, 1).indices.int()
    if tokens > 4:
        chosen[1] = -1                 # a token without experts
        chosen[2, k // 2:] = -1        # a token with fewer
    scale = 1.5
    got = ops.mxfp4_moe_route_bwd(g.cuda(), x.cuda(), chosen.cuda(), score=score, renormalize=renormalize, scale=scale)
    v = x.double().requires_grad_(True)
    w = R.route_weights(v, chosen, score, renormalize, scale)
    (want,) = torch.autograd.grad(w, v, g.double())
    top = scale * g.abs().double().amax(1, keepdim=True) * (2 if renormalize else 1)
    unit = (2 * 2 * x.double().abs().max().item() + 2 * 8 + 2 * (experts / 32 + 5) + k + 12) * U32
    # every gradient entry is at most top; its terms' errors are unit * top each
    close(got, want, 2 * unit * top + (U16 * want.abs() if dtype == "bf16" else U32 * want.abs()), "grad_logits")


def test_route_backward_against_differences():
    x = rnd(6, 20, seed=13)
    chosen = torch.topk(x, 3, 1).indices.int()
    g = rnd(6, 3, seed=14)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            got = ops.mxfp4_moe_route_bwd(g.cuda(), x.cuda(), chosen.cuda(), score=score, renormalize=renormalize).cpu().double()
            h = 1e-5
            for e in range(20):
                d = torch.zeros(20, dtype=torch.float64)
                d[e] = h
                up = (R.route_weights(x.double() + d, chosen, score, renormalize, 1.0) * g).sum(1)
                down = (R.route_weights(x.double() - d, chosen, score, renormalize, 1.0) * g).sum(1)
                # central differences: h^2 times a third derivative below 10 max|g|, and 1e-16 / h of rounding
                assert ((up - down) / (2 * h) - got[:, e]).abs().max() < 1e-5


def test_route_backward_special_rows():
    x = rnd(6, 16, seed=15)
    x[0, 3] = torch.nan
    x[1, 4] = torch.inf
    x[2, 5:] = -torch.inf
    x[3] = torch.nan
    chosen = torch.topk(x.nan_to_num(0.0), 2, 1).indices.int()
    chosen[3] = -1
    chosen[4] = 7                        # the same expert twice: the sum of both
    g = rnd(6, 2, seed=16)
    for score in ("softmax", "sigmoid"):
        got = ops.mxfp4_moe_route_bwd(g.cuda(), x.cuda(), chosen.cuda(), score=score, renormalize=False).cpu()
        assert bool(torch.isnan(got[0]).all()) and bool(torch.isnan(got[1]).all()) and bool((got[3] == 0).all())
        assert bool((got[2, 5:] == 0).all()) and bool(torch.isfinite(got[2]).all())
        v = x[4:5].double().requires_grad_(True)
        (want,) = torch.autograd.grad(R.route_weights(v, chosen[4:5], score, False, 1.0), v, g[4:5].double())
        close(got[4:5], want, 64 * U32 * g[4].abs().sum().double(), "twice")
    wild = chosen.clone()
    wild[5] = 99                         # outside the experts: ignored
    got = ops.mxfp4_moe_route_bwd(g.cuda(), x.cuda(), wild.cuda(), renormalize=True).cpu()
    assert bool((got[5] == 0).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("constant_bias", [False, True])
@pytest.mark.parametrize("experts,groups", [(24, 1), (64, 4), (256, 1), (256, 8), (1000, 10)])
@pytest.mark.parametrize("k", [1, 5])
def test_route_zeros_of_both_signs(dtype, constant_bias, experts, groups, k):
    """+0.0 and -0.0 are equal logits: the lower expert comes first, inside the
    choice, at its end, and between lanes."""
    g = gen(experts + k)
    x = -torch.rand(160, experts, generator=g).to(DT[dtype]) - 1.0
    share = torch.linspace(0.0, 1.0, 160)[:, None] ** 3
    zero = torch.rand(160, experts, generator=g) < share
    sign = torch.rand(160, experts, generator=g) < 0.5
    x = torch.where(zero, torch.where(sign, -0.0, 0.0).to(x.dtype), x)
    x[0] = -1.0
    x[0, 3], x[0, 20] = -0.0, 0.0
    x[1] = -0.0
    x[1, -1] = 0.0
    bias = torch.full((experts,), 0.25) if constant_bias else None
    for score in ("softmax", "sigmoid"):
        check_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2))
        check_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=max(1, groups // 2), group_score="max")


@pytest.mark.parametrize("experts", [64, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("p", [0.942, 0.76, 0.6])
def test_route_key_left_out_with_a_large_score(experts, score, p):
    """An expert whose large score its bias takes back to a key near 0 (so its
    key's error is that of the score), against a last choice of a small score, with
    a third expert of a small score and key between the two in fp32."""
    high, fill, third, last = 5, 6, 7, experts - 3
    one = math.log(p / (1 - p))
    step = 2.0 ** (math.floor(math.log2(one)) - 23)
    at = one + step * torch.arange(-90, 91, dtype=torch.float64)
    small = torch.logspace(-7.4, -6.4, 33, dtype=torch.float64)
    x = torch.full((at.numel(), small.numel(), experts), -60.0, dtype=torch.float64)
    x[:, :, high] = at[:, None]
    # softmax: the fill's logit 0 and the high one's make p; sigmoid: each by itself
    x[:, :, fill] = 0.0
    total = math.log(1 / (1 - p)) if score == "softmax" else 0.0
    x[:, :, last] = small.log()[None, :] + total
    x[:, :, third] = math.log(1e-9) + total
    x = x.view(-1, experts).float()
    bias = torch.zeros(experts)
    bias[high], bias[fill] = -p, -2.0
    v = x.cuda().double()
    key = (torch.sigmoid(v) if score == "sigmoid" else torch.softmax(v, 1)) + bias.cuda().double()
    for k in (1, 2):
        want = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
        r = ops.mxfp4_moe_route(x.cuda(), k, score=score, bias=bias.cuda())
        assert torch.equal(r.experts.long(), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups", [(32, 4), (256, 8), (60, 5)])
def test_route_group_ranks_past_fp32(score, experts, groups):
    """Groups whose two best keys add up to more than fp32 holds."""
    per = experts // groups
    bias = torch.zeros(experts)
    for g in range(groups):
        bias[g * per], bias[g * per + 1] = (2.0 + 0.1 * g) * 1e38, (1.9 + 0.1 * g) * 1e38
    x = rnd(70, experts, seed=31)
    for topk_groups in (1, groups - 1):
        for k in (1, 2):
            check_route(x, k, score=score, bias=bias, num_groups=groups, topk_groups=topk_groups)
            check_route(x, k, score=score, bias=-bias, num_groups=groups, topk_groups=topk_groups)


# ------------------------------------------------------------------ dispatch and combine

def a_plan(tokens, experts, k, seed=0, masked=0.0):
    g = gen(seed)
    chosen = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)]).int() if tokens else torch.zeros(0, k, dtype=torch.int32)
    if masked and tokens:
        chosen[torch.rand(tokens, generator=g) < masked] = -1
        chosen[torch.rand(tokens, generator=g) < masked, -1] = -1
    rows, slots, counts = R.plan(chosen.tolist(), experts)
    return (torch.tensor(rows, dtype=torch.int32).view(tokens, k), torch.tensor(slots, dtype=torch.int32),
            torch.tensor(counts, dtype=torch.int64))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 1), (5, 3, 64), (130, 8, 96), (67, 2, 1001), (33, 4, 7168)])
def test_dispatch_values(dtype, tokens, k, cols):
    rows, slots, _ = a_plan(tokens, 12, k, masked=0.2)
    x = rnd(tokens, cols, seed=1, dtype=DT[dtype])
    out = torch.full((tokens * k + 3, cols), 7.0, dtype=DT[dtype], device="cuda")
    r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), row_count=tokens * k + 3, out=ops.DispatchResult(values=out))
    want = torch.full_like(out, 7.0).cpu()          # rows that no index names stay
    total = int((slots >= 0).sum())
    want[:total] = x[slots[:total].long() // k]
    assert torch.equal(r.values.cpu(), want)


@pytest.mark.parametrize("fmt,mode", [("e2m1", "page"), ("e2m1", "floor"), ("e4m3", "floor")])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 32), (3, 8, 128), (70, 3, 4128), (40, 2, 77), (9, 1, 7168), (50, 5, 192), (20, 3, 33)])
def test_dispatch_quantised(fmt, mode, dtype, tokens, k, cols):
    """Byte for byte the oracle's row-wise quantisation of the token's row, in
    the rows the plan names; other rows and their scales stay."""
    rows, slots, _ = a_plan(tokens, 10, k, seed=3, masked=0.2 if tokens > 5 else 0.0)
    x = rnd(tokens, cols, seed=2, std=3.0)
    x[:, ::17] *= 1000.0
    if cols > 60:
        x[0, :32] = 0.0
        x[-1, 32:64] = 1e-39
    if tokens > 30:
        x[11, 5], x[12, 6], x[13, 7] = torch.nan, torch.inf, -torch.inf
        x[14, 1:40] = -0.0
        x[15] *= 1e-30
        x[16, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)[: min(32, cols)]   # ties
        x[17] *= 1e34 if dtype == "fp32" else 1e30
    x = x.to(DT[dtype])
    n = tokens * k
    width = cols if fmt == "e4m3" else (cols + 1) // 2
    codes = torch.full((n, width), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ops.scales_row_bytes(n, cols, 32, "mma"),), 0x5A, dtype=torch.uint8, device="cuda")
    ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), elem_format=fmt, scale_mode=mode, out=ops.DispatchResult(codes=codes, scales=scales))
    bits = x.view(torch.int16).numpy().view(np.uint16) if dtype == "bf16" else x.numpy()
    q = O.qdq8_rowwise(bits) if fmt == "e4m3" else O.qdq_rowwise(bits, 32, 6.0, O.SCALE_PAGE if mode == "page" else O.SCALE_FLOOR)
    total = int((slots >= 0).sum())
    token = (slots[:total].long() // k).numpy()
    want = np.full((n, width), 0xA5, np.uint8)
    want[:total] = q["codes"][token]
    assert np.array_equal(codes.cpu().numpy(), want)
    nblk = -(-cols // 32)
    full = np.full((-(-n // 128) * 128, -(-nblk // 4) * 4), 0x5A, np.uint8)
    full[n:] = 0                                   # padding is written as zero ...
    full[:total, :nblk] = q["scales"][token]
    full[:total, nblk:] = 0                        # ... also behind the last block of a written row
    assert np.array_equal(scales.cpu().numpy(), O.mma_scale_layout(full).reshape(-1))


@pytest.mark.parametrize("scale_factor", [1.0, 6.0, 20.0, 2.0 ** -70])
def test_dispatch_scale_factors(scale_factor):
    """The whole PAGE rule, also outside the range of the divide-free threshold."""
    x = rnd(33, 256, seed=6, std=2.0, dtype=torch.bfloat16)
    rows = torch.arange(33, dtype=torch.int32).view(33, 1)
    r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), emit_values=False, emit_codes=True, scale_factor=scale_factor)
    q = O.qdq_rowwise(x.view(torch.int16).numpy().view(np.uint16), 32, scale_factor, O.SCALE_PAGE)
    assert np.array_equal(r.codes.cpu().numpy(), q["codes"])
    got = ops.mxfp4_qdq_fwd(x.cuda(), emit_codes=True, scale_factor=scale_factor, scales_layout="mma")
    nb = 512 * 2
    assert torch.equal(r.codes, got.codes_row) and torch.equal(r.scales[:nb], got.scales_row[:nb])


def test_dispatch_every_bf16_value():
    """Every bf16 value beside amaxes that put it in every binade of the format."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    rows_of = [v.float().abs().clamp(min=1e-37) * s for s in (1.0, 2.7, 5.0, 6.5)]
    x = torch.cat([torch.stack([torch.cat([v[i:i + 1], a[i:i + 1].bfloat16()]).repeat(16) for i in range(0, v.numel(), 37)]) for a in rows_of])
    x = x[torch.isfinite(x.float()).all(1)]
    rows = torch.arange(x.shape[0], dtype=torch.int32).view(-1, 1)
    for mode, code in (("page", O.SCALE_PAGE), ("floor", O.SCALE_FLOOR)):
        r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), emit_values=False, emit_codes=True, scale_mode=mode)
        q = O.qdq_rowwise(x.view(torch.int16).numpy().view(np.uint16), 32, 6.0, code)
        assert np.array_equal(r.codes.cpu().numpy(), q["codes"])


@pytest.mark.parametrize("fmt,dtype", [("e2m1", "bf16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_dispatch_of_many_rows(fmt, dtype, masked):
    """Large enough for the scales' second kernel; odd row and block counts, rows left out."""
    tokens, k, cols = 1400, 8, 6176          # 193 blocks: the last atom column holds one
    rows, slots, _ = a_plan(tokens, 20, k, seed=3, masked=masked)
    x = rnd(tokens, cols, seed=2, std=3.0, dtype=DT[dtype])
    n = tokens * k + 5
    assert ops._abi.lib().mxfp4_moe_dispatch_workspace(tokens, k, cols, n) > 0
    width = cols if fmt == "e4m3" else cols // 2
    codes = torch.full((n, width), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ops.scales_row_bytes(n, cols, 32, "mma"),), 0x5A, dtype=torch.uint8, device="cuda")
    ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), elem_format=fmt, scale_mode="floor", row_count=n, out=ops.DispatchResult(codes=codes, scales=scales))
    q = ops.mxfp4_qdq_fwd(x.cuda(), emit_values=False, emit_codes=True, elem_format=fmt, scale_mode="floor")   # checked against the oracle elsewhere
    total = int((slots >= 0).sum())
    token = (slots[:total].long() // k).cuda()
    assert torch.equal(codes[:total], q.codes_row[token]) and bool((codes[total:] == 0xA5).all())
    nblk = cols // 32
    full = np.full((-(-n // 128) * 128, -(-nblk // 4) * 4), 0x5A, np.uint8)
    full[n:] = 0
    full[:total, :nblk] = q.scales_row[token].cpu().numpy()
    full[:total, nblk:] = 0
    assert np.array_equal(scales.cpu().numpy(), O.mma_scale_layout(full).reshape(-1))


def test_dispatch_fp32_values_beside_the_ties():
    """fp32 values one step below, at and above every midpoint and code, both signs, at several scales."""
    base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    near = torch.cat([base, torch.nextafter(base, torch.tensor(0.0)), torch.nextafter(base, torch.tensor(9.0))])
    v = torch.cat([near, -near])
    x = torch.stack([torch.cat([v[i:i + 31].roll(0), torch.tensor([6.0])]) if i + 31 <= v.numel() else torch.cat([v[-31:], torch.tensor([6.0])])
                     for i in range(0, v.numel(), 31)])
    x = torch.cat([x * 2.0 ** e for e in (-120, -60, -3, 0, 5, 100)])
    rows = torch.arange(x.shape[0], dtype=torch.int32).view(-1, 1)
    for mode, code in (("page", O.SCALE_PAGE), ("floor", O.SCALE_FLOOR)):
        r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), emit_values=False, emit_codes=True, scale_mode=mode)
        assert np.array_equal(r.codes.cpu().numpy(), O.qdq_rowwise(x.numpy(), 32, 6.0, code)["codes"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", [32, 64, 96, 77])
def test_dispatch_values_whose_codes_underflow(dtype, cols):
    """Negative values so far below a block's largest that their quotient by
    the scale rounds to zero (code 0, as in the quantiser), or nearly does, and
    scale factors whose quotients exceed fp32."""
    tops = [100.0, 6.0, 1e34, 1e37, 3.0e38, 2.0 ** 100, 2.0 ** -100, 2.0 ** 17, 2.0 ** 20]
    tiny = [2.0 ** -149, 2.0 ** -133, 2.0 ** -140, 1e-39, 2.0 ** -126, 1e-20, 1e-10, 0.0]
    x = torch.zeros(len(tops) * len(tiny), cols, dtype=torch.float64)
    for i, top in enumerate(tops):
        for j, low in enumerate(tiny):
            row = x[i * len(tiny) + j]
            row[0::32] = top
            row[1::32], row[2::32], row[3::32], row[4::32] = -low, low, -top * 2.0 ** -126, -top * 2.0 ** -3
            row[5::32], row[6::32] = -3 * low, -0.0
    x = x.float().to(DT[dtype])
    rows = torch.arange(x.shape[0], dtype=torch.int32).view(-1, 1)
    bits = x.view(torch.int16).numpy().view(np.uint16) if dtype == "bf16" else x.numpy()
    for mode, code, factor in (("page", O.SCALE_PAGE, 6.0), ("floor", O.SCALE_FLOOR, 6.0), ("page", O.SCALE_PAGE, 3.3e38), ("page", O.SCALE_PAGE, 1e-30)):
        r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), emit_values=False, emit_codes=True, scale_mode=mode, scale_factor=factor)
        assert np.array_equal(r.codes.cpu().numpy(), O.qdq_rowwise(bits, 32, factor, code)["codes"]), (mode, factor)
    r = ops.mxfp4_moe_dispatch(x.cuda(), rows.cuda(), emit_values=False, emit_codes=True, elem_format="e4m3", scale_mode="floor")
    assert np.array_equal(r.codes.cpu().numpy(), O.qdq8_rowwise(bits)["codes"])


def test_dispatch_skips_rows_outside_and_strides():
    x = rnd(10, 100, seed=4, dtype=torch.bfloat16).cuda()[:, 1:97]
    rows = torch.arange(20, dtype=torch.int32).view(10, 2)
    rows[3, 1], rows[4, 0], rows[5, 0] = 20, -7, 2 ** 31 - 1
    out = torch.zeros(20, 100, dtype=torch.bfloat16, device="cuda")[:, :96]
    ops.mxfp4_moe_dispatch(x, rows.cuda(), out=ops.DispatchResult(values=out))
    want = torch.zeros(20, 96, dtype=torch.bfloat16)
    for t in range(10):
        for j in range(2):
            if 0 <= rows[t, j] < 20:
                want[rows[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 1), (4, 8, 64), (130, 6, 96), (67, 2, 1001), (19, 32, 40), (33, 4, 7168)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(dtype, tokens, k, cols, residual, weighted):
    """fp32 sums of k products (k roundings of the sums, k of the products
    fused away) and the residual, then one rounding."""
    rows, _, _ = a_plan(tokens, 40, k, seed=5, masked=0.2)
    y = rnd(tokens * k, cols, seed=6, dtype=DT[dtype])
    w = rnd(tokens, k, seed=7) if weighted else None
    res = rnd(tokens, cols, seed=8, dtype=DT[dtype]) if residual else None
    total = int((rows >= 0).sum())
    y[total:] = torch.nan                           # rows no index names must not be read into a result
    got = ops.mxfp4_moe_combine(y.cuda(), rows.cuda(), None if w is None else w.cuda(), residual=None if res is None else res.cuda())
    some = (rows >= 0)[:, :, None]
    picked = torch.where(some, y[rows.long().clamp(min=0)].double(), 0.0) * (1.0 if w is None else w.double()[:, :, None])
    want = picked.sum(1) + (0.0 if res is None else res.double())
    mag = picked.abs().sum(1) + (0.0 if res is None else res.double().abs())
    close(got, want, (k + 2) * U32 * mag + (U16 if dtype == "bf16" else U32) * want.abs() * (1 + 2 ** -7), "combine")


def test_combine_onto_its_residual():
    rows, _, _ = a_plan(50, 8, 2)
    y, w, res = rnd(100, 256, seed=1).cuda(), rnd(50, 2, seed=2).cuda(), rnd(50, 256, seed=3).cuda()
    want = ops.mxfp4_moe_combine(y, rows.cuda(), w, residual=res)
    got = ops.mxfp4_moe_combine(y, rows.cuda(), w, residual=res, out=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 1), (4, 8, 64), (130, 6, 96), (67, 2, 1001), (19, 32, 40), (33, 4, 7168)])
def test_combine_backward(dtype, tokens, k, cols):
    """grad_rows: one product, rounded to fp32 and to the type. grad_weights: a
    thread sums its columns (of 256 threads' pieces), then 5 + 8 additions."""
    rows, slots, _ = a_plan(tokens, 40, k, seed=5, masked=0.2)
    y, g = rnd(tokens * k, cols, seed=6, dtype=DT[dtype]), rnd(tokens, cols, seed=9, dtype=DT[dtype])
    w = rnd(tokens, k, seed=7)
    out = torch.full((tokens * k, cols), 3.0, dtype=DT[dtype], device="cuda")
    gy, gw = ops.mxfp4_moe_combine_bwd(g.cuda(), y.cuda(), rows.cuda(), w.cuda(), out=out)
    total = int((slots >= 0).sum())
    slot = slots[:total].long()
    want = torch.full((tokens * k, cols), 3.0, dtype=torch.float64)
    want[:total] = w.double().reshape(-1)[slot, None] * g.double()[slot // k]
    close(gy, want, (U32 + (U16 if dtype == "bf16" else 0.0)) * want.abs() * (1 + 2 ** -7), "grad_rows")
    prod = torch.where((rows >= 0)[:, :, None], y[rows.long().clamp(min=0)].double() * g.double()[:, None, :], 0.0)
    chain = -(-cols // 256) + 16 + 13
    close(gw, prod.sum(2), chain * U32 * prod.abs().sum(2), "grad_weights")
    only = ops.mxfp4_moe_combine_bwd(g.cuda(), None, rows.cuda(), grad_weights=False, out=torch.zeros_like(out))
    assert only[1] is None and torch.equal(only[0][:total].cpu(), g[slot // k])
    only = ops.mxfp4_moe_combine_bwd(g.cuda(), y.cuda(), rows.cuda(), w.cuda(), grad_rows=False)
    assert only[0] is None and torch.equal(only[1], gw)


def test_moves_without_tokens_rows_or_columns():
    i32 = dict(dtype=torch.int32, device="cuda")
    for t, cols, n in ((0, 64, 0), (0, 64, 5), (3, 64, 0), (3, 0, 6)):
        x, rows = torch.ones(t, cols, device="cuda"), torch.arange(2 * t, **i32).view(t, 2)
        y, w = torch.ones(n, cols, device="cuda"), torch.ones(t, 2, device="cuda")
        for kw in (dict(), dict(emit_values=False, emit_codes=True), dict(emit_codes=True)):
            d = ops.mxfp4_moe_dispatch(x, rows, row_count=n, **kw)
            assert d.values is None or d.values.shape == (n, cols)
            if d.codes is not None:      # scales of rows behind the last are zero, those of rows that no index names undefined
                words = d.scales.view(-1, 32, 4, 4)
                assert not words[:, n:].any() and not words[:, :, 1:].any()
        assert torch.equal(ops.mxfp4_moe_combine(y, rows, w, residual=x), x)
        gy, gw = ops.mxfp4_moe_combine_bwd(x, y, rows, w)
        assert gy.shape == (n, cols) and not gw.any()
        assert ops.mxfp4_moe_combine_bwd(x, None, rows, w, grad_weights=False, row_count=n)[0].shape == (n, cols)


# ------------------------------------------------------------------------------- linear

def operand(rows, k, fmt, seed, lo=126, hi=129):
    g = gen(seed)
    if fmt == "e2m1":
        c = torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8)
    else:
        c = (torch.randn(rows, k, generator=g) * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    nblk = k // 32
    size = 512 * (-(-rows // 128)) * (-(-nblk // 4))
    s = torch.full((size,), 0xFF, dtype=torch.uint8)       # scale padding is NaN: it must not be read as a scale
    r = torch.arange(rows)[:, None]
    b = torch.arange(nblk)[None, :]
    at = 512 * ((r // 128) * (-(-nblk // 4)) + b // 4) + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    s[at.reshape(-1)] = torch.randint(lo, hi, (rows * nblk,), generator=g, dtype=torch.uint8)
    return c, s


def linear_case(sizes, m, n, k, fmt, act="none", out="bf16", bias=False, residual=False, preact=False, list_type=1, seed=0, dense=False):
    """One call against the product in 64 bits. Every product of two operand
    values is exact in fp32; the K partial sums and the bias round (k + 1)
    2^-24 of their magnitudes; an activation passes an error on with at most
    its largest slope (1.13 for gelu; gated: the factors' sizes) and adds a few
    fp32 roundings of its own value; then the residual and one rounding."""
    g = len(sizes)
    a, sa = operand(m, k, fmt, seed)
    parts = [operand(n, k, fmt, seed + 1 + i, 117 if fmt == "e2m1" else 108, 119 if fmt == "e2m1" else 110) for i in range(g)]
    b = torch.stack([p[0] for p in parts])
    sb = torch.cat([p[1] for p in parts])
    width = n // 2 if act == "swiglu" else n
    dt = DT[out]
    bv = rnd(g, n, seed=seed + 90) if bias else None
    res = rnd(m, width, seed=seed + 91, dtype=dt) if residual else None
    y0 = torch.full((m, width), 5.0, dtype=dt, device="cuda")
    z0 = torch.full((m, n), 5.0, dtype=dt, device="cuda") if preact else None
    gl = torch.tensor(sizes if list_type == 1 else np.cumsum(sizes), dtype=torch.int64, device="cuda")
    r = ops.mxfp4_grouped_linear(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), None if dense else gl, k=k, elem_format=fmt,
                                 group_list_type=list_type, bias=None if bv is None else bv.cuda(), activation=act,
                                 residual=None if res is None else res.cuda(), out_dtype=dt,
                                 out=ops.LinearResult(y=y0, preact=z0))
    total = sum(sizes)
    av = R.decode(a, sa, m, k, fmt)
    z, mag = torch.zeros(total, n, dtype=torch.float64), torch.zeros(total, n, dtype=torch.float64)
    first = 0
    for i, size in enumerate(sizes):
        w = R.decode(b[i], parts[i][1], n, k, fmt)
        z[first:first + size] = av[first:first + size] @ w.T
        mag[first:first + size] = av[first:first + size].abs() @ w.abs().T
        if bv is not None:
            z[first:first + size] += bv[i].double()
            mag[first:first + size] += bv[i].double().abs()
        first += size
    ez = (k + 1) * U32 * mag
    last = U16 if out == "bf16" else U32
    want = R.activation(z, act)
    if act == "swiglu":
        gate, up, eg, eu = z[:, 0::2], z[:, 1::2], ez[:, 0::2], ez[:, 1::2]
        ey = 1.1 * eg * (up.abs() + eu) + (gate.abs() + eg) * eu + 12 * U32 * (1 + gate.abs()) * want.abs()
    else:
        ey = 1.13 * ez + (0 if act in ("none", "relu") else 16) * U32 * (1 + z.abs()) * (want.abs() + U32)
        if act == "gelu":          # the published approximation of erfc it uses is off by at most 1.5e-7, of which z / 2 passes on
            ey = ey + 0.75e-7 * z.abs()
        if act == "gelu_tanh":     # its argument's rounding: 4 roundings of |u| <= 0.8 |z| (1 + 0.045 z^2), slope of the logistic 1/4
            ey = ey + 8 * U32 * z.abs() * (1 + 0.1 * z ** 2) * torch.exp(-z.abs()).clamp(max=1.0) * z.abs()
    if res is not None:
        want = want + res[:total].double()
        ey = ey + U32 * want.abs()
    close(r.y[:total], want, ey + last * (want.abs() + ey), "y")
    assert bool((r.y[total:] == 5.0).all())
    if preact:
        close(r.preact[:total], z, ez + last * (z.abs() + ez), "preact")
        assert bool((r.preact[total:] == 5.0).all())
    return r


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("sizes,m", [([1], 1), ([0, 3, 0, 1, 1], 5), ([40, 0, 33, 7], 80), ([130, 65, 0, 200], 395), ([300], 300), ([0, 0], 9)])
@pytest.mark.parametrize("n,k", [(64, 128), (200, 512), (130, 320), (513, 1088)])
def test_linear_product(fmt, sizes, m, n, k):
    linear_case(sizes, m, n, k, fmt)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("everything", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_linear_epilogue(act, out, everything, fmt):
    linear_case([20, 0, 150, 3], 180, 262, 256, fmt, act=act, out=out, bias=everything, residual=everything, preact=everything)


def on_pairs(fmt, m, n, k, groups):
    a = ops._abi.LinearArgs()
    a.elem_format, a.m, a.n, a.k, a.d_dtype = ops._elem_format(fmt), m, n, k, ops._abi.BF16
    a.group_list, a.num_groups = 4096, groups        # not followed
    return ops._abi.mxfp4_grouped_linear_fwd_workspace(a) > 0


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("sizes,m,n,k", [([300], 300, 640, 576), ([600, 0, 513, 1], 1200, 1026, 320), ([257, 256, 255, 129, 640], 1537, 256, 128),
                                         ([8192], 8192, 1026, 2112), ([2000, 0, 4097, 1, 2300], 8500, 1026, 2176), ([257] * 9, 2400, 4096, 2048),
                                         ([1000, 24, 5000, 0], 6300, 2050, 2304)])
def test_linear_of_large_groups(fmt, sizes, m, n, k):
    """Groups of several tiles: ragged groups, features and lengths; the larger
    ones go to pairs of SMs, with more tiles than pairs."""
    if m * n >= 128 * 65536:
        assert on_pairs(fmt, m, n, k, len(sizes))
    linear_case(sizes, m, n, k, fmt, act="swiglu" if n % 4 == 0 else "none", bias=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_linear_epilogue_of_large_groups(act, out, fmt):
    k = 2048 if fmt == "e2m1" else 1056
    assert on_pairs(fmt, 4096, 2310, k, 3)
    linear_case([1300, 0, 2470], 4096, 2310, k, fmt, act=act, out=out, bias=True, residual=True, preact=True, list_type=0)


def test_linear_with_and_without_its_workspace():
    """The two kernels' fp32 sums differ by their order only."""
    m, n, k = 4096, 2304, 4096
    a, sa = operand(m, k, "e2m1", 1)
    b, sb = operand(n, k, "e2m1", 2, 117, 119)
    args = (a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
    one = ops.mxfp4_grouped_linear(*args, k=k, out_dtype=torch.float32).y
    A = ops._abi.LinearArgs()
    two = torch.empty_like(one)
    A.m, A.n, A.k, A.d_dtype = m, n, k, ops._abi.F32
    A.a, A.lda, A.a_scales = args[0].data_ptr(), k // 2, args[1].data_ptr()
    A.b, A.ldb, A.b_scales = args[2].data_ptr(), k // 2, args[3].data_ptr()
    A.y, A.ld_y = two.data_ptr(), n
    assert ops._abi.mxfp4_grouped_linear(A, torch.cuda.current_stream().cuda_stream) == 0
    assert (one - two).norm() <= 2 * k * U32 * one.norm()


@pytest.mark.parametrize("n", [1, 2, 31, 127, 128, 129, 255, 256, 257, 384, 385])
def test_linear_widths(n):
    linear_case([70, 9], 80, n, 192, "e2m1", out="fp32", bias=True, residual=True, preact=True)


@pytest.mark.parametrize("k", [64, 128, 192, 256, 320, 576, 1024])
def test_linear_lengths_e2m1(k):
    linear_case([33, 5], 40, 140, k, "e2m1", out="fp32")


@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 416, 1056])
def test_linear_lengths_e4m3(k):
    linear_case([33, 5], 40, 140, k, "e4m3", out="fp32")


@pytest.mark.parametrize("sizes,m", [([5] * 30, 150), ([64] * 9, 576), ([200] * 5, 1000), ([0] * 50 + [700], 700)])
def test_linear_many_tiles_per_cta(sizes, m):
    """More tiles than SMs, in every token tile width."""
    linear_case(sizes, m, 9000 if m < 700 else 7000, 128, "e2m1", act="swiglu", list_type=0)


def test_linear_dense_and_views():
    linear_case([77], 77, 300, 256, "e4m3", act="gelu", bias=True, residual=True, preact=True, dense=True)
    # strided outputs and residual
    a, sa = operand(50, 128, "e2m1", 1)
    b, sb = operand(64, 128, "e2m1", 2)
    res = rnd(50, 70, seed=3, dtype=torch.bfloat16).cuda()
    y = torch.zeros(50, 99, dtype=torch.bfloat16, device="cuda")
    plain = ops.mxfp4_grouped_linear(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), k=128, residual=res[:, 3:67].contiguous(), bias=rnd(64, seed=4).cuda())
    ops.mxfp4_grouped_linear(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), k=128, residual=res[:, 3:67], bias=rnd(64, seed=4).cuda(),
                             out=ops.LinearResult(y=y[:, 5:69]))
    assert torch.equal(plain.y, y[:, 5:69]) and bool((y[:, :5] == 0).all()) and bool((y[:, 69:] == 0).all())


def test_linear_agrees_with_the_grouped_gemm():
    """Without an epilogue: the same product as mxfp4_grouped_gemm (both fp32 accumulations within the bound)."""
    k, n, sizes = 512, 384, [100, 0, 250, 34]
    a, sa = operand(sum(sizes), k, "e2m1", 5)
    parts = [operand(n, k, "e2m1", 6 + i) for i in range(4)]
    b, sb = torch.stack([p[0] for p in parts]).cuda(), torch.cat([p[1] for p in parts]).cuda()
    gl = torch.tensor(sizes, dtype=torch.int64, device="cuda")
    one = ops.mxfp4_grouped_gemm(a.cuda(), sa.cuda(), b, sb, gl, k=k, group_list_type=1)
    two = ops.mxfp4_grouped_linear(a.cuda(), sa.cuda(), b, sb, gl, k=k, group_list_type=1, out_dtype=torch.float32).y
    assert (one - two).norm() <= 2 * k * U32 * one.norm()


def test_large_linear_captured_and_on_two_streams():
    """The pair kernel and the decoding tiles at once on two streams, and the
    former captured: the eager calls' bytes."""
    n, k = 2304, 2048
    big, small = [2048, 0, 2100], [1, 2, 0]
    b, sb = zip(*(operand(n, k, "e2m1", 30 + e, 117, 119) for e in range(3)))
    b, sb = torch.stack(b).cuda(), torch.cat(sb).cuda()
    def call(sizes, seed, gl):
        a, sa = operand(sum(sizes), k, "e2m1", seed)
        a, sa = a.cuda(), sa.cuda()
        return lambda: ops.mxfp4_grouped_linear(a, sa, b, sb, gl, k=k, group_list_type=1, activation="swiglu", check=False).y
    lists = [torch.tensor(v, dtype=torch.int64, device="cuda") for v in (big, small)]
    assert on_pairs("e2m1", sum(big), n, k, 3)
    calls = [call(big, 1, lists[0]), call(small, 2, lists[1])]
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        captured = calls[0]()
    want = [c() for c in calls]
    for _ in range(2):
        captured.fill_(7.0)
        g.replay()
        assert torch.equal(captured, want[0])
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(6):
        for s, c, o in zip(streams, calls, got):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o.append(c())
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(v, w) for v in o)


def test_linear_invalid_lists():
    a, sa = operand(50, 128, "e2m1", 1)
    b, sb = operand(128, 128, "e2m1", 2)
    args = (a.cuda(), sa.cuda(), b.view(2, 64, -1).cuda(), torch.cat([sb, sb]).cuda())
    for sizes, kind in (([30, 21], 1), ([-1, 20], 1), ([40, 30], 0), ([10, 51], 0), ([2 ** 62, 2 ** 62], 1)):
        gl = torch.tensor(sizes, dtype=torch.int64, device="cuda")
        y = torch.full((50, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(MXFP4ArgumentError):
            ops.mxfp4_grouped_linear(*args, gl, k=128, group_list_type=kind, out=ops.LinearResult(y=y))
        assert bool((y == 3.0).all())
        r = ops.mxfp4_grouped_linear(*args, gl, k=128, group_list_type=kind, check=False)
        assert int(r.status) == 1
        with pytest.raises(MXFP4ArgumentError):
            ops.mxfp4_grouped_linear_bwd(rnd(50, 64).cuda(), rnd(50, 64).cuda(), gl, group_list_type=kind)


@pytest.mark.parametrize("m,n", [(0, 64), (50, 0), (0, 0)])
def test_linear_lists_of_empty_matrices(m, n):
    """A list is checked whatever there is to multiply, forward and backward alike."""
    k = 128
    a = torch.zeros(m, k // 2, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(ops.scales_row_bytes(m, k, 32, "mma"), dtype=torch.uint8, device="cuda")
    b = torch.zeros(2, n, k // 2, dtype=torch.uint8, device="cuda")
    sb = torch.zeros(2 * ops.scales_row_bytes(n, k, 32, "mma"), dtype=torch.uint8, device="cuda")
    z = torch.zeros(m, n, device="cuda")
    for sizes, kind, good in (([0, 0], 1, True), ([0, 0], 0, True), ([m, 0], 1, True), ([m, m], 0, True), ([m, 1], 1, False), ([0, -1], 1, False),
                              ([-1, 1], 1, False), ([m + 1, m + 1], 0, False), ([1, 0], 0, False), ([2 ** 40, 0], 1, False)):
        gl = torch.tensor(sizes, dtype=torch.int64, device="cuda")
        calls = (lambda **kw: ops.mxfp4_grouped_linear(a, sa, b, sb, gl, k=k, group_list_type=kind, **kw),
                 lambda **kw: ops.mxfp4_grouped_linear_bwd(z, z, gl, group_list_type=kind, **kw))
        for call in calls:
            if good:
                call()
            else:
                with pytest.raises(MXFP4ArgumentError):
                    call()
        assert int(calls[0](check=False).status) == (0 if good else 1)
    ops.mxfp4_grouped_linear(a, sa, b[0], sb[: sb.numel() // 2], k=k)
    _, gb = ops.mxfp4_grouped_linear_bwd(z, z)
    assert not gb.any()


def test_invalid_lists_of_large_linears():
    a, sa = operand(4096, 2048, "e2m1", 1)
    b, sb = operand(4608, 2048, "e2m1", 2)
    gl = torch.tensor([4000, 97], dtype=torch.int64, device="cuda")
    y = torch.full((4096, 2304), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(MXFP4ArgumentError):
        ops.mxfp4_grouped_linear(a.cuda(), sa.cuda(), b.view(2, 2304, -1).cuda(), torch.cat([sb, sb])[: 2 * ops.scales_row_bytes(2304, 2048, 32, "mma")].cuda(),
                                 gl, k=2048, group_list_type=1, out=ops.LinearResult(y=y))
    assert bool((y == 3.0).all())


def test_linear_refusals():
    a, sa = operand(50, 128, "e2m1", 1)
    b, sb = operand(64, 128, "e2m1", 2)
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    ok = dict(k=128)
    for bad in (dict(k=96), dict(k=0), dict(k=256), dict(activation="tanh"), dict(out_dtype=torch.float16), dict(elem_format="e5m2"),
                dict(bias=torch.zeros(63, device="cuda")), dict(residual=torch.zeros(50, 63, device="cuda").bfloat16()),
                dict(out=ops.LinearResult(y=torch.zeros(50, 63, device="cuda").bfloat16()))):
        with pytest.raises((ValueError, TypeError)):
            ops.mxfp4_grouped_linear(a, sa, b, sb, **{**ok, **bad})
    empty = torch.zeros(0, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear(a, sa, b, sb, empty, k=128)
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear_bwd(rnd(50, 64).cuda(), rnd(50, 64).cuda(), empty)
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear(a, sa[:100], b, sb, k=128)
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear(a, sa, b, sb[:100], k=128)
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear(a, sa, b[:63], sb, k=128, activation="swiglu")
    with pytest.raises(ValueError):
        ops.mxfp4_grouped_linear(a.t(), sa, b, sb, k=128)
    with pytest.raises(TypeError):
        ops.mxfp4_grouped_linear(a, sa, b, sb, k=128, bias=torch.zeros(64, device="cuda").bfloat16())


def slope_bound(z, act):
    """Rounding of a slope's evaluation: a few fp32 operations on terms of size 1 + |z|
    (gelu's erfc, off by at most 1.5e-7 = 2.6 roundings, halved, among them)."""
    return 24 * U32 * (1 + z.abs()) * (1.0 + (z ** 2).clamp(max=64.0) * (1.0 if act == "gelu_tanh" else 0.0))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes,m,n", [([1], 1, 2), ([40, 0, 70, 1, 200], 320, 264), ([130], 130, 1026), ([0, 0], 5, 64), ([500, 12], 512, 4096)])
def test_linear_backward(act, dtype, sizes, m, n):
    """Against autograd of the activation in 64 bits; the bias sums add the
    unrounded gradients: a thread's rows of a unit of 32, at most 8 rows side by
    side, then the group's units, in order."""
    width = n // 2 if act == "swiglu" else n
    z = rnd(m, n, seed=1, std=2.0, dtype=DT[dtype])
    gy = rnd(m, width, seed=2, dtype=DT[dtype])
    gl = torch.tensor(sizes, dtype=torch.int64, device="cuda")
    out = torch.full((m, n), 9.0, dtype=DT[dtype], device="cuda")
    gz, gb = ops.mxfp4_grouped_linear_bwd(gy.cuda(), z.cuda(), gl, group_list_type=1, activation=act, out=out)
    total = sum(sizes)
    v = z.double().requires_grad_(True)
    (want,) = torch.autograd.grad(R.activation(v, act), v, gy.double())
    if act == "swiglu":
        e = torch.empty_like(want)
        gate, up, g = z.double()[:, 0::2], z.double()[:, 1::2], gy.double().abs()
        e[:, 0::2] = slope_bound(gate, act) * g * up.abs()
        e[:, 1::2] = slope_bound(gate, act) * g
    else:
        e = slope_bound(z.double(), act) * gy.double().abs() if act not in ("none", "relu") else U32 * want.abs()
    close(gz[:total], want[:total], e[:total] + (U16 if dtype == "bf16" else U32) * (want.abs() + e)[:total], "grad_preact")
    assert bool((gz[total:] == 9.0).all())
    first = 0
    for i, size in enumerate(sizes):
        part = want[first:first + size]
        chain = 32 + 8 + size // 32 + 1
        close(gb[i], part.sum(0), e[first:first + size].sum(0) + chain * U32 * part.abs().sum(0), "grad_bias")
        first += size
    none = ops.mxfp4_grouped_linear_bwd(gy.cuda(), z.cuda(), gl, group_list_type=1, activation=act, bias_grad=False, out=torch.zeros_like(out))
    assert none[1] is None and torch.equal(none[0][:total], gz[:total])


def test_linear_backward_large_values():
    z = torch.tensor([[-3e38, -1e20, -100.0, -20.0, 20.0, 100.0, 1e20, 3e38]]).cuda()
    g = torch.ones(1, 8).cuda()
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        gz, gb = ops.mxfp4_grouped_linear_bwd(g, z, activation=act)
        want = torch.tensor([[0.0, 0, 0, 0, 1, 1, 1, 1]])
        close(gz, want.double(), 1e-6, act)
        assert torch.equal(gb.cpu(), gz.cpu())


@pytest.mark.parametrize("m", [1, 40])
def test_gelu_keeps_the_digits_of_small_results(m):
    """z is the bias alone (zero operands). The mass below z is e t P(t): 8
    roundings of P and its product with t (measured over the range in fp32), 5 of
    t (a quotient within 2 units, a sum) of which at most 1.9 times pass on, e =
    exp(-z^2 / 2) by an exponential within 2 + 1.173 z^2 / 2 units whose argument
    rounds once (z^2 / 2), one product: below 24 + 1.7 z^2 roundings of itself.
    What fp32 cannot hold as a normal number counts as 0."""
    n, k = 8192, 64
    z = torch.linspace(-13.0, 13.0, n)
    code = lambda r: (torch.zeros(r, k // 2, dtype=torch.uint8, device="cuda"),  # noqa: E731
                      torch.full((ops.scales_row_bytes(r, k, 32, "mma"),), 127, dtype=torch.uint8, device="cuda"))
    got = ops.mxfp4_grouped_linear(*code(m), *code(n), k=k, bias=z.cuda(), activation="gelu", out_dtype=torch.float32).y
    v = z.double()
    mass, density = 0.5 * torch.special.erfc(-v / math.sqrt(2.0)), torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    for row in got:
        close(row, v * mass, ((25 + 1.7 * v * v) * U32 * mass + 2.0 ** -126) * v.abs(), "gelu")
    gz, _ = ops.mxfp4_grouped_linear_bwd(torch.ones(1, n, device="cuda"), z.view(1, n).cuda(), activation="gelu")
    bound = (25 + 1.7 * v * v) * U32 * (mass + v.abs() * density) + 2.0 ** -126 * (1 + v.abs())
    close(gz[0], mass + v * density, bound, "slope")


def test_linear_backward_strided():
    z, g = rnd(70, 100, seed=1).cuda(), rnd(70, 60, seed=2).cuda()
    one = ops.mxfp4_grouped_linear_bwd(g[:, 7:53], z[:, 3:95], activation="swiglu")
    two = ops.mxfp4_grouped_linear_bwd(g[:, 7:53].contiguous(), z[:, 3:95].contiguous(), activation="swiglu")
    assert torch.equal(one[0], two[0])
    # the same 70 values a column, added in another order: each order is off by at most 69 roundings of the partial sums
    assert bool(((one[1] - two[1]).abs() <= 2 * 69 * U32 * one[0].abs().sum(0)).all())


# ------------------------------------------------------------------- offsets past 32 bits

def test_rows_past_32_bits():
    """2.3e9 elements of expert rows: the last ones as right as the first."""
    t, k, cols = 40000, 8, 7168
    x = torch.randn(t, cols, device="cuda").bfloat16()
    rows = torch.randperm(t * k, device="cuda").int().view(t, k)
    d = ops.mxfp4_moe_dispatch(x, rows, emit_codes=True, elem_format="e4m3", scale_mode="floor")
    q = ops.mxfp4_qdq_fwd(x, emit_values=False, emit_codes=True, elem_format="e4m3", scale_mode="floor")
    for i in (0, 1, t // 2, t - 2, t - 1):
        for j in (0, k - 1):
            r = int(rows[i, j])
            assert torch.equal(d.values[r], x[i]) and torch.equal(d.codes[r], q.codes_row[i])
    high = (rows.long() * cols > 2 ** 31).any(1).nonzero()[-3:, 0].tolist()
    assert high
    for i in high:
        for j in range(k):
            assert torch.equal(d.values[int(rows[i, j])], x[i]) and torch.equal(d.codes[int(rows[i, j])], q.codes_row[i])
    out = ops.mxfp4_moe_combine(d.values, rows)
    assert torch.equal(out, k * x)                 # eight equal values: exact
    del d, q
    gy, gw = ops.mxfp4_moe_combine_bwd(x, out[:1].expand(t * k, cols), rows, grad_weights=False)
    for i in high:
        assert torch.equal(gy[int(rows[i, 0])], x[i])


def test_dispatch_of_a_very_wide_row():
    """More scale columns than one launch of the scales' second kernel has room for."""
    cols = 65536 * 32 * 128                      # one block row of that kernel too many
    x = torch.randn(1 << 16, device="cuda").bfloat16().repeat(cols >> 16).view(1, cols)
    rows = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    r = ops.mxfp4_moe_dispatch(x, rows, emit_values=False, emit_codes=True)
    q = ops.mxfp4_qdq_fwd(x.view(4096, -1), emit_values=False, emit_codes=True)      # the same blocks as shorter rows
    assert torch.equal(r.codes[0], q.codes_row.view(-1)) and torch.equal(r.codes[1], q.codes_row.view(-1))
    got, want = r.scales.view(-1, 512), q.scales_row.view(-1, 4)
    # word 4 (row % 32) + row // 32 of an atom: rows 0 and 1, the others padding
    assert torch.equal(got[:, :4], want) and torch.equal(got[:, 16:20], want)
    assert not got[:, 4:16].any() and not got[:, 20:].any()


def at_the_end(t: torch.Tensor) -> torch.Tensor:
    """A copy of t that ends where a block of the device's memory (2 MB pages) ends."""
    size = t.numel() * t.element_size()
    block = torch.empty((max(size, 1 << 25) + (1 << 21) - 1) >> 21 << 21, dtype=torch.uint8, device="cuda")
    out = block[block.numel() - size:].view(t.dtype).view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols", [8, 96, 256, 1000, 4096])
def test_inputs_at_the_end_of_their_memory(dtype, cols):
    """Nothing is read behind a tensor's last row, however little of the
    threads' reach it fills: the results of the same calls elsewhere."""
    torch.cuda.empty_cache()
    t, k, n = 12, 5, 60
    rows, _, counts = a_plan(t, 7, k)
    x, y, z, g, gz = (rnd(r, c, seed=i, dtype=DT[dtype]).cuda() for i, (r, c) in enumerate(((t, cols), (n, cols), (n, cols), (t, cols), (n, cols // 2))))
    lg, w = rnd(t, 64, seed=9, dtype=DT[dtype]).cuda(), rnd(t, k, seed=8).cuda()
    rows, counts = rows.cuda(), counts.cuda()
    chosen = ops.mxfp4_moe_route(lg, k).experts

    def results(f):
        x2, y2, z2, g2, gz2, lg2, w2, rows2 = (f(v) for v in (x, y, z, g, gz, lg, w, rows))
        zero = lambda: torch.zeros(n, cols, dtype=DT[dtype], device="cuda")  # noqa: E731
        r = ops.mxfp4_moe_route(lg2, k)
        d = ops.mxfp4_moe_dispatch(x2, rows2, emit_codes=True)
        return [r.weights, r.experts, d.values, d.codes, d.scales, ops.mxfp4_moe_combine(y2, rows2, w2, residual=x2),
                *ops.mxfp4_moe_combine_bwd(g2, y2, rows2, w2, out=zero()), ops.mxfp4_moe_route_bwd(w2, lg2, chosen),
                *ops.mxfp4_grouped_linear_bwd(gz2, z2, counts, group_list_type=1, activation="swiglu", out=zero()),
                *ops.mxfp4_grouped_linear_bwd(y2, z2, counts, group_list_type=1, activation="gelu", out=zero())]

    for a, b in zip(results(lambda v: v), results(at_the_end)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("sizes,m,n,k", [([1, 2], 3, 130, 192), ([40, 0, 33], 80, 200, 320), ([2500, 1700], 4200, 2100, 2112)])
def test_operands_at_the_end_of_their_memory(fmt, sizes, m, n, k):
    torch.cuda.empty_cache()
    a, sa = operand(m, k, fmt, 1)
    parts = [operand(n, k, fmt, 2 + i, 117, 119) for i in range(len(sizes))]
    gl = torch.tensor(sizes, dtype=torch.int64)
    args = (a, sa, torch.stack([p[0] for p in parts]), torch.cat([p[1] for p in parts]), gl, rnd(len(sizes), n, seed=5), rnd(m, n // 2, seed=6))

    def result(f):
        a, sa, b, sb, gl, bias, res = (f(v.cuda()) for v in args)
        r = ops.mxfp4_grouped_linear(a, sa, b, sb, gl, k=k, elem_format=fmt, group_list_type=1, bias=bias, activation="swiglu", residual=res,
                                     out_dtype=torch.float32, out=ops.LinearResult(y=torch.zeros(m, n // 2, device="cuda"), preact=torch.zeros(m, n, device="cuda")))
        return r.y, r.preact

    for x, y in zip(result(lambda v: v), result(at_the_end)):
        assert torch.equal(x, y)


def test_results_past_32_bits():
    """2.4e9 results of a product; rows of a slice by themselves give the same bytes."""
    m, n, k = 300032, 8192, 64
    a, sa = operand(m, k, "e2m1", 3)
    b, sb = operand(n, k, "e2m1", 4)
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    y = ops.mxfp4_grouped_linear(a, sa, b, sb, k=k).y
    for first in (0, 256 * 1024, m - 256):
        part = ops.mxfp4_grouped_linear(a[first:first + 256], sa[first * 4:(first + 256) * 4], b, sb, k=k).y
        assert torch.equal(y[first:first + 256], part)


def test_logits_past_32_bits():
    t, e = 2100000, 1024
    x = torch.randn(t, e, device="cuda", dtype=torch.bfloat16)
    r = ops.mxfp4_moe_route(x, 2)
    one = ops.mxfp4_moe_route(x[-100:], 2)
    assert torch.equal(r.experts[-100:], one.experts) and torch.equal(r.weights[-100:], one.weights)
    assert int(r.counts.sum()) == 2 * t
    last = r.slots[r.rows[-1].long()]
    assert last.tolist() == [2 * t - 2, 2 * t - 1]
    g = ops.mxfp4_moe_route_bwd(torch.ones(t, 2, device="cuda"), x, r.experts, renormalize=False)
    assert torch.equal(g[-100:], ops.mxfp4_moe_route_bwd(torch.ones(100, 2, device="cuda"), x[-100:], one.experts, renormalize=False))


# ------------------------------------------------------------------ as they are used together

def layer(x, router, w1, s1, w2, s2, hidden, k, mask=None, check=False):
    """A quantised mixture-of-experts layer: route, dispatch quantised, gated
    product, quantise, product, combine onto the input."""
    experts = router.shape[1]
    t, cols = x.shape
    r = ops.mxfp4_moe_route(x.float() @ router, k, score="sigmoid", num_groups=2, topk_groups=1, token_mask=mask)
    d = ops.mxfp4_moe_dispatch(x, r.rows, emit_values=False, emit_codes=True)
    h = ops.mxfp4_grouped_linear(d.codes, d.scales, w1, s1, r.counts, k=cols, group_list_type=1, activation="swiglu", check=check)
    q = ops.mxfp4_qdq_fwd(h.y, emit_values=False, emit_codes=True, scales_layout="mma")
    y = ops.mxfp4_grouped_linear(q.codes_row, q.scales_row, w2, s2, r.counts, k=hidden, group_list_type=1, check=check)
    return ops.mxfp4_moe_combine(y.y, r.rows, r.weights, residual=x), r


def a_layer(t, cols=256, hidden=128, experts=8, seed=0):
    x = rnd(t, cols, seed=seed, dtype=torch.bfloat16).cuda()
    router = rnd(cols, experts, seed=seed + 1, std=0.1).cuda()
    w1 = rnd(experts, 2 * hidden, cols, seed=seed + 2, std=0.06, dtype=torch.bfloat16)
    w2 = rnd(experts, cols, hidden, seed=seed + 3, std=0.08, dtype=torch.bfloat16)
    ops1 = [ops.mxfp4_mma_operand(w.cuda()) for w in w1]
    ops2 = [ops.mxfp4_mma_operand(w.cuda()) for w in w2]
    pack = lambda o: (torch.stack([c.view(torch.uint8) for c, _ in o]), torch.cat([s.view(torch.uint8) for _, s in o]))  # noqa: E731
    return x, router, pack(ops1), pack(ops2), w1, w2


def layer_plain(x, r, w1, w2, k):
    """The layer on the oracle's fake-quantised values, in 64 bits but for the
    bf16 roundings between its steps."""
    bits = lambda v: v.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    q = lambda v: torch.from_numpy(O.bf16_to_f32(O.qdq_rowwise(bits(v), 32, 6.0, O.SCALE_PAGE)["y"])).double()  # noqa: E731
    out = x.double()
    qx = q(x)
    qw1 = [q(w) for w in w1]
    qw2 = [q(w) for w in w2]
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(r.experts[t, j])
            if e < 0:
                continue
            h = R.activation((qx[t:t + 1] @ qw1[e].T), "swiglu").bfloat16()
            y = (q(h) @ qw2[e].T).bfloat16().double()
            out[t] += float(r.weights[t, j]) * y[0]
    return out


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_layer(tokens):
    k = 3
    x, router, (w1, s1), (w2, s2), f1, f2 = a_layer(tokens)
    mask = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if tokens > 3:
        mask[2] = False
    out, r = layer(x, router, w1, s1, w2, s2, 128, k, mask)
    want = layer_plain(x.cpu(), r, f1, f2, k)
    if tokens > 3:
        assert torch.equal(out[2], x[2])
    # an intermediate that rounds the other way moves one code by at most a step: the result as a whole stays near
    assert (out.double().cpu() - want).norm() <= 2 * U16 * want.norm()


def test_layer_in_a_graph_and_on_streams():
    """Captured and replayed on new inputs, two graphs in turn, and two streams at once: the results of the eager calls."""
    k = 3
    x, router, (w1, s1), (w2, s2), _, _ = a_layer(130)
    xs = [rnd(130, 256, seed=40 + i, dtype=torch.bfloat16).cuda() for i in range(3)]
    want = [layer(v, router, w1, s1, w2, s2, 128, k)[0] for v in xs]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        static = x.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(static, router, w1, s1, w2, s2, 128, k)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = layer(static, router, w1, s1, w2, s2, 128, k)
        graphs.append((g, static, out))
    for v, w in zip(xs, want):
        for g, static, out in graphs:
            static.copy_(v)
            g.replay()
            assert torch.equal(out, w)
    for g, static, out in graphs:   # one after the other without waiting in between
        static.copy_(xs[1])
        g.replay()
    assert torch.equal(graphs[0][2], want[1]) and torch.equal(graphs[1][2], want[1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s, v in zip(streams, xs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([layer(v, router, w1, s1, w2, s2, 128, k)[0] for _ in range(4)])
    torch.cuda.synchronize()
    for w, got in zip(want, outs):
        assert all(torch.equal(w, o) for o in got)


def test_training_step_of_a_layer():
    """Forward and backward through the operators (dispatch of values, product,
    combine, router) against autograd of the same layer in 64 bits."""
    t, cols, n, experts, k = 90, 128, 192, 6, 2
    x = rnd(t, cols, seed=1)
    lg = rnd(t, experts, seed=2)
    bias = rnd(experts, n, seed=4)
    go = rnd(t, n, seed=5)
    r = ops.mxfp4_moe_route(lg.cuda(), k)
    rows, chosen = r.rows.cpu(), r.experts.cpu()
    # fp32 values so that only fp32 roundings separate the two; the product is formed on quantised copies
    d = ops.mxfp4_moe_dispatch(x.cuda(), r.rows, emit_values=True, emit_codes=True, elem_format="e4m3", scale_mode="floor")
    w = [operand(n, cols, "e4m3", 20 + e, 108, 110) for e in range(experts)]
    b, sb = torch.stack([c for c, _ in w]).cuda(), torch.cat([s for _, s in w]).cuda()
    h = ops.mxfp4_grouped_linear(d.codes, d.scales, b, sb, r.counts, k=cols, elem_format="e4m3", group_list_type=1, bias=bias.cuda(),
                                 activation="gelu", out_dtype=torch.float32, emit_preact=True)
    out = ops.mxfp4_moe_combine(h.y, r.rows, r.weights)
    gy, gw = ops.mxfp4_moe_combine_bwd(go.cuda(), h.y, r.rows, r.weights)
    gz, gb = ops.mxfp4_grouped_linear_bwd(gy, h.preact, r.counts, group_list_type=1, activation="gelu")
    gl = ops.mxfp4_moe_route_bwd(gw, lg.cuda(), r.experts)
    # the same in 64 bits, from the quantised rows
    qx = R.decode(d.codes.cpu(), d.scales.cpu(), t * k, cols, "e4m3")
    lgd, bd = lg.double().requires_grad_(True), bias.double().requires_grad_(True)
    weights = R.route_weights(lgd, chosen, "softmax", True, 1.0)
    order = torch.empty(t * k, dtype=torch.long)
    order[rows.reshape(-1).long()] = torch.arange(t * k)
    expert = chosen.reshape(-1).long()[order]
    wd = torch.stack([R.decode(c, s, n, cols, "e4m3") for c, s in w])
    z = torch.einsum("rk,rnk->rn", qx, wd[expert]) + bd[expert]
    z.retain_grad()
    y = R.activation(z, "gelu")
    want = (weights.reshape(-1)[:, None] * y[rows.reshape(-1).long()]).view(t, k, n).sum(1)
    want.backward(go.double())
    for got, ref in ((out, want), (gz, z.grad), (gb, bd.grad), (gl, lgd.grad)):
        # norms: each is a chain of fp32 steps whose products have 128 terms
        assert (got.double().cpu() - ref).norm() <= 512 * U32 * ref.norm()
    # the dispatch's gradient is a combine without weights
    gx = ops.mxfp4_moe_combine(d.values, r.rows)
    assert torch.equal(gx.cpu(), k * x)
