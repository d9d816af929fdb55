"""GPU checks of the mixture-of-experts module API (moe.py): values and
gradients against autograd of the same layer in 64 bits on the fake-quantised
values, and the serving form against the training one."""
from __future__ import annotations

import copy
import pickle

import pytest
import torch

from mxfp4_block_fake_b200 import MXFP4ArgumentError, MXFP4MoE, moe, mxfp4_quant_dequant, ops
from tests import moe_ref as R

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def rnd(*shape, seed=0, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def ste(v: torch.Tensor) -> torch.Tensor:
    """Quantised value, gradient passed through (64 bits)."""
    return v + (mxfp4_quant_dequant(v.detach().float()).double() - v.detach())


@pytest.mark.parametrize("masked", [False, True])
def test_gradients_of_the_functions(masked):
    """fp32 throughout, so that only fp32 roundings separate the two (each
    result is a chain of sums of at most 192 products): norms within 4 * 192
    roundings."""
    t, cols, n, experts, k = 70, 128, 192, 5, 2
    x, lg, w, b = (rnd(t, cols, seed=1), rnd(t, experts, seed=2), rnd(experts, n, cols, seed=3, std=0.1), rnd(experts, n, seed=4))
    go = rnd(t, n // 2, seed=5)
    res = rnd(t, n // 2, seed=6)
    mask = (torch.arange(t) % 7 != 0).cuda() if masked else None
    leaves = [v.clone().requires_grad_(True) for v in (x, lg, w, b, res)]
    r = moe.moe_route(leaves[1], k, score="sigmoid", token_mask=mask)
    y = moe.moe_grouped_linear(moe.moe_dispatch(leaves[0], r), leaves[2], r.counts, leaves[3], activation="swiglu")
    out = moe.moe_combine(y, r, residual=leaves[4])
    out.backward(go)
    ref = [v.double().requires_grad_(True) for v in (x, lg, w, b, res)]
    weights = R.route_weights(ref[1], r.experts, "sigmoid", True, 1.0)
    xq, wq = ste(ref[0]), ste(ref[2])
    want = ref[4].clone()
    for j in range(k):
        e = r.experts[:, j].long().clamp(min=0)
        z = torch.einsum("tk,tnk->tn", xq, wq[e]) + ref[3][e]
        want = want + (weights[:, j] * (r.experts[:, j] >= 0))[:, None] * R.activation(z, "swiglu")
    want.backward(go.double())
    for got, exp in ((out, want), *((a.grad, c.grad) for a, c in zip(leaves, ref))):
        assert (got.double() - exp).norm() <= 4 * 192 * U32 * exp.norm()


@pytest.mark.parametrize("tokens", [1, 33, 700])
def test_module_serves_what_it_trains(tokens):
    """Laid out for serving, the layer gives the training forward's bytes: the same codes go through the same kernels."""
    torch.manual_seed(0)
    m = MXFP4MoE(256, 128, 8, 3, score="sigmoid", num_groups=4, topk_groups=2, balance=True, device="cuda")
    x = rnd(2, tokens, 256, seed=7, dtype=torch.bfloat16)
    mask = torch.ones(2, tokens, dtype=torch.bool, device="cuda")
    mask[1, tokens // 2:] = False
    out, counts = m(x, mask, return_counts=True)
    assert out.requires_grad and int(counts.sum()) == 3 * int(mask.sum())
    assert torch.equal(out[~mask], x[~mask])
    m.lay_out()
    with torch.no_grad():
        assert torch.equal(m(x, mask), out)
    assert m.to("cuda")._laid_out is None      # moved: laid out again when asked
    m.update_balance(counts)
    low = counts.float() < counts.float().mean()
    assert bool((m.balance[low] > 0).all()) and bool((m.balance[~low] <= 0).all())
    out.sum().backward()
    for p in m.parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and float(p.grad.abs().sum()) > 0


def test_module_in_a_graph():
    """The serving forward captured and replayed while eager training goes on."""
    torch.manual_seed(1)
    m = MXFP4MoE(128, 64, 4, 2, device="cuda").lay_out()
    xs = [rnd(40, 128, seed=i, dtype=torch.bfloat16) for i in range(3)]
    with torch.no_grad():
        want = [m(v) for v in xs]
        static = xs[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m(static)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m(static)
    for v, w in zip(xs, want):
        static.copy_(v)
        g.replay()
        m(v).sum().backward()
        assert torch.equal(out, w)


@pytest.mark.parametrize("which", ["route", "dispatch", "combine"])
def test_captured_backwards_are_refused(which):
    """While an eager graph of the same leaves lives: an exception, and the process and the stream go on."""
    x = rnd(20, 64, seed=1).requires_grad_(True)
    lg = rnd(20, 4, seed=2).requires_grad_(True)

    def forward():
        r = moe.moe_route(lg, 2)
        d = moe.moe_dispatch(x, r)
        return {"route": r.weights, "dispatch": d, "combine": moe.moe_combine(d, r)}[which].square().sum()

    alive = forward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            forward().backward()
    alive.backward()
    torch.cuda.synchronize()
    assert bool(torch.isfinite((lg if which == "route" else x).grad).all())


@pytest.mark.parametrize("change", ["step", "load", "replace"])
def test_laid_out_copy_is_not_used_for_changed_weights(change):
    torch.manual_seed(3)
    m, other = (MXFP4MoE(64, 128, 4, 2, device="cuda") for _ in range(2))
    x = rnd(30, 64, seed=3, dtype=torch.bfloat16)
    m.lay_out()
    with torch.no_grad():
        old = m(x)
        if change == "step":
            for p, q in zip(m.parameters(), other.parameters()):
                p.add_(q)
        elif change == "load":
            m.load_state_dict(other.state_dict())
        else:
            m.router, m.w1, m.w2 = other.router, other.w1, other.w2
        got = m(x)
        assert not torch.equal(got, old)
        assert torch.equal(m.lay_out()(x), got)
        if change != "step":
            assert torch.equal(other(x), got)


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64)])
def test_module_without_tokens(shape):
    m = MXFP4MoE(64, 64, 4, 2, device="cuda")
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    out, counts = m(x, return_counts=True)
    assert out.shape == x.shape and not counts.any()
    out.sum().backward()
    assert x.grad.shape == x.shape and not any(p.grad.any() for p in m.parameters())
    m.lay_out()
    with torch.no_grad():
        assert m(x).shape == x.shape


@pytest.mark.parametrize("how", ["deepcopy", "pickle", "parent", "data", "rule"])
def test_laid_out_copy_of_other_weights_is_not_used(how):
    """Copies of a laid-out layer whose count of changes happens to be the same
    again, weights exchanged below autograd, and another scale rule."""
    torch.manual_seed(4)
    a, b, m = (MXFP4MoE(64, 128, 4, 2, device="cuda") for _ in range(3))
    x = rnd(30, 64, seed=3, dtype=torch.bfloat16)
    with torch.no_grad():
        m.load_state_dict(a.state_dict())
        m.lay_out()
        old = m(x)
        if how == "deepcopy":
            m = copy.deepcopy(m)
            m.load_state_dict(b.state_dict())
        elif how == "pickle":
            m = pickle.loads(pickle.dumps(m))
            m.load_state_dict(b.state_dict())
        elif how == "parent":
            torch.nn.ModuleList([m]).load_state_dict(torch.nn.ModuleList([b]).state_dict())
        elif how == "data":
            m.router.data, m.w1.data, m.w2.data = b.router.data.clone(), b.w1.data.clone(), b.w2.data.clone()
        else:
            m.scale_mode = "floor"
        got = m(x)
        assert not torch.equal(got, old)
        assert torch.equal(m.lay_out()(x), got)
        if how != "rule":
            assert torch.equal(b(x), got)


def test_inference_tensors_are_not_laid_out():
    """Their changes leave no trace, so a copy of them could not be known to be current."""
    torch.manual_seed(6)
    x = rnd(30, 64, seed=3, dtype=torch.bfloat16)
    with torch.inference_mode():
        m, other = (MXFP4MoE(64, 128, 4, 2, device="cuda") for _ in range(2))
        with pytest.raises(RuntimeError, match="inference"):
            m.lay_out()
        m(x)
        for p, q in zip(m.parameters(), other.parameters()):
            p.copy_(q)
        assert torch.equal(m(x), other(x))


@pytest.mark.parametrize("build", ["method", "to", "default dtype"])
def test_balance_stays_fp32(build):
    """The balance is a sum of small steps and the routing's fp32 bias: casting the layer casts the weights only."""
    torch.manual_seed(5)
    dtype = torch.get_default_dtype()
    try:
        if build == "default dtype":
            torch.set_default_dtype(torch.bfloat16)
        m = MXFP4MoE(64, 64, 4, 2, balance=True, device="cuda", dtype=torch.bfloat16 if build == "default dtype" else torch.float32)
    finally:
        torch.set_default_dtype(dtype)
    steps = torch.tensor([1.0, -1.0, 1.0, 1.0], device="cuda") * 1.0009765625   # not a bf16 value
    m.balance += steps
    m = m.bfloat16() if build == "method" else m.to(torch.bfloat16)
    assert m.w1.dtype == torch.bfloat16 and m.balance.dtype == torch.float32 and torch.equal(m.balance, steps)
    x = rnd(20, 64, seed=1, dtype=torch.bfloat16)
    out, counts = m(x, return_counts=True)
    out.sum().backward()
    m.update_balance(torch.tensor([1, 9, 1, 1], device="cuda"))
    assert torch.equal(m.balance, steps + 1e-3 * torch.tensor([1.0, -1.0, 1.0, 1.0], device="cuda"))
    m.load_state_dict({n: v.bfloat16() for n, v in m.state_dict().items()}, assign=True)
    m(x)
    assert m.cpu().balance.device.type == "cpu" and m.balance.dtype == torch.float32 and "balance" in m.state_dict()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale_mode", ["page", "floor"])
def test_expert_operands(dtype, scale_mode):
    """Whole scale atoms, ragged ones and transposed storage: expert by expert."""
    for w in (rnd(3, 256, 96, seed=4, dtype=dtype), rnd(3, 72, 64, seed=5, dtype=dtype),
              rnd(3, 64, 128, seed=6, dtype=dtype).transpose(1, 2)):
        codes, scales, values = moe.moe_expert_operands(w, scale_mode=scale_mode, values=True)
        for e in range(3):
            q = ops.mxfp4_qdq_fwd(w[e], block=32, scale_mode=scale_mode, emit_codes=True, scales_layout="mma")
            assert torch.equal(codes[e], q.codes_row) and torch.equal(scales[e], q.scales_row) and torch.equal(values[e], q.y_row)


@pytest.mark.parametrize("counts", [[3, 4], [-1, 2], [7, 0]])
def test_counts_that_do_not_fit(counts):
    x, w = rnd(6, 64, seed=7), rnd(2, 8, 64, seed=8)
    c = torch.tensor(counts).cuda()
    with pytest.raises(MXFP4ArgumentError):
        moe.moe_grouped_linear(x, w, c)
    assert not moe.moe_grouped_linear(x, w, c, check=False).any()


@pytest.mark.parametrize("counts", [[3, 4], [-1, 2], [7, 0]])
@pytest.mark.parametrize("rows", [6, 40])
def test_gradients_for_counts_that_do_not_fit(counts, rows):
    """Results are zeros without a check, and so is every gradient, the bias's too."""
    counts = [c * rows // 6 + (1 if c == 7 else 0) for c in counts]
    x, w, b = (v.requires_grad_(True) for v in (rnd(rows, 64, seed=7), rnd(2, 8, 64, seed=8), rnd(2, 8, seed=9)))
    y = moe.moe_grouped_linear(x, w, torch.tensor(counts).cuda(), b, check=False)
    for _ in range(4):      # what the allocator hands out next is not zero
        torch.full((2, 8), 7.0, device="cuda")
    y.sum().backward()
    for v in (x, w, b):
        assert not v.grad.any()


def test_optimiser_steps_run():
    torch.manual_seed(2)
    m = MXFP4MoE(64, 64, 4, 2, device="cuda", dtype=torch.float32)
    opt = torch.optim.SGD(m.parameters(), lr=1e-2)
    before = [p.detach().clone() for p in m.parameters()]
    for i in range(2):
        opt.zero_grad()
        m(rnd(50, 64, seed=i)).square().mean().backward()
        opt.step()
    assert all(bool(torch.isfinite(p).all()) and not torch.equal(p, q) for p, q in zip(m.parameters(), before))


def test_refusals():
    with pytest.raises(ValueError):
        MXFP4MoE(100, 64, 4, 2)
    with pytest.raises(ValueError):
        MXFP4MoE(64, 64, 4, 2, scale_mode="ceil")
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(rnd(4, 64), rnd(2, 8, 128), torch.tensor([2, 2]).cuda())
    m = MXFP4MoE(64, 64, 4, 2, device="cuda")
    with pytest.raises(ValueError):
        m.update_balance(torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        m(torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(2, dtype=torch.bool, device="cuda"))
