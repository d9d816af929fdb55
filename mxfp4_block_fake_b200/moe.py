"""Mixture-of-experts layers over the CUDA library.

  moe_route(logits, k, ...)          differentiable routing (weights) with its plan
  moe_dispatch(x, route)             token rows in expert order, differentiable
  moe_combine(y, route, weights)     expert rows back per token, differentiable
  moe_grouped_linear(x, weight, ..)  the experts' products on MXFP4 operands, differentiable
  MXFP4MoE                           router, gated experts and combination as one module

The products run on real MXFP4 operands (blocks of 32 along the contraction):
an expert's output is what fake-quantised activations and weights would give,
accumulated in fp32. Their backward is the straight-through one: the
activation's gradient by the library's kernel from the stored pre-activation,
then plain per-expert products with the fake-quantised values.
"""
from __future__ import annotations

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import ops
from .qat import SCALE_FACTOR, _Spec


def _not_captured(what: str) -> None:
    """The backwards here are refused under stream capture: the experts'
    products copy counts to the host, and autograd's own joining of a leaf's
    eager stream with a capturing one ends the process. Forwards can be
    captured, and so can the ops' own backward calls."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"the backward of {what} cannot be captured into a CUDA graph; call the ops entry points instead")


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, kw):
        r = ops.mxfp4_moe_route(logits, k, **kw)
        ctx.save_for_backward(logits, r.experts)
        ctx.rule = {n: kw[n] for n in ("score", "renormalize", "scale") if n in kw}
        ctx.mark_non_differentiable(r.experts, r.rows, r.slots, r.counts)
        return r.weights, r.experts, r.rows, r.slots, r.counts

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, *_):
        _not_captured("moe_route")
        logits, experts = ctx.saved_tensors
        return ops.mxfp4_moe_route_bwd(grad, logits, experts, **ctx.rule), None, None


def moe_route(logits: torch.Tensor, k: int, **kw) -> ops.RouteResult:
    """ops.mxfp4_moe_route whose weights carry gradients to the logits."""
    return ops.RouteResult(*_Route.apply(logits, k, kw))


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows):
        ctx.save_for_backward(rows)
        out = torch.zeros((rows.numel(), x.shape[1]), dtype=x.dtype, device=x.device)  # rows of no pair: zero
        return ops.mxfp4_moe_dispatch(x, rows, out=ops.DispatchResult(values=out)).values

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        _not_captured("moe_dispatch")
        (rows,) = ctx.saved_tensors
        return ops.mxfp4_moe_combine(grad, rows), None


def moe_dispatch(x: torch.Tensor, route: ops.RouteResult) -> torch.Tensor:
    """x [tokens, cols] -> [tokens * k, cols] in the route's expert order; rows
    behind the last pair are zero."""
    return _Dispatch.apply(x, route.rows)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, rows, weights, residual):
        ctx.save_for_backward(y, rows, weights)
        ctx.has_residual = residual is not None
        return ops.mxfp4_moe_combine(y, rows, weights, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        _not_captured("moe_combine")
        y, rows, weights = ctx.saved_tensors
        need_y, _, need_w, _ = ctx.needs_input_grad
        gy = gw = None
        if need_y or need_w:
            gy, gw = ops.mxfp4_moe_combine_bwd(grad, y, rows, weights, grad_rows=need_y, grad_weights=need_w,
                                               out=torch.zeros_like(y) if need_y else None)
        return gy, None, gw, grad if ctx.has_residual else None


def moe_combine(y: torch.Tensor, route: ops.RouteResult, weights: torch.Tensor | None = None,
                residual: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = residual[t] + sum_j weights[t, j] y[rows[t, j]]; weights
    default to the route's."""
    return _Combine.apply(y, route.rows, route.weights if weights is None else weights, residual)


def _operand(spec: _Spec, x: torch.Tensor, values: bool) -> ops.QDQResult:
    """Codes and MMA-layout scales of x's rows, and on request the values they stand for."""
    return ops.mxfp4_qdq_fwd(x, block=32, scale_factor=spec.divisor, scale_mode=spec.rule, emit_values=values,
                             emit_codes=True, scales_layout="mma")


def moe_expert_operands(weight: torch.Tensor, scale_factor: float = SCALE_FACTOR, scale_mode: str = "page",
                        values: bool = False):
    """Expert weights [E, n, k] as the operand of mxfp4_grouped_linear: codes
    [E, n, k / 2], E scale buffers, and (values) the values they stand for."""
    spec = _Spec.of(32, scale_factor, scale_mode)
    e, n, k = weight.shape
    if n % 128 == 0 and weight.is_contiguous():  # whole scale atoms: the experts' buffers are those of one matrix
        q = _operand(spec, weight.detach().view(e * n, k), values)
        return q.codes_row.view(e, n, -1), q.scales_row.view(e, -1), q.y_row.view(e, n, k) if values else None
    parts = [_operand(spec, w, values) for w in weight.detach()]
    codes = torch.stack([p.codes_row for p in parts])
    scales = torch.stack([p.scales_row for p in parts])
    return codes, scales, torch.stack([p.y_row for p in parts]) if values else None


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, counts, activation, scale_factor, scale_mode, check):
        spec = _Spec.of(32, scale_factor, scale_mode)
        xq = _operand(spec, x, True)
        codes, scales, wq = moe_expert_operands(weight, scale_factor, scale_mode, values=True)
        m, n = x.shape[0], weight.shape[1]
        zeros = lambda cols: torch.zeros((m, cols), dtype=x.dtype, device=x.device)  # noqa: E731 (rows of no expert)
        out = ops.LinearResult(y=zeros(n // 2 if activation == "swiglu" else n), preact=zeros(n))
        r = ops.mxfp4_grouped_linear(xq.codes_row, xq.scales_row, codes, scales, counts, k=x.shape[1], group_list_type=1,
                                     bias=bias, activation=activation, out_dtype=x.dtype, out=out, check=check)
        ctx.save_for_backward(xq.y_row, wq, r.preact, counts)
        ctx.activation, ctx.has_bias = activation, bias is not None
        return r.y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        _not_captured("moe_grouped_linear")
        xq, wq, preact, counts = ctx.saved_tensors
        gz, gb = ops.mxfp4_grouped_linear_bwd(grad, preact, counts, group_list_type=1, activation=ctx.activation,
                                              bias_grad=ctx.has_bias, check=False, out=torch.zeros_like(preact))
        gx, gw = torch.zeros_like(xq), torch.zeros_like(wq)
        first = 0
        for e, size in enumerate(counts.tolist()):
            if size:
                rows = slice(first, first + size)
                torch.mm(gz[rows], wq[e], out=gx[rows])
                torch.mm(gz[rows].t(), xq[rows], out=gw[e])
            first += size
        return gx, gw, gb, None, None, None, None, None


def moe_grouped_linear(x: torch.Tensor, weight: torch.Tensor, counts: torch.Tensor, bias: torch.Tensor | None = None,
                       activation: str = "none", scale_factor: float = SCALE_FACTOR, scale_mode: str = "page",
                       check: bool = True) -> torch.Tensor:
    """act(Q(x_e) Q(W_e)^T + b_e) for the rows that counts gives to each expert
    (x in expert order; rows behind them give zero). weight [E, n, k], k a
    multiple of 64; bias float32 [E, n]; activation as in
    ops.mxfp4_grouped_linear. check synchronises and raises for counts that are
    negative or exceed the rows (without it such counts give zeros, and zero
    gradients); counts of moe_route need none. The backward copies counts to
    the host."""
    if weight.ndim != 3 or x.ndim != 2 or weight.shape[2] != x.shape[1] or weight.dtype != x.dtype:
        raise ValueError("x must be [rows, k] and weight [experts, n, k], of one dtype")
    return _GroupedLinear.apply(x, weight, bias, counts, activation, scale_factor, scale_mode, bool(check))


class MXFP4MoE(nn.Module):
    """out = x + sum_j w_j E_j(x) over each token's k experts, with gated experts
    E(x) = (silu(x G^T) * (x U^T)) D^T on MXFP4 operands.

    Parameters: router [experts, cols]; w1 [experts, 2 hidden, cols], whose rows
    are gate and up rows in turn; w2 [experts, cols, hidden]. cols and hidden
    are multiples of 64. The router's logits are formed in the layer's dtype, and
    groups are ranked by their two best keys. balance (with balance=True) is a
    buffer added to the scores for the choice only; update_balance moves it
    against the load. It stays float32 when the layer is cast or loaded.

    With gradients enabled the forward quantises the weights each call. For
    serving, lay_out() quantises them once, and forwards without gradients use
    that copy until a weight is loaded, changed, replaced or moved, or the scale
    rule changes (in-place changes as autograd counts them; call it again after
    others, such as through .data or by a replayed graph). A copy of the layer
    starts without one, and weights made in inference mode, whose changes are
    not counted, are refused."""

    def __init__(self, cols: int, hidden: int, experts: int, k: int, *, score: str = "softmax", num_groups: int = 1,
                 topk_groups: int | None = None, renormalize: bool = True, scale: float = 1.0, balance: bool = False,
                 scale_factor: float = SCALE_FACTOR, scale_mode: str = "page", device=None, dtype=torch.bfloat16) -> None:
        super().__init__()
        if cols % 64 or hidden % 64:
            raise ValueError("cols and hidden must be multiples of 64")
        _Spec.of(32, scale_factor, scale_mode)
        self.k, self.scale_factor, self.scale_mode = k, float(scale_factor), scale_mode
        self.rule = dict(score=score, num_groups=num_groups, topk_groups=topk_groups, renormalize=renormalize, scale=scale)
        kw = dict(device=device, dtype=dtype)
        self.router = nn.Parameter(torch.randn(experts, cols, **kw) * cols ** -0.5)
        self.w1 = nn.Parameter(torch.randn(experts, 2 * hidden, cols, **kw) * cols ** -0.5)
        self.w2 = nn.Parameter(torch.randn(experts, cols, hidden, **kw) * hidden ** -0.5)
        self.register_buffer("balance", torch.zeros(experts, dtype=torch.float32, device=device) if balance else None)
        self._laid_out = None

    def lay_out(self) -> "MXFP4MoE":
        """Quantises the experts' weights for serving."""
        if self.w1.is_inference() or self.w2.is_inference():
            raise RuntimeError("weights made in inference mode cannot be laid out: their changes are not counted")
        q = dict(scale_factor=self.scale_factor, scale_mode=self.scale_mode)
        self._laid_out = (moe_expert_operands(self.w1, **q)[:2], moe_expert_operands(self.w2, **q)[:2], (self.w1, self.w2), self._changes())
        return self

    def _changes(self):
        """The storage and the count of in-place changes of the experts' weights, and the scale rule."""
        weights = [(w.data_ptr(), -1 if w.is_inference() else w._version) for w in (self.w1, self.w2)]
        return weights, self.scale_factor, self.scale_mode

    def _copy_is_current(self) -> bool:
        if self._laid_out is None:
            return False
        _, _, (w1, w2), changes = self._laid_out
        return w1 is self.w1 and w2 is self.w2 and changes == self._changes()

    def __getstate__(self):
        return {**self.__dict__, "_laid_out": None}  # a copy's weights count their changes from 0 again

    def _apply(self, fn, recurse=True):
        self._laid_out = None  # moved or cast: the copy is of the old weights
        balance = self.balance
        super()._apply(fn, recurse)
        if balance is not None and self.balance.dtype != torch.float32:  # cast with the weights: its fp32 value again
            self.balance = balance.to(self.balance.device)
        return self

    def _load_from_state_dict(self, *args, **kw):
        self._laid_out = None
        super()._load_from_state_dict(*args, **kw)
        if self.balance is not None:
            self.balance = self.balance.float()  # (assigned, it may be of another type)

    @torch.no_grad()
    def update_balance(self, counts: torch.Tensor, rate: float = 1e-3) -> None:
        """Raises the balance of experts below the mean load, lowers the others'."""
        if self.balance is None:
            raise ValueError("the layer was built without balance")
        load = counts.float()
        self.balance += rate * torch.sign(load.mean() - load)

    def forward(self, x: torch.Tensor, token_mask: torch.Tensor | None = None, return_counts: bool = False):
        shape = x.shape
        x2 = x.reshape(-1, shape[-1])
        logits = torch.nn.functional.linear(x2, self.router).float()
        mask = None if token_mask is None else token_mask.reshape(-1)
        r = moe_route(logits, self.k, bias=self.balance, token_mask=mask, **self.rule)
        q = dict(scale_factor=self.scale_factor, scale_mode=self.scale_mode)
        if torch.is_grad_enabled() or not self._copy_is_current():
            h = moe_grouped_linear(moe_dispatch(x2, r), self.w1, r.counts, activation="swiglu", check=False, **q)
            y = moe_grouped_linear(h, self.w2, r.counts, check=False, **q)
        else:
            (c1, s1), (c2, s2), *_ = self._laid_out
            d = ops.mxfp4_moe_dispatch(x2, r.rows, emit_values=False, emit_codes=True, **q)
            h = ops.mxfp4_grouped_linear(d.codes, d.scales, c1, s1, r.counts, k=x2.shape[1], group_list_type=1,
                                         activation="swiglu", out_dtype=x2.dtype, check=False).y
            hq = _operand(_Spec.of(32, self.scale_factor, self.scale_mode), h, False)
            y = ops.mxfp4_grouped_linear(hq.codes_row, hq.scales_row, c2, s2, r.counts, k=h.shape[1], group_list_type=1,
                                         out_dtype=x2.dtype, check=False).y
        out = moe_combine(y, r, residual=x2).view(shape)
        return (out, r.counts) if return_counts else out
