"""Autograd layers over the library's kernels: Float8Linear, a Linear layer whose GEMMs
run in FP8; AddNorm, the normalization of a residual stream with the addition into it;
route, an expert router whose sorted rows and offsets the grouped GEMMs take.

Float8Linear is one autograd node with a hand-written backward, as in "FP8
Training: Quantization, Autograd, Torchao", section 6: the quantization and
the scaled GEMMs are not recorded op by op. Forward and backward are single
calls of the C ABI (fp8_linear_fwd / fp8_linear_bwd), so every step of the
math runs in this package's HIP kernels; this module only allocates outputs
and workspaces and reshapes.

Recipes ("FP8 training on AMD GPUs with TorchTitan and TorchAO", Figure 1
caption):
  - "rowwise": per-row e4m3 scales for x and w in the forward, e5m2 per row
    for grad_out, w per column for grad-input, grad-weight in BF16;
  - "tensorwise": one scale per tensor, all three GEMMs in FP8 (the
    grad-weight GEMM takes grad_out and x transposed, written by one dual
    quantization launch); needs a multiple of 16 rows.

What the backward keeps: the bf16 input and weight (references, no copy).
The kernels write every FP8 operand in the layout its GEMM reads straight
from bf16, so the backward re-quantizes instead of transposing FP8 copies
saved by the forward; a deterministic quantizer gives the forward's bytes.

AddNorm and route are one node each as well (fp8_add_norm_quant_row / fp8_add_norm_bwd,
fp8_moe_route / fp8_moe_route_bwd). As for any node, a backward pass captured into a
graph needs leaves whose gradients were not accumulated on another stream: capture
forward and backward together, with torch.autograd.grad or fresh gradients.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import (E4M3_NATIVE, GATE_SIGMOID, GATE_SOFTMAX, GATE_SOFTMAX_TOPK, NORM_LAYER, NORM_RMS, OUT_BF16,
               RECIPE_ROWWISE_BF16_WGRAD, RECIPE_TENSORWISE, fp8_add_norm_bwd, fp8_add_norm_bwd_ws_bytes,
               fp8_add_norm_quant_row, fp8_linear_bwd, fp8_linear_fwd, fp8_linear_ws_bytes, fp8_moe_route,
               fp8_moe_route_bwd, fp8_moe_route_ws_bytes, load)

_NORMS = {"rms": NORM_RMS, "layer": NORM_LAYER}
_GATES = {"softmax": GATE_SOFTMAX, "softmax_topk": GATE_SOFTMAX_TOPK, "sigmoid": GATE_SIGMOID}
_RECIPES = {"rowwise": RECIPE_ROWWISE_BF16_WGRAD, "tensorwise": RECIPE_TENSORWISE}


def _check_operand(t: torch.Tensor, name: str):
    if t.device.type != "cuda":
        raise RuntimeError(f"Float8Linear: {name} must be on a ROCm GPU (got {t.device})")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"Float8Linear: {name} must be bfloat16 (got {t.dtype})")


class Float8LinearFunction(torch.autograd.Function):
    """y = x w^T through fp8_linear_fwd; grad_x, grad_w through fp8_linear_bwd.
    x [..., K] and w [N, K] bf16 on the GPU; y [..., N] bf16."""

    @staticmethod
    def forward(ctx, x, weight, recipe: int, eps: float):
        _check_operand(x, "input")
        _check_operand(weight, "weight")
        K = x.shape[-1]
        N = weight.shape[0]
        if weight.shape[1] != K:
            raise ValueError(f"Float8Linear: input has {K} features, weight expects {weight.shape[1]}")
        x2 = x.reshape(-1, K).contiguous()
        w = weight.contiguous()
        M = x2.shape[0]
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        ws = torch.empty(fp8_linear_ws_bytes(M, N, K, recipe), dtype=torch.uint8, device=x.device)
        fp8_linear_fwd(x2, w, recipe, eps, OUT_BF16, y, ws)
        ctx.save_for_backward(x2, w)
        ctx.recipe, ctx.eps, ctx.x_shape = recipe, eps, x.shape
        return y.reshape(*x.shape[:-1], N)

    @staticmethod
    def backward(ctx, grad_out):
        x2, w = ctx.saved_tensors
        M, K = x2.shape
        N = w.shape[0]
        gy = grad_out.reshape(-1, N)
        if gy.dtype != torch.bfloat16:
            gy = gy.to(torch.bfloat16)
        gy = gy.contiguous()
        gx = torch.empty((M, K), dtype=torch.bfloat16, device=x2.device)
        gw = torch.empty((N, K), dtype=torch.bfloat16, device=x2.device)
        ws = torch.empty(fp8_linear_ws_bytes(M, N, K, ctx.recipe), dtype=torch.uint8, device=x2.device)
        fp8_linear_bwd(gy, x2, w, ctx.recipe, ctx.eps, gx, gw, ws)
        return gx.reshape(ctx.x_shape), gw, None, None


class Float8Linear(torch.nn.Module):
    """Drop-in Linear (bf16 parameters) whose matmuls run in FP8.

    in_features must be a multiple of 16 and out_features a multiple of 16
    (the FP8 GEMM's contraction and the backward's column quantization); the
    tensorwise recipe also needs a multiple of 16 rows in the flattened
    input. The bias, if any, is added in bf16 after the FP8 GEMM."""

    def __init__(self, in_features: int, out_features: int, bias: bool = False, recipe: str = "rowwise",
                 eps: float = 1e-12, device=None):
        super().__init__()
        if recipe not in _RECIPES:
            raise ValueError(f"recipe must be one of {sorted(_RECIPES)}")
        self.in_features, self.out_features = in_features, out_features
        self.recipe, self.eps = recipe, float(eps)
        kw = dict(dtype=torch.bfloat16, device=device)
        self.weight = torch.nn.Parameter(torch.empty((out_features, in_features), **kw))
        self.bias = torch.nn.Parameter(torch.empty(out_features, **kw)) if bias else None
        self.reset_parameters()

    def reset_parameters(self):
        # the default initialization of torch.nn.Linear
        torch.nn.init.kaiming_uniform_(self.weight, a=math.sqrt(5))
        if self.bias is not None:
            bound = 1 / math.sqrt(self.in_features) if self.in_features > 0 else 0
            torch.nn.init.uniform_(self.bias, -bound, bound)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, recipe: str = "rowwise", eps: float = 1e-12):
        """A Float8Linear holding a bf16 copy of `linear`'s parameters."""
        m = cls(linear.in_features, linear.out_features, bias=linear.bias is not None, recipe=recipe, eps=eps,
                device=linear.weight.device)
        with torch.no_grad():
            m.weight.copy_(linear.weight.to(torch.bfloat16))
            if linear.bias is not None:
                m.bias.copy_(linear.bias.to(torch.bfloat16))
        return m

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        load()
        y = Float8LinearFunction.apply(x, self.weight, _RECIPES[self.recipe], self.eps)
        return y if self.bias is None else y + self.bias

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, recipe={self.recipe}")


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and from 16 bytes on, as the norm's kernels read it: a gradient may be a
    contiguous piece of a longer tensor, at any offset."""
    c = t.contiguous()
    return c if c.data_ptr() % 16 == 0 else c.clone()


class AddNormFunction(torch.autograd.Function):
    """h = x + res (bf16) and y = norm(h) through fp8_add_norm_quant_row, both differentiable; the
    gradients of x, res, gamma and beta through fp8_add_norm_bwd. res None: y alone, h = x."""

    @staticmethod
    def forward(ctx, x, res, gamma, beta, kind: int, norm_eps: float):
        for t, name in ((x, "input"), (res, "residual"), (gamma, "weight"), (beta, "bias")):
            if t is None:
                continue
            if t.device.type != "cuda":
                raise RuntimeError(f"AddNorm: {name} must be on a ROCm GPU (got {t.device})")
            if t.dtype != torch.bfloat16:
                raise TypeError(f"AddNorm: {name} must be bfloat16 (got {t.dtype})")
        if res is not None and res.shape != x.shape:
            raise ValueError(f"AddNorm: input {tuple(x.shape)} and residual {tuple(res.shape)} differ in shape")
        cols = x.shape[-1]
        for t, name in ((gamma, "weight"), (beta, "bias")):
            if t is not None and t.shape != (cols,):
                raise ValueError(f"AddNorm: input has {cols} features, {name} has {tuple(t.shape)}")
        x2 = _dense(x.reshape(-1, cols))
        rows = x2.shape[0]
        r2 = None if res is None else _dense(res.reshape(-1, cols))
        # the outputs have their own shape, not a view's: they may be changed in place
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h = x2 if res is None else torch.empty_like(y)
        stats = dict(dtype=torch.float32, device=x.device)
        mean = torch.empty(rows, **stats) if kind == NORM_LAYER else None
        rstd = torch.empty(rows, **stats)
        g = _dense(gamma)
        fp8_add_norm_quant_row(x2, r2, g, None if beta is None else _dense(beta), kind, norm_eps, E4M3_NATIVE,
                               1e-12, None if res is None else h.view(rows, cols), y.view(rows, cols), None, None,
                               mean=mean, rstd=rstd)
        ctx.save_for_backward(h, g, mean, rstd)
        ctx.kind, ctx.shape = kind, x.shape
        ctx.set_materialize_grads(False)
        return y if res is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, gamma, mean, rstd = ctx.saved_tensors
        cols = h.shape[-1]
        h = h.view(-1, cols)
        rows = h.shape[0]
        flat = lambda g: None if g is None else _dense(g.to(torch.bfloat16).reshape(rows, cols))  # noqa: E731
        dy, dh = flat(dy), flat(dh)
        if dy is None:  # only the stream behind h has a gradient
            dx = None if dh is None else dh.reshape(ctx.shape)
            return dx, dx, None, None, None, None
        dx = torch.empty_like(h)
        dgamma = torch.empty_like(gamma) if ctx.needs_input_grad[2] else None
        dbeta = torch.empty_like(gamma) if ctx.needs_input_grad[3] else None
        ws = None
        if dgamma is not None or dbeta is not None:
            ws = torch.empty(fp8_add_norm_bwd_ws_bytes(rows, cols, ctx.kind), dtype=torch.uint8, device=h.device)
        fp8_add_norm_bwd(dy, dh, h, gamma, mean, rstd, ctx.kind, dx, dgamma, dbeta, ws)
        dx = dx.reshape(ctx.shape)
        return dx, dx if ctx.needs_input_grad[1] else None, dgamma, dbeta, None, None


class AddNorm(torch.nn.Module):
    """RMSNorm ("rms") or LayerNorm ("layer") of a residual stream with bf16 parameters:
    forward(x, res) adds x into the stream and returns (norm(h), h) with h = x + res;
    forward(x) returns (norm(x), x). features must be a multiple of 8, at most 16384."""

    def __init__(self, features: int, kind: str = "rms", norm_eps: float = 1e-5, device=None):
        super().__init__()
        if kind not in _NORMS:
            raise ValueError(f"kind must be one of {sorted(_NORMS)}")
        self.features, self.kind, self.norm_eps = features, kind, float(norm_eps)
        kw = dict(dtype=torch.bfloat16, device=device)
        self.weight = torch.nn.Parameter(torch.ones(features, **kw))
        self.bias = torch.nn.Parameter(torch.zeros(features, **kw)) if kind == "layer" else None

    def forward(self, x: torch.Tensor, res: torch.Tensor | None = None):
        load()
        out = AddNormFunction.apply(x, res, self.weight, self.bias, _NORMS[self.kind], self.norm_eps)
        return (out, x) if res is None else out

    def extra_repr(self) -> str:
        return f"features={self.features}, kind={self.kind}, norm_eps={self.norm_eps}"


class Routing(NamedTuple):
    """A router's answer for T tokens: ids and weights [T][k] (the weights differentiable), the grouped
    GEMMs' offsets [E + 1], order [T * k] (the pair t * k + j of each sorted row, -1 behind the last)
    and slot [T][k] (the sorted row of each pair, -1 for none)."""

    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    order: torch.Tensor
    slot: torch.Tensor


class RouteFunction(torch.autograd.Function):
    """fp8_moe_route on logits [T][E]; the gradient of the weights through fp8_moe_route_bwd."""

    @staticmethod
    def forward(ctx, logits, k: int, gate: int):
        if logits.device.type != "cuda":
            raise RuntimeError(f"route: logits must be on a ROCm GPU (got {logits.device})")
        if logits.dim() != 2:
            raise ValueError(f"route: logits must be [tokens][experts] (got {tuple(logits.shape)})")
        l = logits.contiguous()
        T, E = l.shape
        i32 = dict(dtype=torch.int32, device=l.device)
        ids, weights = torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=l.device)
        offsets, order, slot = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty((T, k), **i32)
        ws = torch.empty(fp8_moe_route_ws_bytes(T, E, k), dtype=torch.uint8, device=l.device)
        fp8_moe_route(l, gate, ids, weights, offsets, order, slot, ws)
        ctx.save_for_backward(l, ids, weights)
        ctx.gate = gate
        ctx.mark_non_differentiable(ids, offsets, order, slot)
        ctx.set_materialize_grads(False)
        return ids, weights, offsets, order, slot

    @staticmethod
    @once_differentiable
    def backward(ctx, _ids, dweights, _offsets, _order, _slot):
        if dweights is None:
            return None, None, None
        l, ids, weights = ctx.saved_tensors
        dlogits = torch.empty_like(l)
        fp8_moe_route_bwd(l, ctx.gate, ids, weights, dweights.float().contiguous(), dlogits)
        return dlogits, None, None


def route(logits: torch.Tensor, k: int, gate: str = "softmax") -> Routing:
    """The k experts of each token with the largest logits ([T][E], bf16 or fp32), their gate weights
    ("softmax" over all experts, "softmax_topk" over the chosen, "sigmoid") and the rows sorted by
    expert, as fp8_moe_route defines them."""
    if gate not in _GATES:
        raise ValueError(f"gate must be one of {sorted(_GATES)}")
    load()
    return Routing(*RouteFunction.apply(logits, int(k), _GATES[gate]))
