"""Token rows sorted by expert and back in token order, with their gradients.

For experts of the caller's own between the library's dispatch and its
weighted return: ``permute_rows`` copies each token's row to its k segment
slots, ``unpermute_rows`` sums a token's k rows with the routing weights. Both
take part in autograd (in ``x``; in ``y_perm``, ``routing_weights`` and
``shared_out``), once and in reverse mode: tensors with a forward-mode tangent
are refused. Plan and routing weights must stay as they are until the backward
pass (overwriting them makes it raise). ``permute_rows_backward`` and
``unpermute_rows_backward`` are their gradients as plain calls. The plan is
what ``dispatch`` or ``dispatch_slots`` returned for the same problem.

    plan = stm.dispatch(p, selected_experts)
    rows = stm.permute_rows(p, x, plan)                 # [T*k, H], by expert
    y = my_experts(rows, plan["offsets"])
    out = stm.unpermute_rows(p, y, plan, routing_weights)

Forward and backward can be captured in a CUDA graph. Capture ``backward()``
only while no eager graph of the same leaves is alive (drop its outputs
first), or take the gradients with ``torch.autograd.grad``: autograd adds a
leaf's gradient on the stream of the first graph that it is part of, which a
capture on another stream does not survive.
"""

from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import DTYPES, TORCH_DTYPE, Problem, _launch, _ptr, _req, lib


def _req_at(t, name: str, shape: Tuple[int, ...], dtype: torch.dtype, index: int) -> None:
    """_req, on the CUDA device of that index."""
    if (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype == dtype and t.shape == shape
            and t.is_contiguous()):
        return
    _req(t, name, shape, dtype)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _plan(p: Problem, plan: Dict[str, torch.Tensor], index: int) -> Tuple[torch.Tensor, torch.Tensor]:
    pair_pos, offsets = plan["pair_pos"], plan["offsets"]
    _req_at(pair_pos, "pair_pos", (p.T * p.k,), torch.int32, index)
    _req_at(offsets, "offsets", (p.E + 1,), torch.int32, index)
    return pair_pos, offsets


def _req_y(p: Problem, y_perm) -> int:
    """The moe_dtype of y_perm [T*k, H]: fp32, or the problem's."""
    if isinstance(y_perm, torch.Tensor) and y_perm.dtype == torch.float32:
        _req(y_perm, "y_perm", (p.T * p.k, p.H), torch.float32)
        return DTYPES["f32"]
    _req(y_perm, "y_perm", (p.T * p.k, p.H), TORCH_DTYPE[p.dtype])
    return DTYPES[p.dtype]


def _permute(p: Problem, x, pair_pos, offsets):
    dev = x.device
    out = torch.empty(p.T * p.k, p.H, dtype=x.dtype, device=dev)
    _launch(lib().moe_permute_rows, dev, p._struct(), x.data_ptr(), pair_pos.data_ptr(), offsets.data_ptr(), out.data_ptr())
    return out


def _permute_backward(p: Problem, dx_perm, pair_pos):
    dev = dx_perm.device
    dx = torch.empty(p.T, p.H, dtype=dx_perm.dtype, device=dev)
    _launch(lib().moe_permute_rows_backward, dev, p._struct(), dx_perm.data_ptr(), pair_pos.data_ptr(), dx.data_ptr())
    return dx


def _unpermute(p: Problem, yd: int, y_perm, pair_pos, routing_weights, shared_out):
    dev = y_perm.device
    out = torch.empty(p.T, p.H, dtype=TORCH_DTYPE[p.dtype], device=dev)
    _launch(lib().moe_unpermute_rows, dev, p._struct(), yd, y_perm.data_ptr(), pair_pos.data_ptr(), _ptr(routing_weights),
            _ptr(shared_out), out.data_ptr())
    return out


def _unpermute_backward(p: Problem, yd: int, dout, y_perm, pair_pos, offsets, routing_weights, rows: bool,
                        weights: bool):
    dev = dout.device
    dy = torch.empty(p.T * p.k, p.H, dtype=torch.float32 if yd == DTYPES["f32"] else TORCH_DTYPE[p.dtype],
                     device=dev) if rows else None
    dw = torch.empty(p.T, p.k, dtype=torch.float32, device=dev) if weights else None
    if rows or weights:
        _launch(lib().moe_unpermute_rows_backward, dev, p._struct(), yd, dout.data_ptr(), _ptr(y_perm), pair_pos.data_ptr(),
                offsets.data_ptr(), _ptr(routing_weights), _ptr(dy), _ptr(dw))
    return dy, dw


def _whole(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and on a 16-byte boundary: autograd may hand on a view of any strides and offset."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _tangent(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether one of them has a forward-mode tangent. (Such a tensor need not require a gradient, and a call past
    autograd would drop the tangent; asked only while a level is open, which costs a call nothing.)"""
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _no_jvp(*_):
    raise NotImplementedError("permute_rows and unpermute_rows have no forward-mode derivative")


class _PermuteRows(torch.autograd.Function):
    jvp = staticmethod(_no_jvp)

    @staticmethod
    def forward(ctx, x, p, pair_pos, offsets):
        ctx.p = p
        ctx.save_for_backward(pair_pos)
        return _permute(p, x, pair_pos, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dx_perm):
        (pair_pos,) = ctx.saved_tensors
        return _permute_backward(ctx.p, _whole(dx_perm), pair_pos), None, None, None


class _UnpermuteRows(torch.autograd.Function):
    jvp = staticmethod(_no_jvp)

    @staticmethod
    def forward(ctx, y_perm, routing_weights, shared_out, p, yd, pair_pos, offsets):
        ctx.p, ctx.yd = p, yd
        needs_y = ctx.needs_input_grad[1]  # the rows themselves enter the weights' gradient only
        ctx.save_for_backward(y_perm if needs_y else None, routing_weights, pair_pos, offsets)
        return _unpermute(p, yd, y_perm, pair_pos, routing_weights, shared_out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y_perm, routing_weights, pair_pos, offsets = ctx.saved_tensors
        dout = _whole(dout)
        rows, weights, shared = ctx.needs_input_grad[:3]
        dy, dw = _unpermute_backward(ctx.p, ctx.yd, dout, y_perm, pair_pos, offsets, routing_weights, rows, weights)
        return dy, dw, dout.float() if shared else None, None, None, None, None


def permute_rows(p: Problem, x, plan: Dict[str, torch.Tensor]):
    """x_perm [T*k, H]: each token's row of x [T, H] copied to its k sorted
    positions. Rows past the last segment are zeros. Differentiable in x."""
    _req(x, "x", (p.T, p.H), TORCH_DTYPE[p.dtype])
    pair_pos, offsets = _plan(p, plan, x.get_device())
    if (x.requires_grad and torch.is_grad_enabled()) or _tangent(x):
        return _PermuteRows.apply(x, p, pair_pos, offsets)
    return _permute(p, x, pair_pos, offsets)


def permute_rows_backward(p: Problem, dx_perm, plan: Dict[str, torch.Tensor]):
    """dx [T, H] from dx_perm [T*k, H] (both in the problem's dtype): the sum
    of each token's k rows, in fp32, rounded once."""
    _req(dx_perm, "dx_perm", (p.T * p.k, p.H), TORCH_DTYPE[p.dtype])
    pair_pos, _ = _plan(p, plan, dx_perm.get_device())
    return _permute_backward(p, dx_perm, pair_pos)


def unpermute_rows(p: Problem, y_perm, plan: Dict[str, torch.Tensor], routing_weights=None, shared_out=None):
    """out [T, H]: sum over each token's slots of routing_weights [T, k] (fp32;
    1 when None) times its row of y_perm [T*k, H] (fp32 or the problem's
    dtype), plus shared_out [T, H] fp32 when given; summed in fp32, rounded
    once to the problem's dtype. A slot without a row adds nothing.
    Differentiable in y_perm, routing_weights and shared_out."""
    yd = _req_y(p, y_perm)
    index = y_perm.get_device()
    pair_pos, offsets = _plan(p, plan, index)
    grad = y_perm.requires_grad
    if routing_weights is not None:
        _req_at(routing_weights, "routing_weights", (p.T, p.k), torch.float32, index)
        grad = grad or routing_weights.requires_grad
    if shared_out is not None:
        _req_at(shared_out, "shared_out", (p.T, p.H), torch.float32, index)
        grad = grad or shared_out.requires_grad
    if (grad and torch.is_grad_enabled()) or _tangent(y_perm, routing_weights, shared_out):
        return _UnpermuteRows.apply(y_perm, routing_weights, shared_out, p, yd, pair_pos, offsets)
    return _unpermute(p, yd, y_perm, pair_pos, routing_weights, shared_out)


def unpermute_rows_backward(p: Problem, dout, y_perm, plan: Dict[str, torch.Tensor], routing_weights=None):
    """(dy_perm [T*k, H] in y_perm's dtype, d_routing_weights [T, k] fp32) for
    dout [T, H]: each row's gradient is its weight times dout (rows past the
    last segment are zeros), each weight's the product of dout and its row (0
    for a slot without a row)."""
    yd = _req_y(p, y_perm)
    index = y_perm.get_device()
    _req_at(dout, "dout", (p.T, p.H), TORCH_DTYPE[p.dtype], index)
    pair_pos, offsets = _plan(p, plan, index)
    if routing_weights is not None:
        _req_at(routing_weights, "routing_weights", (p.T, p.k), torch.float32, index)
    return _unpermute_backward(p, yd, dout, y_perm, pair_pos, offsets, routing_weights, True, True)
