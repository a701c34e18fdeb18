"""Microscaled 4-bit floating point: quantisation, the grouped products of
4-bit rows with 4-bit expert weights, and the layer that runs its routed
experts with both.

A value is an e2m1 code, and every 32 along the last dimension share one
power-of-two scale (``include/moe.h`` gives the format and the rounding).

    gate_up = stm.mx4_quantize(weights["gate_up"])      # once, after loading
    plan = stm.dispatch(p, selected_experts)
    rows = stm.mx4_permute_rows(p, x, plan)             # sorted by expert, 4 bits
    h = stm.mx4_grouped_gate_up(rows, gate_up, plan["offsets"], quantize=True)
    y = stm.mx4_grouped_matmul(h, down, plan["offsets"])
    out = stm.unpermute_rows(p, y, plan, routing_weights)

``Mx4SparseMoE`` is that as a layer, called like ``SparseMoE``.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import (DTYPES, TORCH_DTYPE, Problem, SparseMoE, _launch, _ptr, _req, dispatch, lib, new_workspace, route,
               shared_expert)
from .rows import _plan, _same_device, unpermute_rows

_DTYPE_ID = {TORCH_DTYPE[name]: i for name, i in DTYPES.items()}


@dataclass(frozen=True)
class Mx4:
    """Rows of 4-bit values: ``data`` uint8 [..., K/2], ``scale`` uint8 [..., 16*ceil(K/512)]."""

    data: torch.Tensor
    scale: torch.Tensor

    @property
    def K(self) -> int:
        return 2 * self.data.shape[-1]

    @property
    def shape(self) -> torch.Size:
        return self.data.shape[:-1] + (self.K,)

    @property
    def device(self) -> torch.device:
        return self.data.device

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        return mx4_dequantize(self, dtype)


def _scale_bytes(K: int) -> int:
    return 16 * -(-K // 512)


def _req_k(K: int, name: str) -> None:
    if K <= 0 or K % 32 != 0:
        raise ValueError(f"{name}: the last dimension is {K}, expected a positive multiple of 32")


def _req_mx4(q: Mx4, name: str, lead: Optional[Sequence[int]] = None) -> int:
    """K of q, which has leading dimensions `lead` (None: any)."""
    if not isinstance(q, Mx4):
        raise ValueError(f"{name} must be an Mx4")
    if not isinstance(q.data, torch.Tensor) or q.data.dim() < 1:
        raise ValueError(f"{name}.data must be a CUDA tensor of at least one dimension")
    shape = q.data.shape
    K = 2 * shape[-1]
    _req_k(K, name)
    lead = tuple(shape[:-1] if lead is None else lead)
    _req(q.data, f"{name}.data", lead + (K // 2,), torch.uint8)
    _req(q.scale, f"{name}.scale", lead + (_scale_bytes(K),), torch.uint8)
    if q.scale.get_device() != q.data.get_device():
        raise ValueError(f"{name}.scale is on {q.scale.device}, expected {q.data.device}")
    return K


def _new(lead: Tuple[int, ...], K: int, device) -> Mx4:
    return Mx4(torch.empty(lead + (K // 2,), dtype=torch.uint8, device=device),
               torch.empty(lead + (_scale_bytes(K),), dtype=torch.uint8, device=device))


def mx4_quantize(x: torch.Tensor) -> Mx4:
    """x [..., K] (bf16 or fp32, contiguous, K a multiple of 32) in 4 bits."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPE_ID:
        raise ValueError("x must be a bf16 or fp32 CUDA tensor")
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must have at least one dimension")
    _req(x, "x", shape, x.dtype)
    K = shape[-1]
    _req_k(K, "x")
    dev = x.device
    q = _new(tuple(shape[:-1]), K, dev)
    _launch(lib().moe_mx4_quantize, dev, x.numel() // K, K, _DTYPE_ID[x.dtype], x.data_ptr(), q.data.data_ptr(),
            q.scale.data_ptr())
    return q


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values q stands for, [..., K] in bf16 or fp32."""
    K = _req_mx4(q, "q")
    if dtype not in _DTYPE_ID:
        raise ValueError(f"dtype {dtype}, expected bf16 or fp32")
    dev = q.data.device
    out = torch.empty(q.data.shape[:-1] + (K,), dtype=dtype, device=dev)
    _launch(lib().moe_mx4_dequantize, dev, out.numel() // K, K, _DTYPE_ID[dtype], q.data.data_ptr(),
            q.scale.data_ptr(), out.data_ptr())
    return out


def mx4_permute_rows(p: Problem, x, plan: Dict[str, torch.Tensor]) -> Mx4:
    """``mx4_quantize(permute_rows(p, x, plan))``, each token quantised once:
    [T*k, H] in 4 bits, sorted by expert; rows past the last segment are zeros."""
    _req(x, "x", (p.T, p.H), TORCH_DTYPE[p.dtype])
    _req_k(p.H, "x")
    pair_pos, offsets = _plan(p, plan)
    dev = x.device
    _same_device(dev, pair_pos=pair_pos, offsets=offsets)
    q = _new((p.T * p.k,), p.H, dev)
    _launch(lib().moe_mx4_permute_rows, dev, p.c(), x.data_ptr(), pair_pos.data_ptr(), offsets.data_ptr(),
            q.data.data_ptr(), q.scale.data_ptr())
    return q


def _req_product(a: Mx4, w: Mx4, offsets, ws) -> int:
    """K of the product."""
    K = _req_mx4(a, "a")
    if _req_mx4(w, "w") != K:
        raise ValueError(f"a has K {K}, w {w.K}")
    if a.data.dim() != 2 or w.data.dim() != 3:
        raise ValueError("a must be [rows, K] and w [E, N, K]")
    _req(offsets, "offsets", (w.data.shape[0] + 1,), torch.int32)
    if ws is not None and (not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.numel() * ws.element_size() < 256):
        raise ValueError("ws must be a workspace")
    _same_device(a.data.device, w=w.data, offsets=offsets, ws=ws)
    return K


def mx4_grouped_matmul(a: Mx4, w: Mx4, offsets, out_dtype: torch.dtype = torch.bfloat16, ws=None) -> torch.Tensor:
    """[rows, N]: each row of a [rows, K] times its expert's w [E, N, K], for
    the segments of offsets [E+1]; fp32 accumulation, bf16 or fp32 result.
    Rows outside every segment are not written. N must be a multiple of 8.
    ``ws``: a workspace for the error bits (``read_device_error``)."""
    K = _req_product(a, w, offsets, ws)
    if out_dtype not in _DTYPE_ID:
        raise ValueError(f"out_dtype {out_dtype}, expected bf16 or fp32")
    rows, (E, N, _) = a.data.shape[0], w.data.shape
    dev = a.data.device
    out = torch.empty(rows, N, dtype=out_dtype, device=dev)
    _launch(lib().moe_mx4_grouped_matmul, dev, rows, E, N, K, _DTYPE_ID[out_dtype], a.data.data_ptr(),
            a.scale.data_ptr(), offsets.data_ptr(), w.data.data_ptr(), w.scale.data_ptr(), out.data_ptr(), _ptr(ws))
    return out


def mx4_grouped_gate_up(a: Mx4, w: Mx4, offsets, quantize: bool = False, ws=None):
    """SwiGLU of each row of a [rows, H] with its expert's w [E, 2I, H] (gate
    rows first): h [rows, I] bf16, or with ``quantize`` that in 4 bits (the
    same bits as ``mx4_quantize`` of it). Rows outside every segment are not
    written. I must be a multiple of 32."""
    K = _req_product(a, w, offsets, ws)
    rows, (E, two_i, _) = a.data.shape[0], w.data.shape
    if two_i % 64 != 0:
        raise ValueError(f"w has {two_i} rows per expert, expected a multiple of 64 (twice a multiple of 32)")
    I = two_i // 2
    dev = a.data.device
    h = _new((rows,), I, dev) if quantize else torch.empty(rows, I, dtype=torch.bfloat16, device=dev)
    data, scale = (h.data, h.scale.data_ptr()) if quantize else (h, None)
    _launch(lib().moe_mx4_grouped_gate_up, dev, rows, E, I, K, a.data.data_ptr(), a.scale.data_ptr(),
            offsets.data_ptr(), w.data.data_ptr(), w.scale.data_ptr(), data.data_ptr(), scale, _ptr(ws))
    return h


class Mx4SparseMoE(SparseMoE):
    """A ``SparseMoE`` whose routed experts hold 4-bit weights and run 4-bit
    products. ``weights`` as there; gate_up and down in the problem's dtype
    (quantised here, once) or as ``Mx4``. The router and the shared expert keep
    their weights; the shared expert runs on the caller's stream. bf16
    problems, H and I multiples of 32."""

    def __init__(self, p: Problem, weights: Dict[str, Optional[torch.Tensor]], device="cuda",
                 overlap_shared: bool = False):
        if p.dtype != "bf16":
            raise ValueError("4-bit experts need a bf16 problem")
        if overlap_shared:
            raise ValueError("4-bit experts run the shared expert on the caller's stream")
        _req_k(p.H, "H")
        _req_k(p.I, "I")
        dt = p.torch_dtype
        w = dict(weights)
        for name, shape in (("gate_up", (p.E, 2 * p.I, p.H)), ("down", (p.E, p.H, p.I))):
            if not isinstance(w[name], Mx4):
                _req(w[name], name, shape, dt)
                w[name] = mx4_quantize(w[name])
            _req_mx4(w[name], name, shape[:2])
            if w[name].K != shape[2]:
                raise ValueError(f"{name}: K {w[name].K}, expected {shape[2]}")
        _req(w["gate_w"], "gate_w", (p.E, p.H), dt)
        if (p.bias_mode != "none") != (w.get("bias") is not None):
            raise ValueError("a bias goes with bias_mode 'logit' or 'select'")
        if (p.shared == "sigmoid_gated") != (w.get("shared_gate") is not None):
            raise ValueError("shared_gate goes with shared 'sigmoid_gated'")
        self.p, self.w = p, w
        self.device = torch.device(device)
        self.ws = new_workspace(p, self.device)
        self.aux = None
        self._counts = torch.zeros(p.E, dtype=torch.int32, device=self.device)

    def forward(self, x, out=None, routing_weights=None, selected_experts=None, events=None):
        """out, routing_weights, selected_experts = moe(x), as SparseMoE's."""
        if events is not None:
            raise ValueError("stage events are recorded by SparseMoE only")
        p, w = self.p, self.w
        rw, sel, gamma = route(p, x, w["gate_w"], w.get("bias"), w.get("shared_gate"), ws=self.ws)
        plan = dispatch(p, sel, ws=self.ws)
        self._counts = plan["counts"]
        rows = mx4_permute_rows(p, x, plan)
        h = mx4_grouped_gate_up(rows, w["gate_up"], plan["offsets"], quantize=True, ws=self.ws)
        y = mx4_grouped_matmul(h, w["down"], plan["offsets"], ws=self.ws)
        shared = None
        if p.shared != "none":
            shared = shared_expert(p, x, w["shared_gate_up"], w["shared_down"], gamma, ws=self.ws)
        with torch.no_grad():
            got = unpermute_rows(p, y, plan, rw, shared)
        for given, made in ((out, got), (routing_weights, rw), (selected_experts, sel)):
            if given is not None:
                given.copy_(made)
        return (got if out is None else out, rw if routing_weights is None else routing_weights,
                sel if selected_experts is None else selected_experts)

    __call__ = forward

    def forward_counts(self) -> torch.Tensor:
        """Per-expert counts [E] int32 of the last forward."""
        return self._counts
