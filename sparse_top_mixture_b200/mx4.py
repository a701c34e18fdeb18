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

``Mx4SparseMoE`` is that as a layer, called like ``SparseMoE``. Nothing here
takes part in autograd.
"""

from __future__ import annotations

from typing import Dict, NamedTuple, Optional, Sequence, Tuple

import torch

from . import DTYPES, TORCH_DTYPE, Problem, SparseMoE, _launch, _ptr, _req, _written, lib, new_workspace
from .rows import _plan, _req_at

_DTYPE_ID = {TORCH_DTYPE[name]: i for name, i in DTYPES.items()}


class Mx4(NamedTuple):
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
    data, scale = q
    if not isinstance(data, torch.Tensor) or data.dim() < 1:
        raise ValueError(f"{name}.data must be a CUDA tensor of at least one dimension")
    shape = data.shape
    K = 2 * shape[-1]
    lead = shape[:-1] if lead is None else tuple(lead)
    if not (K > 0 and K % 32 == 0 and data.is_cuda and data.dtype == torch.uint8 and data.is_contiguous()
            and shape[:-1] == lead and isinstance(scale, torch.Tensor) and scale.get_device() == data.get_device()
            and scale.dtype == torch.uint8 and scale.is_contiguous()
            and scale.shape == lead + (16 * -(-K // 512),)):  # which of it, in words:
        _req_k(K, name)
        _req(data, f"{name}.data", lead + (K // 2,), torch.uint8)
        _req(scale, f"{name}.scale", lead + (_scale_bytes(K),), torch.uint8)
        raise ValueError(f"{name}.scale is on {scale.device}, expected {data.device}")
    return K


def _new(lead: Tuple[int, ...], K: int, device) -> Mx4:
    # (sizes as arguments of their own: a tuple of them costs torch another 0.7 us)
    return Mx4(torch.empty(*lead, K // 2, dtype=torch.uint8, device=device),
               torch.empty(*lead, _scale_bytes(K), dtype=torch.uint8, device=device))


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
    out = torch.empty(*q.data.shape[:-1], K, dtype=dtype, device=dev)
    _launch(lib().moe_mx4_dequantize, dev, out.numel() // K, K, _DTYPE_ID[dtype], q.data.data_ptr(),
            q.scale.data_ptr(), out.data_ptr())
    return out


def mx4_permute_rows(p: Problem, x, plan: Dict[str, torch.Tensor]) -> Mx4:
    """``mx4_quantize(permute_rows(p, x, plan))``, each token quantised once:
    [T*k, H] in 4 bits, sorted by expert; rows past the last segment are zeros."""
    _req(x, "x", (p.T, p.H), TORCH_DTYPE[p.dtype])
    _req_k(p.H, "x")
    dev = x.device
    pair_pos, offsets = _plan(p, plan, dev.index)
    q = _new((p.T * p.k,), p.H, dev)
    _launch(lib().moe_mx4_permute_rows, dev, p._struct(), x.data_ptr(), pair_pos.data_ptr(), offsets.data_ptr(),
            q.data.data_ptr(), q.scale.data_ptr())
    return q


def _req_product(a: Mx4, w: Mx4, offsets, ws) -> int:
    """K of the product."""
    K = _req_mx4(a, "a")
    if _req_mx4(w, "w") != K:
        raise ValueError(f"a has K {K}, w {w.K}")
    if a.data.dim() != 2 or w.data.dim() != 3:
        raise ValueError("a must be [rows, K] and w [E, N, K]")
    index = a.data.get_device()
    _req_at(offsets, "offsets", (w.data.shape[0] + 1,), torch.int32, index)
    if w.data.get_device() != index:
        raise ValueError(f"w is on {w.device}, expected cuda:{index}")
    if ws is not None and (not isinstance(ws, torch.Tensor) or ws.get_device() != index
                           or ws.numel() * ws.element_size() < 256):
        raise ValueError(f"ws must be a workspace on cuda:{index}")
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
    problems, H and I multiples of 32. For inference: it has no backward pass."""

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
            if _req_mx4(w[name], name, shape[:2]) != shape[2]:
                raise ValueError(f"{name}: K {w[name].K}, expected {shape[2]}")
        _req(w["gate_w"], "gate_w", (p.E, p.H), dt)
        if (p.bias_mode != "none") != (w.get("bias") is not None):
            raise ValueError("a bias goes with bias_mode 'logit' or 'select'")
        if w.get("bias") is not None:
            _req(w["bias"], "bias", (p.E,), torch.float32)
        if (p.shared == "sigmoid_gated") != (w.get("shared_gate") is not None):
            raise ValueError("shared_gate goes with shared 'sigmoid_gated'")
        if w.get("shared_gate") is not None:
            _req(w["shared_gate"], "shared_gate", (p.H,), dt)
        if p.shared != "none":
            _req(w["shared_gate_up"], "shared_gate_up", (2 * p.I_shared, p.H), dt)
            _req(w["shared_down"], "shared_down", (p.H, p.I_shared), dt)
        self.p, self.w = p, w
        self.device = torch.device(device)
        self.ws = new_workspace(p, self.device)
        self.aux = None
        self._counts = torch.zeros(p.E, dtype=torch.int32, device=self.device)
        on = [w["gate_up"].data, w["down"].data] + [w.get(name) for name in ("gate_w", "bias", "shared_gate",
                                                                             "shared_gate_up", "shared_down")]
        if any(t is not None and t.device != self.ws.device for t in on):
            raise ValueError(f"the weights must be on {self.ws.device}")

    def _another(self) -> "Mx4SparseMoE":
        other = super()._another()
        other._counts = torch.zeros_like(self._counts)
        return other

    def forward(self, x, out=None, routing_weights=None, selected_experts=None, events=None):
        """out, routing_weights, selected_experts = moe(x), as SparseMoE's."""
        if events is not None:
            raise ValueError("stage events are recorded by SparseMoE only")
        p, w, ws = self.p, self.w, self.ws
        given = (out, routing_weights, selected_experts)
        out, rw, sel = self._outputs(x, out, routing_weights, selected_experts)
        dev = ws.device
        _req_at(x, "x", (p.T, p.H), torch.bfloat16, dev.index)
        _req_at(out, "out", (p.T, p.H), torch.bfloat16, dev.index)
        _req_at(rw, "routing_weights", (p.T, p.k), torch.float32, dev.index)
        _req_at(sel, "selected_experts", (p.T, p.k), torch.int64, dev.index)
        gate = w.get("shared_gate")
        gamma = None if gate is None else torch.empty(p.T, dtype=torch.float32, device=dev)
        _launch(lib().moe_route, dev, p._struct(), x.data_ptr(), w["gate_w"].data_ptr(), _ptr(w.get("bias")), _ptr(gate),
                rw.data_ptr(), sel.data_ptr(), _ptr(gamma), ws.data_ptr(), ws.numel())
        # the counts stay in one buffer, so that a replayed graph's are the last forward's too
        table = torch.empty(p.E + 1, dtype=torch.int32, device=dev)
        pairs, pos = (torch.empty(p.T * p.k, dtype=torch.int32, device=dev) for _ in range(2))
        _launch(lib().moe_dispatch, dev, p._struct(), sel.data_ptr(), None, self._counts.data_ptr(), table.data_ptr(),
                pairs.data_ptr(), pos.data_ptr(), None, ws.data_ptr(), ws.numel())
        rows = mx4_permute_rows(p, x, {"pair_pos": pos, "offsets": table})
        h = mx4_grouped_gate_up(rows, w["gate_up"], table, quantize=True, ws=ws)
        # The rows in bf16: their rounding moves the result by at most 2e-3 of its norm, the 4 bits by 0.1 to 0.3.
        y = mx4_grouped_matmul(h, w["down"], table, ws=ws)
        shared = None
        if p.shared != "none":
            shared = torch.empty(p.T, p.H, dtype=torch.float32, device=dev)
            _launch(lib().moe_shared_expert, dev, p._struct(), x.data_ptr(), w["shared_gate_up"].data_ptr(),
                    w["shared_down"].data_ptr(), _ptr(gamma), shared.data_ptr(), ws.data_ptr(), ws.numel())
        _launch(lib().moe_unpermute_rows, dev, p._struct(), DTYPES["bf16"], y.data_ptr(), pos.data_ptr(), rw.data_ptr(),
                _ptr(shared), out.data_ptr())
        _written(*given)
        return out, rw, sel

    __call__ = forward

    def forward_counts(self) -> torch.Tensor:
        """Per-expert counts [E] int32 of the last forward (overwritten by the
        next one)."""
        return self._counts
