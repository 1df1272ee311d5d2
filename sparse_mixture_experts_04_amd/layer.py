"""Device buffers for one MoE layer configuration, and a forward call.

Plumbing only: torch allocates the caller-owned buffers the C ABI expects
(outputs, routing and dispatch results, workspace), and ``MoELayer.forward``
hands them to ``moe_forward``.  No arithmetic of the layer happens here.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib


def torch_dtype(cfg: _lib.MoeConfig):
    return torch.bfloat16 if cfg.dtype == _lib.MOE_BF16 else torch.float32


@dataclass
class ForwardBuffers:
    out: torch.Tensor             # [T, d]
    topk_ids: torch.Tensor        # [T, k] int32
    topk_w: torch.Tensor          # [T, k] float32
    expert_counts: torch.Tensor   # [E] int32
    expert_offsets: torch.Tensor  # [E+1] int32
    perm: torch.Tensor            # [T*k] int32
    inv_perm: torch.Tensor        # [T*k] int32
    ws: torch.Tensor              # uint8 workspace
    expert_order: Optional[torch.Tensor] = None  # [T, E] uint8 (rerouting forward only)
    op: int = _lib.MOE_OP_FORWARD                # the forward the workspace is sized and laid out for

    @staticmethod
    def allocate(cfg: _lib.MoeConfig, device="cuda", reroute: bool = False, op: Optional[int] = None) -> "ForwardBuffers":
        T, d, E, k = cfg.num_tokens, cfg.hidden_size, cfg.num_experts, cfg.num_experts_per_tok
        i32 = dict(dtype=torch.int32, device=device)
        if op is None:
            op = _lib.MOE_OP_FORWARD_REROUTE if reroute else _lib.MOE_OP_FORWARD
        return ForwardBuffers(
            out=torch.empty((T, d), dtype=torch_dtype(cfg), device=device),
            topk_ids=torch.empty((T, k), **i32),
            topk_w=torch.empty((T, k), dtype=torch.float32, device=device),
            expert_counts=torch.empty(E, **i32),
            expert_offsets=torch.empty(E + 1, **i32),
            perm=torch.empty(T * k, **i32),
            inv_perm=torch.empty(T * k, **i32),
            ws=torch.empty(max(1, _lib.moe_workspace_size(cfg, op)), dtype=torch.uint8, device=device),
            expert_order=torch.empty((T, E), dtype=torch.uint8, device=device) if reroute else None,
            op=op,
        )

    def _dispatch_op(self) -> int:
        return _lib.MOE_OP_DISPATCH_REROUTE if self.expert_order is not None else _lib.MOE_OP_DISPATCH

    def _plain_layout(self) -> None:
        if self.op == _lib.MOE_OP_FORWARD_MX:
            raise ValueError("the workspace of moe_forward_mx holds microscaled codes: it has no such view")

    def scratch_view(self, cfg: _lib.MoeConfig, name: str) -> torch.Tensor:
        """The router ("route") or dispatcher ("dispatch") scratch inside the forward workspace."""
        self._plain_layout()
        a = lambda b: (b + 255) // 256 * 256  # noqa: E731
        r = _lib.moe_workspace_size(cfg, _lib.MOE_OP_ROUTE)
        d = _lib.moe_workspace_size(cfg, self._dispatch_op())
        if name == "route":
            return self.ws[:max(r, 1)]
        return self.ws[a(r):a(r) + max(d, 1)]

    def workspace_view(self, cfg: _lib.MoeConfig, name: str) -> torch.Tensor:
        """Xp, H or Yp as a tensor view into the forward workspace (the layout moe_forward uses:
        router scratch, dispatch scratch, then Xp, H, Yp, each 256-byte aligned)."""
        T, d, F, k = cfg.num_tokens, cfg.hidden_size, cfg.intermediate_size, cfg.num_experts_per_tok
        self._plain_layout()
        es = 2 if cfg.dtype == _lib.MOE_BF16 else 4
        a = lambda b: (b + 255) // 256 * 256  # noqa: E731
        disp = a(_lib.moe_workspace_size(cfg, _lib.MOE_OP_ROUTE)) + a(_lib.moe_workspace_size(cfg, self._dispatch_op()))
        xp = a(T * k * d * es)
        h = a(T * k * F * es)
        start, cols = {"Xp": (disp, d), "H": (disp + xp, F), "Yp": (disp + xp + h, d)}[name]
        n = T * k * cols * es
        return self.ws[start:start + n].view(torch_dtype(cfg)).view(T * k, cols)


class MoELayer:
    """Weights of one layer resident on the GPU, plus its forward buffers.
    ``reroute``: over-capacity pairs move to their token's next-best expert
    with room instead of being dropped (``moe_forward_reroute``)."""

    def __init__(self, cfg: _lib.MoeConfig, Wg: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                 gate_bias: Optional[torch.Tensor] = None, device="cuda", reroute: bool = False):
        self.cfg = cfg
        self.reroute = reroute
        self.Wg, self.W1, self.W2, self.gate_bias = Wg, W1, W2, gate_bias
        self.buf = ForwardBuffers.allocate(cfg, device, reroute)

    def forward(self, X: torch.Tensor, stream=None) -> torch.Tensor:
        b = self.buf
        if self.reroute:
            _lib.moe_forward_reroute(self.cfg, X, self.Wg, self.gate_bias, self.W1, self.W2, b.out, b.topk_ids,
                                     b.topk_w, b.expert_order, b.expert_counts, b.expert_offsets, b.perm, b.inv_perm,
                                     b.ws, stream=stream)
        else:
            _lib.moe_forward(self.cfg, X, self.Wg, self.gate_bias, self.W1, self.W2, b.out, b.topk_ids, b.topk_w,
                             b.expert_counts, b.expert_offsets, b.perm, b.inv_perm, b.ws, stream=stream)
        return b.out


def _mx_kind(x: torch.Tensor) -> int:
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"microscaled arrays are made from bfloat16 or float32, not {x.dtype}")
    return _lib.MOE_BF16 if x.dtype == torch.bfloat16 else _lib.MOE_F32


def mx_quantize(x: torch.Tensor, fmt: int = _lib.MOE_MXFP4, stream=None):
    """x [..., n] (bfloat16 or float32 on the GPU, n a multiple of 32) as microscaled codes (uint8 [..., n/2] for
    MOE_MXFP4, [..., n] for MOE_MXFP8) and scales (uint8 [..., n/32])."""
    if fmt not in (_lib.MOE_MXFP4, _lib.MOE_MXFP8):
        raise ValueError(f"fmt must be MOE_MXFP4 or MOE_MXFP8, not {fmt!r}")
    n = x.shape[-1]
    codes = torch.empty((*x.shape[:-1], n // 2 if fmt == _lib.MOE_MXFP4 else n), dtype=torch.uint8, device=x.device)
    scales = torch.empty((*x.shape[:-1], n // 32), dtype=torch.uint8, device=x.device)
    _lib.moe_mx_quantize(_mx_kind(x), fmt, x.numel() // n if n else 0, n, x, codes, scales, stream=stream)
    return codes, scales


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, fmt: int = _lib.MOE_MXFP4, dtype=torch.bfloat16,
                  stream=None) -> torch.Tensor:
    """The values of microscaled codes and scales, as mx_quantize gives them."""
    if fmt not in (_lib.MOE_MXFP4, _lib.MOE_MXFP8):
        raise ValueError(f"fmt must be MOE_MXFP4 or MOE_MXFP8, not {fmt!r}")
    n = scales.shape[-1] * 32
    expected = (*scales.shape[:-1], n // 2 if fmt == _lib.MOE_MXFP4 else n)
    if tuple(codes.shape) != expected:
        raise ValueError(f"codes of shape {tuple(codes.shape)} do not go with scales of shape {tuple(scales.shape)}: "
                         f"expected {expected}")
    x = torch.empty((*scales.shape[:-1], n), dtype=dtype, device=codes.device)
    _lib.moe_mx_dequantize(_mx_kind(x), fmt, x.numel() // n if n else 0, n, codes, scales, x, stream=stream)
    return x


class MxMoELayer:
    """A residual layer's norm and experts with microscaled expert weights (``moe_forward_mx``): W1 [E, F, d] and
    W2 [E, d, F] are quantised to 4 bits once, here, and not kept; the token rows and the experts' inner values run
    in ``fmt`` (MOE_MXFP8 or MOE_MXFP4).  The weights are quantised on the current stream: a forward on another one
    must wait for it.  ``forward`` returns the experts' combined output and leaves the residual
    stream (X + residual) in ``sum``."""

    def __init__(self, cfg: _lib.MoeConfig, gamma: torch.Tensor, Wg: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                 gate_bias: Optional[torch.Tensor] = None, fmt: int = _lib.MOE_MXFP8, eps: float = 1e-5,
                 device="cuda"):
        d, F, E = cfg.hidden_size, cfg.intermediate_size, cfg.num_experts
        for name, t, shape in (("gamma", gamma, (d,)), ("W1", W1, (E, F, d)), ("W2", W2, (E, d, F))):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if fmt not in (_lib.MOE_MXFP4, _lib.MOE_MXFP8):
            raise ValueError(f"fmt must be MOE_MXFP4 or MOE_MXFP8, not {fmt!r}")
        self.cfg, self.fmt, self.eps = cfg, fmt, eps
        self.gamma, self.Wg, self.gate_bias = gamma, Wg, gate_bias
        self.W1, self.W2 = mx_quantize(W1), mx_quantize(W2)  # (codes, scales)
        self.buf = ForwardBuffers.allocate(cfg, device, op=_lib.MOE_OP_FORWARD_MX)
        self.sum = torch.empty((cfg.num_tokens, cfg.hidden_size), dtype=torch_dtype(cfg), device=device)

    def forward(self, X: torch.Tensor, residual: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        b = self.buf
        _lib.moe_forward_mx(self.cfg, self.fmt, X, residual, self.gamma, self.eps, self.Wg, self.gate_bias, *self.W1,
                            *self.W2, self.sum, b.out, b.topk_ids, b.topk_w, b.expert_counts, b.expert_offsets,
                            b.perm, b.inv_perm, b.ws, stream=stream)
        return b.out
