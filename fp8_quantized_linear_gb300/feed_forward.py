"""The feed-forward half of a Llama-3-8B-shaped layer on its residual stream:
norm, gate/up product with its SiLU gate, down product with the addition back
to the stream.

"Marlin fp8" quotes decode latency for whole layers; `block.DecodeBlock` chains
the layer's four products with stand-ins where the gate and the residual
addition belong, and `paged_block.PagedAttentionBlock` is the layer's attention.
Here the stand-ins are the operations themselves, each inside the call before
or after it:

    w8a8   fp8_add_rmsnorm_quant   stream += attention output; norm; E4M3
                                   codes with a scale per token
           fp8_linear              gate/up, SiLU gate, E4M3 result with a
                                   static scale
           fp8_linear              down, straight from those codes, added to
                                   the stream in place
    w8a16  fp8_add_rmsnorm_quant   the same without codes
           fp8_w8a16_linear        gate/up, SiLU gate, 16-bit result
           fp8_w8a16_linear        down, added to the stream in place

Every call goes through the binding to the library's kernels; this module only
owns the weights and the order of the calls.
"""
from __future__ import annotations

import torch

from . import _binding as b
from .block import HIDDEN, SHAPES

INNER = SHAPES["down"][1]  # gate (and up) channels


class FeedForwardBlock:
    """weights: {"gate_up", "down"} of 16-bit [N, K] on the device (quantized
    per channel at construction; gate_up holds the gate rows, then the up
    rows).  gate_scale: the static E4M3 scale of the gated product ("w8a8"; its
    expected maximum / 448).  biases: optional, by the same names."""

    def __init__(self, weights: dict, kind: str = "w8a8", gamma: torch.Tensor | None = None,
                 gate_scale: float = 16.0 / 448.0, eps: float = 1e-5, biases: dict | None = None):
        if kind not in ("w8a16", "w8a8"):
            raise ValueError(kind)
        dev = weights["gate_up"].device
        self.kind, self.eps = kind, eps
        self.w, self.sw = {}, {}
        self.bias = biases or {}
        for name in ("gate_up", "down"):
            if tuple(weights[name].shape) != SHAPES[name]:
                raise ValueError(f"{name} is {SHAPES[name]}")
            self.w[name], self.sw[name] = b.fp8_quant_per_row(weights[name])
            if kind == "w8a16":
                self.w[name] = b.fp8_pack_w8a16_weights(self.w[name])
        self.gamma = gamma if gamma is not None else torch.ones(HIDDEN, dtype=torch.bfloat16,
                                                                device=dev)
        self.gate_scale = torch.full((1,), gate_scale, dtype=torch.float32, device=dev)

    def norm(self, x: torch.Tensor, stream: torch.Tensor):
        """stream += x, in place; returns its norm: (codes, scales) or (None,
        the 16-bit values)."""
        if self.kind == "w8a8":
            codes, scale, _, _ = b.fp8_add_rmsnorm_quant(x, stream, self.gamma, self.eps,
                                                         "per_token", total=stream)
            return codes, scale
        _, _, _, h = b.fp8_add_rmsnorm_quant(x, stream, self.gamma, self.eps, "norm_only",
                                             total=stream)
        return None, h

    def gate_up(self, codes, h) -> torch.Tensor:
        """SiLU(gate) * up [tokens, INNER]: E4M3 codes, or 16 bits."""
        w, sw, bias = self.w["gate_up"], self.sw["gate_up"], self.bias.get("gate_up")
        if self.kind == "w8a8":
            return b.fp8_linear(codes, w, h, sw, bias=bias, activation="silu", gated=True,
                                out_dtype=torch.uint8, out_scale=self.gate_scale,
                                per_token=True, stable_weights=True)
        return b.fp8_w8a16_linear(h, w, sw, bias=bias, activation="silu", gated=True, packed=True,
                                  stable_weights=True)

    def down(self, inner: torch.Tensor, stream: torch.Tensor) -> torch.Tensor:
        """stream += down product, in place."""
        w, sw, bias = self.w["down"], self.sw["down"], self.bias.get("down")
        if self.kind == "w8a8":
            return b.fp8_linear(inner, w, self.gate_scale, sw, bias=bias, residual=stream, y=stream,
                                per_token=False, stable_weights=True)
        return b.fp8_w8a16_linear(inner, w, sw, bias=bias, residual=stream, y=stream, packed=True,
                                  stable_weights=True)

    def forward(self, x: torch.Tensor, stream: torch.Tensor) -> torch.Tensor:
        """x: the attention's output [tokens, HIDDEN] of gamma's 16-bit type;
        stream: the residual stream, updated in place and returned."""
        return self.down(self.gate_up(*self.norm(x, stream)), stream)
