"""A Llama-3-8B-shaped attention layer over a paged FP8 cache: the part of a
decode layer between its norm and its o product, for steps that mix prompt
chunks, drafted tokens and single decoded tokens.

"Marlin fp8" quotes decode latency with a static cache; `block.DecodeBlock`
chains the layer's four products with stand-ins between them.  Here the
stand-in between q/k/v and o is the attention itself:

    plan       fp8_kv_plan              pages and slots of the step's tokens
                                        (once per step, for every layer)
    qkv        fp8_rmsnorm_quant,       norm and dynamic E4M3 quantization,
               fp8_scaled_mm            then the fused q/k/v product
    append     fp8_qk_norm_rope_append  per-head norms, rotation, keys and
                                        values quantized into the cache
    attention  fp8_kv_attention         E4M3 output with a static scale
    o          fp8_scaled_mm            straight from those codes

Every call goes through the binding to the library's kernels; this module only
owns the buffers and the order of the calls.
"""
from __future__ import annotations

import torch

from . import _binding as b
from .block import HIDDEN, SHAPES

HEADS, KV_HEADS, HEAD_DIM = 32, 8, 128


def rotation_table(max_positions: int, rot: int = HEAD_DIM, base: float = 5e5,
                   device=None) -> torch.Tensor:
    """float32 [max_positions, rot]: cosines, then sines, of position * base^(-2i / rot)."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


class PagedAttentionBlock:
    """Weights, cache and free pages of one layer.  weights: {"qkv", "o"} of
    bf16 [N, K] on the device (quantized per channel at construction);
    attention_scale: the static E4M3 scale of the attention's output (its
    expected maximum / 448)."""

    def __init__(self, weights: dict, num_pages: int, requests: int, max_tokens: int,
                 page_size: int = 64, gamma: torch.Tensor | None = None,
                 q_gamma: torch.Tensor | None = None, k_gamma: torch.Tensor | None = None,
                 attention_scale: float = 4.0 / 448.0, eps: float = 1e-5):
        dev = weights["qkv"].device
        self.device, self.page_size, self.eps = dev, page_size, eps
        self.w, self.sw = {}, {}
        for name in ("qkv", "o"):
            assert tuple(weights[name].shape) == SHAPES[name]
            self.w[name], self.sw[name] = b.fp8_quant_per_row(weights[name])
        self.gamma = gamma if gamma is not None else torch.ones(HIDDEN, dtype=torch.bfloat16,
                                                                device=dev)
        self.q_gamma, self.k_gamma = q_gamma, k_gamma
        self.cache = b.kv_cache(num_pages, page_size, KV_HEADS, HEAD_DIM, dev)
        self.width = -(-max_tokens // page_size)
        self.table = torch.full((requests, self.width), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(num_pages, dtype=torch.int32, device=dev)
        self.kv_lens = torch.zeros(requests, dtype=torch.int32, device=dev)
        # (a request's last page can hold tokens past max_tokens)
        self.cos_sin = rotation_table(self.width * page_size, device=dev)
        self.out_scale = torch.full((1,), attention_scale, dtype=torch.float32, device=dev)
        self.ws = b.workspace(dev)

    def plan(self, q_lens: torch.Tensor, tokens: int) -> b.KvPlan:
        """Places the step's tokens (q_lens: int32 [requests] on the device,
        `tokens` rows in all) in pages."""
        return b.fp8_kv_plan(q_lens, self.kv_lens, self.table, self.free, tokens, self.page_size)

    def forward(self, x: torch.Tensor, plan: b.KvPlan, max_q_len: int) -> torch.Tensor:
        """The layer's attention output for x [tokens, HIDDEN] (bf16), rows in
        the plan's order; max_q_len: the most new tokens of a request.  The
        plan has placed every token (its used[1] is 0)."""
        codes, scale, _ = b.fp8_rmsnorm_quant(x, self.gamma, self.eps, ws=self.ws)
        qkv = b.fp8_scaled_mm(codes, self.w["qkv"], scale, self.sw["qkv"], ws=self.ws,
                              stable_weights=True)
        q = b.fp8_qk_norm_rope_append(qkv, self.cache, plan.positions, plan.slots, self.cos_sin,
                                      self.q_gamma, self.k_gamma, eps=self.eps)
        att, _ = b.fp8_kv_attention(q, self.cache, self.table, plan.q_offsets, plan.kv_lens,
                                    max_q_len, out_dtype=torch.uint8, out_scale=self.out_scale)
        return b.fp8_scaled_mm(att.view(x.shape[0], HIDDEN), self.w["o"], self.out_scale,
                               self.sw["o"], ws=self.ws, stable_weights=True)

    def commit(self, plan: b.KvPlan, pages_taken: int) -> None:
        """Ends the step: the plan's lengths become the cache's, and the pages
        it took (plan.used[0], which a scheduler that counts pages on the host
        knows without reading it back) leave the free list."""
        self.kv_lens.copy_(plan.kv_lens)
        self.free = self.free[pages_taken:].contiguous()

    def release(self, request: int) -> None:
        """Ends a request: its pages return to the free list, and another
        request can take its place.  (A page starts anew, codes and scales,
        when a token is written at its offset 0.)"""
        pages = -(-int(self.kv_lens[request]) // self.page_size)
        self.free = torch.cat([self.free, self.table[request, :pages]])
        self.table[request] = -1
        self.kv_lens[request] = 0

    def step(self, x: torch.Tensor, q_lens: list[int]) -> torch.Tensor:
        """plan, forward and commit of one step, with the lengths on the host.
        Raises before anything is computed when a token finds no page (too few
        free pages, or a request past its table's); the cache, the lengths and
        the free pages are then as before, and a later step may be tried."""
        if sum(q_lens) > x.shape[0]:
            raise ValueError(f"{sum(q_lens)} new tokens, but x has {x.shape[0]} rows")
        lens = torch.tensor(q_lens, dtype=torch.int32, device=self.device)
        plan = self.plan(lens, x.shape[0])
        taken, lost = plan.used.tolist()
        if lost:
            raise RuntimeError(f"{lost} of the step's {x.shape[0]} tokens found no page")
        y = self.forward(x, plan, max(q_lens))
        self.commit(plan, taken)
        return y
