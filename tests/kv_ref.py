"""Plain 64-bit implementation of the paged FP8 cache operators, for the
tests: tables of codes, loops over requests, pages and heads, no shared code
with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

MIN_SCALE = 2.0 ** -64


def e4m3_table() -> np.ndarray:
    """Values of the 256 codes by the format's definition (NaN for 0x7f, 0xff)."""
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return t


TABLE = e4m3_table()


def ulp(x):
    """Spacing of E4M3 values around |x| (its binade, 2^-9 at least)."""
    a = np.clip(np.abs(x), 2.0 ** -6, 448.0)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def nearest_code_ok(value, code_value, slack):
    """Whether code_value is the saturated E4M3 rounding of a value within
    `slack` of `value`."""
    v = np.clip(value, -448.0, 448.0)
    return np.abs(code_value - v) <= 0.5 * np.maximum(ulp(v), ulp(code_value)) + slack


def pages_view(codes: torch.Tensor) -> np.ndarray:
    """Codes as uint8 [num_pages, kv_heads, page_size, head_dim]."""
    p, h, octs, chunks = codes.shape[:4]
    return codes.permute(0, 1, 2, 4, 3, 5).reshape(p, h, octs * 8, chunks * 16).cpu().numpy()


def to_layout(rows: np.ndarray) -> torch.Tensor:
    """uint8 [num_pages, kv_heads, page_size, head_dim] in the cache's order."""
    p, h, page, dim = rows.shape
    t = torch.from_numpy(np.ascontiguousarray(rows))
    return t.view(p, h, page // 8, 8, dim // 16, 16).transpose(3, 4).contiguous()


def plan(q_lens, kv_lens, table, free, tokens, page):
    R, W = table.shape
    table = table.copy()
    off, kv_out, pos, slots = [0], [], [0] * tokens, [-1] * tokens
    taken = lost = asked = 0
    for r in range(R):
        q, kv = max(int(q_lens[r]), 0), max(int(kv_lens[r]), 0)
        q = min(q, tokens - off[-1])
        old = -(-kv // page)
        need = max(min(-(-(kv + q) // page), W) - old, 0)
        got = 0
        for k in range(need):
            ok = asked < len(free)
            table[r, old + k] = free[asked] if ok else -1
            asked += 1
            got += ok
        taken += got
        kv_out.append(min(kv + q, (old + got) * page))
        for i in range(q):
            t, x = off[-1] + i, kv + i
            pos[t] = x
            if x < kv_out[-1]:
                slots[t] = int(table[r, x // page]) * page + x % page
            else:
                lost += 1
        off.append(off[-1] + q)
    return dict(table=table, q_offsets=np.array(off), kv_lens=np.array(kv_out),
                positions=np.array(pos), slots=np.array(slots), used=np.array([taken, lost]))


def norm_rotate(x, gamma, eps, cos_sin, positions, interleaved):
    """x [T, H, D] float64."""
    x = x.copy()
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    if cos_sin is None or cos_sin.shape[1] == 0:
        return x
    rot = cos_sin.shape[1]
    half = rot // 2
    row = cos_sin[np.clip(positions, 0, cos_sin.shape[0] - 1)]
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = row[:, None, i], row[:, None, half + i]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def runs(slots, page, num_pages):
    """(first token, count) of the tokens that share a page."""
    out, t, n = [], 0, len(slots)
    while t < n:
        if not 0 <= slots[t] < num_pages * page:
            t += 1
            continue
        e = t + 1
        while e < n and slots[e] == slots[e - 1] + 1 and slots[e] % page:
            e += 1
        out.append((t, e - t))
        t = e
    return out


def attention(q, k, v, q_offsets, kv_lens, sm_scale, window):
    """q [T, H, D] float64 on any device; k, v: lists per request of [Hkv, L,
    D] float64.  Returns out, lse, and per output the sum of weight times
    |value|, the largest weight per row and the largest sum of |q_d k_d|."""
    T, H, D = q.shape
    out = torch.zeros_like(q)
    spread = torch.zeros_like(q)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros((T, H), dtype=torch.float64, device=q.device)
    for r in range(len(kv_lens)):
        a, b, L = int(q_offsets[r]), int(q_offsets[r + 1]), int(kv_lens[r])
        if a == b or L == 0:
            continue
        group = H // k[r].shape[0]
        pos = L - (b - a) + torch.arange(b - a, device=q.device)
        j = torch.arange(L, device=q.device)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(H):
            kk, vv = k[r][h // group], v[r][h // group]
            s = (q[a:b, h] @ kk.T) * sm_scale
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            some = seen.any(1)
            lse[a:b, h] = torch.logsumexp(s, 1)
            p = torch.where(some[:, None], torch.softmax(s, 1), torch.zeros_like(s)).nan_to_num(0.0)
            out[a:b, h] = p @ vv
            spread[a:b, h] = p @ vv.abs()
            reach[a:b, h] = (torch.where(seen, q[a:b, h].abs() @ kk.abs().T,
                                         torch.zeros_like(s)) * sm_scale).amax(1)
    return out, lse, spread, reach
