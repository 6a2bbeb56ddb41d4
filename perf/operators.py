"""Measured cases of the paged FP8 cache: the plan that places a step's tokens
in pages, the per-head norm + rotation + append into the cache, and the
attention that reads it.

Each case is one call of one operator.  `own` selects between the plain form
(elementary torch operations in 32 bits) and the library's entry point.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MIN_SCALE = 2.0 ** -64  # smallest block scale (a block of zeros)


# --------------------------------------------------------------------- cases

def listed():
    def plan(name, **kw):
        return dict(name=name, op="plan", **kw)

    def append(name, **kw):
        return dict(name=name, op="append", **kw)

    def attn(name, **kw):
        return dict(name=name, op="attention", **kw)

    return [
        # one decode step's bookkeeping of a medium batch
        plan("plan_decode_64", requests=64, q_min=1, q_max=1, kv_min=1, kv_max=8192, page=64,
             pattern=1),
        # a busy server's mixed step: prompt chunks among decodes, short pages, an odd batch
        plan("plan_mixed_1021", requests=1021, q_min=1, q_max=47, kv_min=0, kv_max=4096, page=16,
             pattern=2),
        # one sequence decoding: latency
        append("append_decode_1", requests=1, q_min=1, q_max=1, kv_min=777, kv_max=777, page=64,
               q_heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, norm=True,
               dtype="bf16", pattern=3),
        # a decode step of a large batch, 64 query heads
        append("append_decode_256", requests=256, q_min=1, q_max=1, kv_min=1, kv_max=4096, page=64,
               q_heads=64, kv_heads=8, dim=128, rot=128, interleaved=False, norm=True,
               dtype="bf16", pattern=4),
        # ragged prompt chunks, half the head rotated in interleaved pairs, no norm, fp16
        append("append_chunks_f16", requests=9, q_min=1, q_max=301, kv_min=0, kv_max=1000, page=16,
               q_heads=16, kv_heads=2, dim=64, rot=32, interleaved=True, norm=False,
               dtype="f16", pattern=5),
        # prefill of a large token batch
        append("append_prefill_13k", requests=7, q_min=1500, q_max=3000, kv_min=0, kv_max=512,
               page=128, q_heads=32, kv_heads=8, dim=128, rot=128, interleaved=False, norm=True,
               dtype="bf16", pattern=6),
        # one short sequence decoding: latency
        attn("attn_decode_1x129", requests=1, q_min=1, q_max=1, kv_min=128, kv_max=128, page=64,
             q_heads=32, kv_heads=8, dim=128, window=0, dtype="bf16", out="bf16", lse=False,
             pattern=7),
        # an ordinary decode step, ragged lengths
        attn("attn_decode_64x4k", requests=64, q_min=1, q_max=1, kv_min=100, kv_max=8192, page=64,
             q_heads=32, kv_heads=8, dim=128, window=0, dtype="bf16", out="bf16", lse=False,
             pattern=8),
        # few long contexts, 64 query heads, static FP8 output for the o product
        attn("attn_decode_5x100k", requests=5, q_min=1, q_max=1, kv_min=60001, kv_max=131071,
             page=128, q_heads=64, kv_heads=8, dim=128, window=0, dtype="bf16", out="e4m3",
             lse=False, pattern=9),
        # five drafted tokens per sequence, short pages, sliding window, fp16, small heads
        attn("attn_draft_33_window", requests=33, q_min=5, q_max=5, kv_min=0, kv_max=5000, page=16,
             q_heads=16, kv_heads=4, dim=64, window=1024, dtype="f16", out="f16", lse=True,
             pattern=10),
        # ragged prompts without and with cached prefixes
        attn("attn_prefill_ragged", requests=6, q_min=17, q_max=1500, kv_min=0, kv_max=900, page=32,
             q_heads=32, kv_heads=8, dim=128, window=0, dtype="bf16", out="bf16", lse=True,
             pattern=11),
        # one long prompt's last chunk
        attn("attn_prefill_4k_of_20k", requests=1, q_min=4096, q_max=4096, kv_min=16384,
             kv_max=16384, page=64, q_heads=32, kv_heads=8, dim=128, window=0, dtype="bf16",
             out="bf16", lse=False, pattern=12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "append", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    pattern = rng.randrange(1 << 20)
    if op == "plan":
        q_max = rng.choice([1, 1, 5, log(1, 200)])
        return dict(op=op, requests=log(1, 1500 if q_max < 50 else 300), q_min=min(1, q_max),
                    q_max=q_max, kv_min=0, kv_max=log(1, 8192), page=page, pattern=pattern)
    group, kv_heads = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "append":
        if rng.random() < 0.5:
            requests, q_min, q_max = log(1, 256), 1, rng.choice([1, 1, 4])
        else:
            requests, q_min, q_max = log(1, 12), 0, log(2, 1300)
        return dict(op=op, requests=requests, q_min=q_min, q_max=q_max, kv_min=0,
                    kv_max=log(1, 2000), page=page, q_heads=group * kv_heads, kv_heads=kv_heads,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.7, dtype=dtype,
                    pattern=pattern)
    out = rng.choice([dtype, dtype, "e4m3"])
    common = dict(op=op, page=page, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                  window=rng.choice([0, 0, 0, log(16, 2048)]), dtype=dtype, out=out,
                  lse=rng.random() < 0.3, pattern=pattern)
    if rng.random() < 0.65:  # decode, drafts among it
        q = rng.choice([1, 1, 1, 2, 4, 8])
        kv_max = log(1, 60000)
        requests = min(log(1, 128), max(1, 300000 // kv_max))
        return dict(common, requests=requests, q_min=q, q_max=q, kv_min=rng.choice([0, kv_max // 2]),
                    kv_max=kv_max)
    q_max = log(16, 2000)
    requests = min(log(1, 8), max(1, 5000 // q_max))
    return dict(common, requests=requests, q_min=rng.choice([0, 1, q_max]), q_max=q_max, kv_min=0,
                kv_max=log(1, 4000))


def _lengths(case):
    """Host lists: new tokens and cached tokens of each request."""
    rng = random.Random(case["pattern"])
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["requests"])]
    if sum(q) == 0:
        q[0] = 1
    kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(case["requests"])]
    return q, kv


def _pages(n, page):
    return -(-n // page)


# -------------------------------------------------------------------- inputs

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(gen, blocks, width, spare):
    """A block table of `blocks[r]` pages each, drawn without repetition, -1
    beyond; the pages left over as the free list; the number of pages."""
    total = sum(blocks) + spare
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    n = _ints(blocks).long()
    start = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=DEV)
    table = torch.where(col < n[:, None], perm[(start[:, None] + col).clamp(max=total - 1)],
                        perm.new_tensor(-1))
    return table.contiguous(), perm[sum(blocks):].contiguous(), total


def _random_cache(gen, pages, heads, page, dim, first=None, sink=None):
    """Codes [pages, heads, page/8, dim/16, 8, 16] and scales [pages, heads] of
    normal values; the magnitude varies by page and channel; `sink` [heads,
    dim] replaces the token at offset 0 of the pages `first`."""
    codes = torch.empty((pages, heads, page // 8, dim // 16, 8, 16), dtype=torch.uint8, device=DEV)
    scales = torch.empty((pages, heads), dtype=torch.float32, device=DEV)
    channel = torch.exp(0.3 * torch.randn(heads, 1, dim, generator=gen, device=DEV))
    size = torch.exp(0.3 * torch.randn(pages, heads, 1, 1, generator=gen, device=DEV))
    step = max(1, (1 << 27) // (heads * page * dim))
    for p0 in range(0, pages, step):
        p1 = min(pages, p0 + step)
        x = torch.randn(p1 - p0, heads, page, dim, generator=gen, device=DEV)
        x *= channel * size[p0:p1]
        if first is not None:
            here = first[(first >= p0) & (first < p1)].long() - p0
            x[here, :, 0, :] = sink
        s = (x.abs().amax(dim=(2, 3)) / 448.0).clamp(min=MIN_SCALE)
        c = (x / s[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c = c.view(p1 - p0, heads, page // 8, 8, dim // 16, 16).transpose(3, 4)
        codes[p0:p1] = c
        scales[p0:p1] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    q, kv = _lengths(case)
    page, tokens = case["page"], sum(q)
    after = [a + b for a, b in zip(q, kv)]
    s = dict(case=case, op=case["op"], page=page, tokens=tokens)
    if case["op"] == "plan":
        width = max(_pages(n, page) for n in after)
        spare = sum(_pages(n, page) - _pages(k, page) for n, k in zip(after, kv)) + 5
        table, free, _ = _table(gen, [_pages(k, page) for k in kv], width, spare)
        s.update(table=table, free=free, q_lens=_ints(q), kv_lens=_ints(kv))
        return s
    width = max(1, max(_pages(n, page) for n in after))
    table, _, pages = _table(gen, [_pages(n, page) for n in after], width, 3)
    off = [0]
    for n in q:
        off.append(off[-1] + n)
    heads, kv_heads, dim = case["q_heads"], case["kv_heads"], case["dim"]
    dtype = _DTYPES[case["dtype"]]
    if case["op"] == "append":
        qkv = torch.randn(tokens, heads + 2 * kv_heads, dim, generator=gen, device=DEV)
        # keys have a few strong channels, values vary by head
        qkv[:, heads:heads + kv_heads] *= torch.exp(
            0.5 * torch.randn(kv_heads, dim, generator=gen, device=DEV))
        qkv[:, heads + kv_heads:] *= torch.exp(
            0.5 * torch.randn(kv_heads, 1, generator=gen, device=DEV))
        k_codes, k_scale = _random_cache(gen, pages, kv_heads, page, dim)
        v_codes, v_scale = _random_cache(gen, pages, kv_heads, page, dim)
        token = torch.arange(tokens, device=DEV)
        request = torch.searchsorted(_ints(off[1:]).long(), token, right=True)
        pos = _ints(kv).long()[request] + token - _ints(off).long()[request]
        slots = table[request, pos // page].long() * page + pos % page
        rot, longest = case["rot"], max(after) + 1
        freq = 1e4 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * freq
        s.update(qkv=qkv.reshape(tokens, -1).to(dtype), positions=pos.to(torch.int32),
                 slots=slots.to(torch.int32),
                 cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float().contiguous(),
                 k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale,
                 q_gamma=None, k_gamma=None)
        if case["norm"]:
            for name in ("q_gamma", "k_gamma"):
                s[name] = (1 + 0.2 * torch.randn(dim, generator=gen, device=DEV)).to(dtype)
    else:
        # queries share a direction per kv head with the key of the first
        # token, which therefore draws a large part of every row's weight
        u = torch.randn(kv_heads, dim, generator=gen, device=DEV)
        u /= u.norm(dim=1, keepdim=True)
        x = torch.randn(tokens, kv_heads, heads // kv_heads, dim, generator=gen, device=DEV)
        x += 0.7 * math.sqrt(dim) * u[:, None, :]
        first = table[:, 0][_ints(after) > 0]
        k_codes, k_scale = _random_cache(gen, pages, kv_heads, page, dim, first,
                                         0.8 * math.sqrt(dim) * u)
        v_codes, v_scale = _random_cache(gen, pages, kv_heads, page, dim)
        s.update(q=x.reshape(tokens, heads, dim).to(dtype), table=table, q_offsets=_ints(off),
                 kv_lens=_ints(after), q_max=max(q), kv_max=max(after), sm_scale=dim ** -0.5,
                 k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale,
                 out_scale=torch.full((1,), 4.0 / 448.0, device=DEV))
    return s


# ----------------------------------------------------------------- the calls

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import fp8_quantized_linear_gb300 as fl
    if s["op"] == "plan":
        p = fl.fp8_kv_plan(s["q_lens"], s["kv_lens"], s["table"], s["free"], s["tokens"], s["page"])
        return dict(table=s["table"], q_offsets=p.q_offsets, kv_lens=p.kv_lens,
                    positions=p.positions, slots=p.slots, used=p.used)
    c = s["case"]
    cache = fl.KvCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if s["op"] == "append":
        q = fl.fp8_qk_norm_rope_append(s["qkv"], cache, s["positions"], s["slots"],
                                       s["cos_sin"], s["q_gamma"], s["k_gamma"], eps=1e-6,
                                       interleaved=c["interleaved"])
        return dict(q=q, k=s["k_codes"].view(torch.float8_e4m3fn),
                    v=s["v_codes"].view(torch.float8_e4m3fn), k_scale=s["k_scale"],
                    v_scale=s["v_scale"])
    e4m3 = c["out"] == "e4m3"
    out, lse = fl.fp8_kv_attention(s["q"], cache, s["table"], s["q_offsets"], s["kv_lens"],
                                   s["q_max"], sm_scale=s["sm_scale"], window=c["window"],
                                   out_dtype=torch.uint8 if e4m3 else s["q"].dtype,
                                   out_scale=s["out_scale"] if e4m3 else None,
                                   want_lse=c["lse"])
    res = dict(out=out.view(torch.float8_e4m3fn) if e4m3 else out)
    if c["lse"]:
        res["lse"] = lse
    return res


def _plain_plan(s):
    page, T, free = s["page"], s["tokens"], s["free"].long()
    table, F = s["table"], s["free"].numel()
    kv = s["kv_lens"].long()
    off = torch.cumsum(s["q_lens"].long(), 0)
    off = torch.cat([off.new_zeros(1), off]).clamp(max=T)
    total = kv + off[1:] - off[:-1]
    old = (kv + page - 1) // page
    need = (((total + page - 1) // page).clamp(max=table.shape[1]) - old).clamp(min=0)
    base = torch.cumsum(need, 0) - need
    got = torch.minimum((F - base).clamp(min=0), need)
    kv_out = torch.minimum(total, (old + got) * page)
    k = torch.arange(table.shape[1], device=DEV) - old[:, None]
    idx = base[:, None] + k
    fresh = torch.where(idx < F, free[idx.clamp(0, max(F - 1, 0))], -1)
    table.copy_(torch.where((k >= 0) & (k < need[:, None]), fresh.to(torch.int32), table))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(off[1:], t, right=True)
    real = r < kv.numel()
    r = r.clamp(max=kv.numel() - 1)
    pos = kv[r] + t - off[r]
    placed = real & (pos < kv_out[r])
    where = table[r, (pos // page).clamp(max=table.shape[1] - 1)].long()
    used = torch.stack([need.sum().clamp(max=F), (real & ~placed).sum()])
    i32 = torch.int32
    return dict(table=table, q_offsets=off.to(i32), kv_lens=kv_out.to(i32),
                positions=torch.where(real, pos, 0).to(i32),
                slots=torch.where(placed, where * page + pos % page, -1).to(i32),
                used=used.to(i32))


def _rotate(x, cos_sin, positions, interleaved):
    half = cos_sin.shape[1] // 2
    c, s = cos_sin[positions.long()][:, None, :].split(half, dim=2)
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_write(x, codes, scales, slots, entry, lead, page):
    """Quantizes x [T, heads, dim] by page and head into the cache; `entry`
    numbers the page of each token, `lead` are the first tokens."""
    T, heads, dim = x.shape
    amax = torch.zeros((T, heads), device=DEV).scatter_reduce(
        0, entry[:, None].expand(T, heads), x.abs().amax(2), "amax")[:lead.numel()]
    where, offset = slots[lead] // page, (slots[lead] % page)[:, None]
    fresh = (amax / 448.0).clamp(min=MIN_SCALE)
    old = scales[where]
    s = torch.where(offset == 0, fresh, torch.maximum(old, fresh))
    # tokens already in the page, to the new scale
    before = codes[where].view(torch.float8_e4m3fn).float()
    again = (before * old[:, :, None, None, None, None]) / s[:, :, None, None, None, None]
    place = torch.arange(page, device=DEV).view(page // 8, 1, 8, 1)
    again = torch.where(place < offset.view(-1, 1, 1, 1, 1, 1), again, before)
    codes[where] = again.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[where] = s
    new = (x / s[entry][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    o = slots % page
    codes[slots // page, :, o // 8, :, o % 8, :] = new.view(T, heads, dim // 16, 16)


def _plain_append(s):
    c, page = s["case"], s["page"]
    heads, kv_heads, dim = c["q_heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].float().view(s["tokens"], heads + 2 * kv_heads, dim)
    q, k, v = x.split([heads, kv_heads, kv_heads], dim=1)
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(2, keepdim=True) + 1e-6) * s["q_gamma"].float()
        k = k * torch.rsqrt((k * k).mean(2, keepdim=True) + 1e-6) * s["k_gamma"].float()
    q = _rotate(q, s["cos_sin"], s["positions"], c["interleaved"])
    k = _rotate(k, s["cos_sin"], s["positions"], c["interleaved"])
    slots = s["slots"].long()
    first = (slots % page == 0) | (slots != torch.roll(slots, 1) + 1)
    first[0] = True
    entry, lead = torch.cumsum(first, 0) - 1, first.nonzero()[:, 0]
    _plain_write(k, s["k_codes"], s["k_scale"], slots, entry, lead, page)
    _plain_write(v, s["v_codes"], s["v_scale"], slots, entry, lead, page)
    return dict(q=q.to(s["qkv"].dtype), k=s["k_codes"].view(torch.float8_e4m3fn),
                v=s["v_codes"].view(torch.float8_e4m3fn), k_scale=s["k_scale"],
                v_scale=s["v_scale"])


def _gathered(codes, scales, table):
    """[requests, heads, blocks * page, dim] float values of the table's pages."""
    t = table.clamp(min=0).long()
    x = codes[t].view(torch.float8_e4m3fn).float() * scales[t][..., None, None, None, None]
    R, B, H, octs, chunks = x.shape[:5]
    return x.permute(0, 2, 1, 3, 5, 4, 6).reshape(R, H, B * octs * 8, chunks * 16)


def _plain_attention(s):
    c = s["case"]
    q, off, kv = s["q"].float(), s["q_offsets"].long(), s["kv_lens"].long()
    T, heads, dim = q.shape
    kv_heads, n = c["kv_heads"], s["q_max"]
    group, R = heads // kv_heads, kv.numel()
    row = torch.arange(n, device=DEV)
    lens = off[1:] - off[:-1]
    at = (off[:-1, None] + row).clamp(max=T - 1)
    x = q[at].view(R, n, kv_heads, group, dim).permute(0, 2, 1, 3, 4).reshape(
        R, kv_heads, n * group, dim)
    k = _gathered(s["k_codes"], s["k_scale"], s["table"])
    v = _gathered(s["v_codes"], s["v_scale"], s["table"])
    key = torch.arange(k.shape[2], device=DEV)
    last = (kv - lens)[:, None] + row  # the row's own position
    seen = (key <= last[:, :, None]) & (key < kv[:, None, None])
    if c["window"]:
        seen &= key > last[:, :, None] - c["window"]
    seen = seen.repeat_interleave(group, dim=1)[:, None]
    p = (x @ k.transpose(2, 3)) * s["sm_scale"]
    p = p.masked_fill_(~seen, -math.inf)
    m = p.amax(3, keepdim=True)
    p = torch.exp_(p.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)))
    total = p.sum(3, keepdim=True)
    v = torch.where((key < kv[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + m)[..., 0]

    token = torch.arange(T, device=DEV)
    r = torch.searchsorted(off[1:], token, right=True)
    i = token - off[r]
    o = o.view(R, kv_heads, n, group, dim).permute(0, 2, 1, 3, 4)[r, i].reshape(T, heads, dim)
    if c["out"] == "e4m3":
        o = (o / s["out_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    res = dict(out=o if c["out"] == "e4m3" else o.to(s["q"].dtype))
    if c["lse"]:
        res["lse"] = lse.view(R, kv_heads, n, group).permute(0, 2, 1, 3)[r, i].reshape(T, heads)
    return res


_PLAIN = {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}


# ------------------------------------------------------------- floors, truth

def work(case):
    q, kv = _lengths(case)
    page, T, R = case["page"], sum(q), case["requests"]
    after = [a + b for a, b in zip(q, kv)]
    if case["op"] == "plan":
        new = sum(_pages(n, page) - _pages(k, page) for n, k in zip(after, kv))
        return {"bytes": 8 * R + 4 * (R + 1) + 4 * R + 8 * T + 8 * new + 8, "flops": 0}
    heads, kv_heads, dim = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        touched = sum(_pages(n, page) - k // page for n, k in zip(after, kv) if n > k)
        return {"bytes": T * (2 * heads + 2 * kv_heads) * dim * 2 + T * 2 * kv_heads * dim
                + 8 * T + 8 * touched * kv_heads + 4 * case["rot"] * min(T, max(after)),
                "flops": T * (heads + 2 * kv_heads) * dim * 10}
    pairs = keys = 0
    for n, total in zip(q, after):
        w = case["window"] or total
        first = total - n
        # keys seen by the row at position p: min(p + 1, window)
        full = max(0, min(n, w - 1 - first))  # rows that see all p + 1 keys
        pairs += full * first + full * (full + 1) // 2 + (n - full) * w if n else 0
        keys += min(total, w + n - 1) if n else 0
    width = 1 if case["out"] == "e4m3" else 2
    return {"bytes": T * heads * dim * (2 + width) + 2 * keys * kv_heads * dim
            + 8 * kv_heads * _pages(keys, page) + (4 * T * heads if case["lse"] else 0),
            "flops": 4 * dim * heads * pairs}


def _e4m3_64(x):
    """The nearest E4M3 values (ties to even) of doubles, saturated at 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6)
    e = torch.where(a < torch.exp2(e), e - 1, e).clamp(min=-6)
    ulp = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / ulp) * ulp, x)


def _values_64(codes):
    """Doubles of codes, by the format's definition."""
    b = codes.long()
    e, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -x, x)


def _exact_append(s):
    c, page, T = s["case"], s["page"], s["tokens"]
    heads, kv_heads, dim, rot = c["q_heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].double().reshape(T, -1, dim)
    cs = s["cos_sin"].double()[s["positions"].long()]
    if c["interleaved"]:
        one, two = torch.arange(0, rot, 2, device=DEV), torch.arange(1, rot, 2, device=DEV)
    else:
        one = torch.arange(rot // 2, device=DEV)
        two = one + rot // 2

    def turned(y, gamma):
        if gamma is not None:
            y = y / (y.pow(2).sum(2, keepdim=True) / dim + 1e-6).sqrt() * gamma.double()
        z = y.clone()
        co, si = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        z[:, :, one] = y[:, :, one] * co - y[:, :, two] * si
        z[:, :, two] = y[:, :, two] * co + y[:, :, one] * si
        return z

    res = dict(q=turned(x[:, :heads], s["q_gamma"]))
    slots = s["slots"].tolist()
    runs, t = [], 0
    while t < T:
        e = t + 1
        while e < T and slots[e] == slots[e - 1] + 1 and slots[e] % page:
            e += 1
        runs.append((t, e))
        t = e
    for name, y in (("k", turned(x[:, heads:heads + kv_heads], s["k_gamma"])),
                    ("v", x[:, heads + kv_heads:])):
        # page rows as [page, token, head, dim]
        cache = _values_64(s[name + "_codes"]).permute(0, 2, 4, 1, 3, 5)
        cache = cache.reshape(-1, page, kv_heads, dim).contiguous()
        scale = s[name + "_scale"].double().clone()
        for t, e in runs:
            where, o = slots[t] // page, slots[t] % page
            new = (y[t:e].abs().amax(dim=(0, 2)) / 448).clamp(min=MIN_SCALE)
            if o:
                old, new = scale[where], torch.maximum(scale[where], new)
                cache[where, :o] = _e4m3_64(cache[where, :o] * (old / new)[:, None])
            cache[where, o:o + e - t] = _e4m3_64(y[t:e] / new[:, None])
            scale[where] = new
        res[name + "_scale"] = scale
        res[name] = cache.view(-1, page // 8, 8, kv_heads, dim // 16, 16).permute(
            0, 3, 1, 4, 2, 5).contiguous()
    return res


def _exact_attention(s):
    c, page = s["case"], s["page"]
    heads, kv_heads, dim = c["q_heads"], c["kv_heads"], c["dim"]
    group = heads // kv_heads
    T = s["tokens"]
    out = torch.zeros((T, heads, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=DEV)
    off, lens = s["q_offsets"].tolist(), s["kv_lens"].tolist()
    for r, total in enumerate(lens):
        a, b = off[r], off[r + 1]
        if a == b or total == 0:
            continue
        pages = s["table"][r, :_pages(total, page)].long()
        p = total - (b - a) + torch.arange(b - a, device=DEV)
        j = torch.arange(total, device=DEV)
        hidden = j[None, :] > p[:, None]
        if c["window"]:
            hidden |= j[None, :] <= p[:, None] - c["window"]
        for g in range(kv_heads):
            def rows(codes, scale):
                x = _values_64(codes[pages, g]) * scale[pages, g].double().view(-1, 1, 1, 1, 1)
                return x.transpose(2, 3).reshape(-1, dim)[:total]
            k, v = rows(s["k_codes"], s["k_scale"]), rows(s["v_codes"], s["v_scale"])
            for h in range(g * group, (g + 1) * group):
                z = (s["q"][a:b, h].double() @ k.T).mul_(s["sm_scale"])
                z[hidden] = -math.inf
                lse[a:b, h] = torch.logsumexp(z, 1)
                out[a:b, h] = torch.softmax(z, 1).nan_to_num_(0.0) @ v
    if c["out"] == "e4m3":
        out = _e4m3_64(out / s["out_scale"].double())
    return dict(out=out, lse=lse) if c["lse"] else dict(out=out)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
