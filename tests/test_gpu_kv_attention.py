"""fp8_kv_attention against the formulas in 64 bits.

Bounds, with A = sum_j p_j |v_j| of an output: rounding to the output's type
(unit roundoff 2^-8 bf16, 2^-11 fp16 of it); weights rounded to 11 bits (2^-11 A), or to
2^-25 of the row's largest weight w = p * block scale (n keys of at most 448);
float32 sums and exponentials (2^-17 A); the scores' float32 sums (D
roundings of 2^-24 of sum_d |q_d k_d|, twice for numerator and denominator),
which change every weight by that factor.  lse: the same score error plus
2^-18 of itself.  E4M3 outputs are the rounding of a value that close."""
import math

import numpy as np
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import kv_ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def make(dtype, page, hq, hkv, dim, q_lens, kv_lens, seed=0, sink=0.0, spare=3, v_spread=0.5,
         zero_pages=False, stride=None, magnitude=1.0):
    """Queries, a cache whose unused parts hold NaN codes and NaN scales, and
    the 64-bit keys and values of each request."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    blocks = [-(-int(n) // page) for n in kv_lens]
    num_pages = sum(blocks) + spare
    ids = rng.permutation(num_pages)
    width = max(1, max(blocks)) + 1
    table = np.full((len(kv_lens), width), -1)
    codes = np.full((2, num_pages, hkv, page, dim), 0x7F, np.uint8)
    scales = np.full((2, num_pages, hkv), np.nan, np.float32)
    u = rng.standard_normal((hkv, dim))
    u /= np.linalg.norm(u, axis=1, keepdims=True)
    at = 0
    for r, L in enumerate(kv_lens):
        table[r, :blocks[r]] = ids[at:at + blocks[r]]
        at += blocks[r]
        for b in range(blocks[r]):
            n = min(page, int(L) - b * page)
            pg = table[r, b]
            c = rng.integers(0, 256, (2, hkv, n, dim), dtype=np.uint8)
            c[(c & 127) == 127] = 3
            # codes of normal-like magnitude: exponents 4..14
            c[:, :, :, :] = (c & 0x87) | (rng.integers(4, 15, c.shape) << 3).astype(np.uint8)
            c[(c & 127) == 127] = 0x70
            codes[:, pg, :, :n] = c
            scales[0, pg] = np.exp(0.2 * rng.standard_normal(hkv)) / 100 * magnitude
            scales[1, pg] = np.exp(v_spread * rng.standard_normal(hkv)) / 100
            if zero_pages and b % 2:
                codes[1, pg, :, :n] = 0
                scales[1, pg] = kv_ref.MIN_SCALE
            if sink and b == 0:
                k0 = np.clip(u * 200, -240, 240)
                codes[0, pg, :, 0] = torch.from_numpy(k0).to(torch.float8_e4m3fn).view(
                    torch.uint8).numpy()
    T = int(sum(q_lens))
    x = torch.randn(T, stride or hq * dim, generator=gen)
    if sink:
        x[:, :hq * dim] += sink * torch.from_numpy(np.repeat(u, hq // hkv, 0).reshape(-1)).float()
    q = x.to(dtype).to(DEV)[:, :hq * dim].unflatten(1, (hq, dim))
    cache = fl.KvCache(kv_ref.to_layout(codes[0]).to(DEV), kv_ref.to_layout(codes[1]).to(DEV),
                       torch.from_numpy(scales[0]).to(DEV), torch.from_numpy(scales[1]).to(DEV))
    value = torch.from_numpy(kv_ref.TABLE).to(DEV)

    def rows(i):
        out = []
        for r, L in enumerate(kv_lens):
            pg = torch.from_numpy(table[r, :blocks[r]].copy()).to(DEV)
            c = value[torch.from_numpy(codes[i]).to(DEV)[pg].long()]
            s = torch.from_numpy(scales[i]).to(DEV)[pg].double()
            y = (c * s[:, :, None, None]).permute(1, 0, 2, 3).reshape(hkv, -1, dim)
            out.append(y[:, :int(L)].contiguous())
        return out

    off = np.concatenate([[0], np.cumsum(q_lens)])
    return dict(q=q, cache=cache, table=i32(table), off=off, kv=np.asarray(kv_lens), k=rows(0),
                v=rows(1), v_scale=scales[1], n=max(int(x) for x in q_lens))


def run(s, **kw):
    return fl.fp8_kv_attention(s["q"], s["cache"], s["table"], i32(s["off"]), i32(s["kv"]),
                               kw.pop("max_q_len", s["n"]), **kw)


def check(s, window=0, out="same", sm_scale=None, **kw):
    dim = s["q"].shape[2]
    scale = dim ** -0.5 if sm_scale is None else sm_scale
    os = torch.full((1,), 0.02, device=DEV) if out == "e4m3" else None
    got, lse = run(s, window=window, out_dtype=torch.uint8 if out == "e4m3" else None,
                   out_scale=os, want_lse=True, sm_scale=sm_scale, **kw)
    want, want_lse, spread, reach = kv_ref.attention(s["q"].double(), s["k"], s["v"], s["off"],
                                                     s["kv"], scale, window)
    longest = max([int(n) for n in s["kv"]] + [1])
    top = np.nanmax(np.where(np.isnan(s["v_scale"]), 0, s["v_scale"]))
    score = dim * 2.0 ** -24 * reach[:, :, None]
    slack = spread * (2.0 ** -11 + 2.0 ** -17 + 2 * score) + longest * 448 * top * 2.0 ** -25
    if out == "e4m3":
        # half a step of the coded value, and the saturation
        c = kv_ref.TABLE[got.cpu().numpy()]
        ok = kv_ref.nearest_code_ok((want / 0.02).cpu().numpy(), c, (slack / 0.02).cpu().numpy())
        assert ok.all(), (np.argwhere(~ok)[:5], c[~ok][:5], (want / 0.02).cpu().numpy()[~ok][:5])
    else:
        half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -11
        err = (got.double() - want).abs()
        bound = slack + half * (want.abs() + slack) + 2.0 ** -25
        assert bool((err <= bound).all()), (err / bound).max().item()
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    e = (lse.double() - want_lse).abs()[~empty]
    assert bool((e <= (2.0 ** -18 * (1 + want_lse.abs()) + score[:, :, 0])[~empty]).all()), e.max()
    if empty.any():
        assert bool((got[empty] == 0).all())
    return got, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 64), (32, 8, 128), (6, 2, 128), (3, 3, 64)])
def test_decode(page, hq, hkv, dim, dtype):
    kv = [1, 2, 15, 16, 17, 127, 128, 129, 300, 1000]
    check(make(dtype, page, hq, hkv, dim, [1] * len(kv), kv, seed=page + hq))


@pytest.mark.parametrize("group", [1, 2, 5, 8, 16, 32, 48])
def test_query_groups(group):
    check(make(torch.bfloat16, 64, 2 * group, 2, 128, [1, 1, 1], [700, 33, 256], seed=group))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [2, 3, 5, 8, 13])
@pytest.mark.parametrize("dim", [64, 128])
def test_drafted_tokens(n, dim, dtype):
    kv = [n, n + 1, 64 + n, 500, 129]
    check(make(dtype, 16, 8, 2, dim, [n] * 5, kv, seed=n), window=0)
    check(make(dtype, 64, 4, 1, dim, [n, 0, 1, n, 2], kv, seed=n), window=100)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,dim,window", [(16, 64, 0), (64, 128, 0), (128, 128, 200),
                                             (32, 128, 1), (64, 64, 77)])
def test_prompts(page, dim, window, dtype):
    q = [130, 0, 1, 257, 64, 31]
    kv = [130, 40, 900, 600, 64, 1031]
    check(make(dtype, page, 8, 2, dim, q, kv, seed=page + window), window=window)


def test_long_prompt_few_heads():
    check(make(torch.bfloat16, 64, 2, 1, 128, [1500], [3001], seed=3))


@pytest.mark.parametrize("n", [1, 60])
def test_one_long_context(n):
    s = make(torch.bfloat16, 128, 8, 1, 128, [n], [70001], seed=4, sink=8.0)
    check(s)
    check(s, window=33333)


@pytest.mark.parametrize("q_lens", [[1] * 37, [200, 1, 7]])
def test_e4m3_output(q_lens):
    kv = [n + 61 * (i + 1) for i, n in enumerate(q_lens)]
    check(make(torch.bfloat16, 64, 8, 2, 128, q_lens, kv, seed=9), out="e4m3")
    check(make(torch.float16, 32, 4, 4, 64, q_lens, kv, seed=9), out="e4m3", window=40)


@pytest.mark.parametrize("q_lens", [[5, 1, 3], [90, 1, 40]])
def test_rows_that_see_no_key(q_lens):
    # fewer keys than rows: the first rows have nothing to see
    check(make(torch.bfloat16, 16, 4, 2, 64, q_lens, [3, 0, 2], seed=1))


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_first_token_that_draws_the_weight(n, dtype):
    check(make(dtype, 64, 8, 2, 128, [n], [4000], seed=6, sink=14.0))


@pytest.mark.parametrize("n", [1, 100])
def test_block_scales_far_apart(n):
    check(make(torch.bfloat16, 16, 8, 2, 128, [n], [777], seed=7, v_spread=3.0))
    check(make(torch.bfloat16, 16, 8, 2, 128, [n], [777], seed=7, zero_pages=True))


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("magnitude", [1e-3, 30.0])
def test_flat_and_sharp_scores(n, magnitude):
    check(make(torch.bfloat16, 32, 8, 2, 128, [n], [900], seed=8, magnitude=magnitude))


@pytest.mark.parametrize("n", [1, 70])
def test_strided_queries_and_scale(n):
    s = make(torch.bfloat16, 64, 4, 2, 128, [n, n], [500, 129], seed=2, stride=8 * 128)
    assert s["q"].stride(0) == 1024
    check(s, sm_scale=0.2)


@pytest.mark.parametrize("n", [1, 3, 80])
def test_rows_outside_the_requests_are_not_written(n):
    s = make(torch.bfloat16, 64, 4, 2, 128, [n, n], [200, 100], seed=2)
    T = 2 * n
    q = torch.cat([s["q"], torch.full((3, 4, 128), math.nan, device=DEV).bfloat16()])
    out = torch.full((T + 3, 4, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    a, _ = run(s)
    b, _ = run(dict(s, q=q), out=out)
    assert torch.equal(b[:T], a) and bool((b[T:] == 7.0).all())


@pytest.mark.parametrize("n", [1, 4, 90])
def test_same_bits_every_time_and_on_another_stream(n):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n] * 5, [3000, 200, 1, 800, 5000], seed=2)
    first, lse = run(s, want_lse=True)
    for _ in range(3):
        again, l2 = run(s, want_lse=True)
        assert torch.equal(first, again) and torch.equal(lse, l2)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        other, _ = run(s)
    main, _ = run(s)  # may overlap the other stream's call
    side.synchronize()
    assert torch.equal(first, other) and torch.equal(first, main)


@pytest.mark.parametrize("n", [1, 4, 90])
def test_graph_capture_and_replay_with_new_lengths(n):
    s = make(torch.float16, 16, 8, 2, 64, [n] * 3, [1000, 1200, 950], seed=5)
    off, kv = i32(s["off"]), i32(s["kv"])
    call = lambda: fl.fp8_kv_attention(s["q"], s["cache"], s["table"], off, kv, s["n"])  # noqa: E731
    eager, _ = call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = call()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    kv.copy_(i32([n, 700, 333]))
    eager, _ = call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


@pytest.mark.parametrize("n", [1, 70])
def test_offsets_past_32_bits(n):
    # pages beyond 4 GB of codes, slots beyond 2^22
    page, hkv, dim = 128, 8, 128
    s = make(torch.bfloat16, page, 8, hkv, dim, [n, n], [400, 150], seed=3)
    small = s["cache"]
    num = 40000
    shift = num - small.num_pages
    assert num * page * hkv * dim > 2 ** 32
    big = [torch.empty((num,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in small]
    for b, t in zip(big, small):
        b[shift:] = t
    table = torch.where(s["table"] >= 0, s["table"] + shift, s["table"])
    a, _ = run(s)
    b, _ = run(dict(s, cache=fl.KvCache(*big), table=table))
    assert torch.equal(a, b)


@pytest.mark.parametrize("most", [1, 3, 24])
def test_many_requests(most):
    # more requests than a block has threads, empty ones among them
    rng = np.random.default_rng(most)
    q = rng.integers(0, most + 1, 700)
    kv = q + rng.integers(0, 90, 700) * (rng.random(700) < 0.7)
    q[::7], kv[::7] = 0, 0
    q[3], kv[3] = most, 2000
    check(make(torch.bfloat16, 16, 4, 2, 64, q, kv, seed=most))


def test_runs_of_small_prompts_after_full_row_tiles():
    # a block then walks more pieces without rows for its second half (over
    # 128) than the ring that hands out the pieces has slots
    q = ([150] + [20] * 29) * 5
    kv = [n + 40 * (i % 3) for i, n in enumerate(q)]
    check(make(torch.bfloat16, 32, 32, 16, 64, q, kv, seed=4))


@pytest.mark.parametrize("n", [1, 30])
def test_a_larger_bound_of_new_tokens_gives_the_same_rows(n):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [700, 90], seed=2)
    for bound in (n, n + 1, 5 * n + 40, 10 ** 6):
        check(s, max_q_len=bound)


def test_no_rows():
    s = make(torch.bfloat16, 64, 4, 2, 128, [1], [200], seed=2)
    out, lse = fl.fp8_kv_attention(s["q"][:0], s["cache"], s["table"], i32([0, 0]), i32([200]), 1,
                                   want_lse=True)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    fresh = torch.full((1, 4, 128), 5.0, device=DEV, dtype=torch.bfloat16)
    out, _ = fl.fp8_kv_attention(s["q"], s["cache"], s["table"], i32([0, 0]), i32([200]), 1,
                                 out=fresh)
    assert bool((out == 5.0).all())


def rising(s, page):
    """Every tile of 128 keys scores higher than the one before: the running
    reference moves in each, a piece's last among them."""
    for r, n in enumerate(s["kv"]):
        for b in range(-(-int(n) // page)):
            pg = int(s["table"][r, b])
            old = s["cache"].k_scale[pg].clone()
            s["cache"].k_scale[pg] *= 1 + b * page // 128
            grown = (s["cache"].k_scale[pg].double() / old.double())[:, None, None]
            s["k"][r][:, b * page:(b + 1) * page] *= grown
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 3, 7, 100])
def test_references_that_move_in_every_tile(n, dtype):
    kv = [1500, 900, 129, 257, 640, 2000]
    s = rising(make(dtype, 64, 8, 2, 128, [n] * len(kv), kv, seed=12 + n), 64)
    first, lse = check(s)
    for _ in range(100):
        again, l2 = run(s, want_lse=True)
        assert torch.equal(first, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("n", [1, 3, 7, 60])
def test_a_scale_of_zero_is_a_block_of_zeros(n):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [1000, 300], seed=33)
    for r, L in enumerate(s["kv"]):
        for b in range(0, -(-int(L) // 64), 2):
            page = int(s["table"][r, b])
            s["cache"].k_scale[page, 0] = s["cache"].v_scale[page] = 0.0
            s["k"][r][0, b * 64:(b + 1) * 64] = 0
            s["v"][r][:, b * 64:(b + 1) * 64] = 0
    check(s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 3, 7, 60])
def test_one_query_channel_a_thousand_times_the_others(n, dtype):
    # The parts of a query stop at E4M3's step of 2^-9 under a row's largest
    # element of 2^7 at least: up to 32 rows per kv head the last part is
    # scaled by 16 (bf16) or 256 (fp16), so an element is within 2^-10 / 2^7 /
    # 16 or / 256 of the largest, above within 2^-17.  Keys are 0 in the strong
    # channel, so that the scores are those of the weak ones.
    s = make(dtype, 64, 8, 2, 128, [n, n], [900, 300], seed=40)
    s["q"][:, :, 3] = 1000.0
    s["cache"].k[:, :, :, 0, :, 3] = 0
    for k in s["k"]:
        k[:, :, 3] = 0
    got, lse = run(s, want_lse=True)
    q = s["q"].double()
    want, want_lse, spread, reach = kv_ref.attention(q, s["k"], s["v"], s["off"], s["kv"],
                                                     128 ** -0.5, 0)
    bits = 17 if 4 * n > 32 else (21 if dtype == torch.bfloat16 else 25)
    keys = max(k.abs().sum(2).max().item() for k in s["k"])
    score = (2.0 ** -bits * 1000 * keys * 128 ** -0.5 + 128 * 2.0 ** -24 * reach)[:, :, None]
    top = np.nanmax(np.where(np.isnan(s["v_scale"]), 0, s["v_scale"]))
    slack = spread * (2.0 ** -11 + 2.0 ** -17 + torch.expm1(2 * score)) + 900 * 448 * top * 2.0 ** -25
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    err = (got.double() - want).abs()
    assert bool((err <= slack + half * (want.abs() + slack) + 2.0 ** -25).all())
    assert bool(((lse.double() - want_lse).abs() <=
                 2.0 ** -18 * (1 + want_lse.abs()) + score[:, :, 0]).all())


@pytest.mark.parametrize("n", [1, 90])
def test_given_outputs(n):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [700, 90], seed=41)
    want, want_lse = run(s, want_lse=True)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    got, got_lse = run(s, out=out, lse=lse)
    assert got is out and got_lse is lse
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    scale = torch.full((1,), 0.02, device=DEV)
    codes, _ = run(s, out_dtype=torch.uint8, out_scale=scale)
    given = torch.empty(codes.shape, dtype=torch.float8_e4m3fn, device=DEV)
    got, none = run(s, out=given, out_dtype=torch.float8_e4m3fn, out_scale=scale)
    assert none is None and got is given and torch.equal(given.view(torch.uint8), codes)


def test_codes_of_few_rows_take_weights_of_16_bits():
    # Two keys of like weight, so that a weight's rounding shows in the output
    # (2^-16 of it, or 2^-29 of the row's largest), and small scores, whose own
    # float32 error is less.  16.8 million codes: few are near enough a border.
    dim, hq, hkv, n = 64, 32, 8, 512
    scale = torch.full((1,), 0.02, device=DEV)
    for seed in range(16):
        s = make(torch.bfloat16, 16, hq, hkv, dim, [1] * n, [2] * n, seed=seed, magnitude=0.05)
        got, _ = run(s, out_dtype=torch.uint8, out_scale=scale)
        k, v = (torch.stack(s[x]).repeat_interleave(hq // hkv, 1) for x in ("k", "v"))
        q = s["q"].double()
        p = torch.softmax(torch.einsum("rhd,rhjd->rhj", q, k) * dim ** -0.5, 2)
        want, spread = (torch.einsum("rhj,rhjd->rhd", p, x) for x in (v, v.abs()))
        reach = torch.einsum("rhd,rhjd->rhj", q.abs(), k.abs()).amax(2) * dim ** -0.5
        score = (dim * 2.0 ** -24 * reach)[:, :, None]
        assert score.max().item() < 2.0 ** -17
        top = np.nanmax(np.where(np.isnan(s["v_scale"]), 0, s["v_scale"]))
        slack = spread * (2.0 ** -16 + 2.0 ** -17 + 2 * score) + 2 * 448 * top * 2.0 ** -29
        unit = scale.double()
        ok = kv_ref.nearest_code_ok((want / unit).cpu().numpy(), kv_ref.TABLE[got.cpu().numpy()],
                                    (slack / unit).cpu().numpy())
        assert ok.all(), (seed, (~ok).sum())


@pytest.mark.parametrize("n", [10, 100])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 6, 2 ** 40, 64 * 4])
def test_a_window_wider_than_every_context(n, window):
    # more rows than keys, so that the first positions are negative
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [3, 190], seed=60 + n)
    want, want_lse = run(s, want_lse=True)
    got, lse = run(s, want_lse=True, window=window)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
