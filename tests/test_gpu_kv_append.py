"""fp8_qk_norm_rope_append against the formulas in 64 bits.

q is one rounding to 16 bits of a float32 result: within the format's unit
roundoff (2^-8 of the value for bf16's 8-bit significand, 2^-11 for fp16's 11
bits) plus float32 errors, at most
2^-19 of the row's largest value (a norm's sum of 128 terms, products and one
rotation, a handful of roundings of 2^-24 each, amplified by the sum of two
products).  Scales are a float32 maximum and quotient: relative 2^-18.  A
code has to be the E4M3 rounding, under the kernel's own scale, of a value
that close to the exact one; an earlier token's code of dec(c) s_old / s."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import kv_ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -19


def table_of_angles(n, rot):
    f = 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def case(dtype, page, hq, hkv, dim, slots, rot, interleaved, norm, seed=0, num_pages=None,
         magnitude=1.0, stride=None, zero_values=False):
    rng = np.random.default_rng(seed)
    slots = np.asarray(slots)
    T = len(slots)
    num_pages = num_pages or int(max(slots.max(), 0)) // page + 2
    positions = rng.integers(0, 500, T)
    gen = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * dim
    x = torch.randn(T, stride or width, generator=gen) * magnitude
    if zero_values:
        x[:, (hq + hkv) * dim:] = 0
    x = x.to(dtype).to(DEV)[:, :width]
    gamma = [(1 + 0.3 * torch.randn(dim, generator=gen)).to(dtype).to(DEV) if norm else None
             for _ in range(2)]
    cs = torch.from_numpy(table_of_angles(500, rot)).to(DEV) if rot else None
    codes = rng.integers(0, 256, (2, num_pages, hkv, page, dim), dtype=np.uint8)
    codes[(codes & 127) == 127] = 5
    scales = rng.uniform(0.001, 0.02, (2, num_pages, hkv)).astype(np.float32) * magnitude
    cache = fl.KvCache(kv_ref.to_layout(codes[0]).to(DEV), kv_ref.to_layout(codes[1]).to(DEV),
                       torch.from_numpy(scales[0].copy()).to(DEV),
                       torch.from_numpy(scales[1].copy()).to(DEV))
    pos_t = torch.tensor(positions, dtype=torch.int32, device=DEV)
    slot_t = torch.tensor(slots, dtype=torch.int32, device=DEV)
    q = fl.fp8_qk_norm_rope_append(x, cache, pos_t, slot_t, cs, gamma[0], gamma[1], eps=1e-6,
                                   interleaved=interleaved)
    torch.cuda.synchronize()

    x64 = x.double().cpu().numpy().reshape(T, -1, dim)
    cs64 = cs.double().cpu().numpy() if rot else None
    g64 = [g.double().cpu().numpy() if g is not None else None for g in gamma]
    want_q = kv_ref.norm_rotate(x64[:, :hq], g64[0], 1e-6, cs64, positions, interleaved)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tiny = 0.0 if dtype == torch.bfloat16 else 2.0 ** -25
    got_q = q.double().cpu().numpy()
    slack = np.abs(want_q).max(-1, keepdims=True) * F32
    assert np.all(np.abs(got_q - want_q) <= half * 1.0001 * np.abs(want_q) + slack + tiny)

    rows = {"k": kv_ref.norm_rotate(x64[:, hq:hq + hkv], g64[1], 1e-6, cs64, positions,
                                    interleaved), "v": x64[:, hq + hkv:]}
    for i, name in enumerate(("k", "v")):
        got = kv_ref.pages_view(getattr(cache, name))
        got_s = getattr(cache, name + "_scale").double().cpu().numpy()
        want_s = scales[i].astype(np.float64)
        touched = np.zeros((num_pages, page), bool)
        for t, n in kv_ref.runs(slots, page, num_pages):
            pg, o = slots[t] // page, slots[t] % page
            new = np.maximum(np.abs(rows[name][t:t + n]).max((0, 2)) / 448, kv_ref.MIN_SCALE)
            s_old = want_s[pg].copy()
            s = np.maximum(new, s_old) if o else new
            assert np.all(np.abs(got_s[pg] - s) <= s * F32), (name, pg)
            s = got_s[pg]
            want_s[pg] = s
            for h in range(hkv):
                v = rows[name][t:t + n, h] / s[h]
                slack = np.abs(v).max() * F32
                c = kv_ref.TABLE[got[pg, h, o:o + n]]
                assert np.all(kv_ref.nearest_code_ok(v, c, slack)), (name, pg, h)
                before = codes[i, pg, h, :o]
                if o and s[h] > s_old[h]:
                    v = kv_ref.TABLE[before] * s_old[h] / s[h]
                    c = kv_ref.TABLE[got[pg, h, :o]]
                    assert np.all(kv_ref.nearest_code_ok(v, c, np.abs(v) * F32)), (name, pg, h)
                else:
                    assert np.array_equal(got[pg, h, :o], before), (name, pg, h)
            touched[pg, :o + n] = True
        # nothing else moves
        keep = ~touched[:, None, :, None] & np.ones_like(got, bool)
        assert np.array_equal(got[keep], codes[i][keep])
        assert np.array_equal(got_s, want_s)
    return cache, q


def decode_slots(n, page, seed):
    rng = np.random.default_rng(seed)
    pages = rng.permutation(2 * n)[:n]
    return pages * page + rng.integers(0, page, n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,hq,hkv,dim", [(16, 8, 2, 64), (64, 32, 8, 128), (128, 5, 1, 128),
                                             (32, 3, 3, 64)])
@pytest.mark.parametrize("T", [1, 7, 65])
def test_decode(T, page, hq, hkv, dim, dtype):
    case(dtype, page, hq, hkv, dim, decode_slots(T, page, T), dim, False, True, seed=T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page,dim,rot,interleaved,norm",
                         [(16, 64, 32, True, False), (32, 128, 128, False, True),
                          (64, 128, 48, False, False), (128, 128, 64, True, True),
                          (128, 64, 64, False, True), (64, 64, 0, False, True),
                          (16, 128, 16, False, True)])
def test_prompt_chunks(page, dim, rot, interleaved, norm, dtype):
    # requests start inside pages and end inside pages; one has three tokens
    slots = []
    for first, n, p0 in ((5, 200, 3), (0, 128, 40), (page - 1, 3, 60), (page - 2, 77, 70)):
        for i in range(n):
            slots.append((p0 + (first + i) // page) * page + (first + i) % page)
    case(dtype, page, 4, 2, dim, slots, rot, interleaved, norm, seed=page + rot)


def test_many_tokens_use_long_chunks():
    page, slots = 64, []
    for r in range(9):
        for i in range(301):
            slots.append((r * 7 + (i + r) // page) * page + (i + r) % page)
    case(torch.bfloat16, page, 2, 1, 64, slots, 64, False, True)


def test_padding_rows_and_bad_slots_are_left_out():
    page = 16
    slots = [-1, 16, 17, 18, -1, 10 ** 6, 32, -7, 2 ** 31 - 1, 0]
    case(torch.bfloat16, page, 4, 2, 64, slots, 64, False, True, num_pages=4)


@pytest.mark.parametrize("magnitude", [1e-6, 1e4])
def test_magnitudes(magnitude):
    case(torch.bfloat16, 32, 4, 2, 128, decode_slots(20, 32, 3), 128, False, False,
         magnitude=magnitude)


def test_zero_values_get_the_smallest_scale():
    slots = list(range(64, 64 + 40))
    cache, _ = case(torch.bfloat16, 64, 2, 1, 64, slots, 64, False, True, zero_values=True)
    assert cache.v_scale[1, 0].item() == kv_ref.MIN_SCALE


def test_strided_rows():
    case(torch.float16, 16, 4, 2, 64, decode_slots(9, 16, 2), 64, False, True, stride=8 * 64 + 40)


def test_appending_twice_is_the_same():
    cache, q = case(torch.bfloat16, 64, 8, 2, 128, decode_slots(33, 64, 8), 128, False, True)
    x = torch.randn(33, 12 * 128, device=DEV).bfloat16()
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    slot = torch.tensor(decode_slots(33, 64, 9) % (cache.num_pages * 64), dtype=torch.int32,
                        device=DEV)
    first = [fl.fp8_qk_norm_rope_append(x, cache, pos, slot)] + [t.clone() for t in cache]
    again = [fl.fp8_qk_norm_rope_append(x, cache, pos, slot)] + list(cache)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_given_q():
    x = torch.randn(33, 12 * 128, device=DEV).bfloat16()
    pos = torch.arange(33, dtype=torch.int32, device=DEV)
    caches = [fl.kv_cache(4, 16, 2, 128, DEV) for _ in range(2)]
    want = fl.fp8_qk_norm_rope_append(x, caches[0], pos, pos)
    given = torch.empty_like(want)
    assert fl.fp8_qk_norm_rope_append(x, caches[1], pos, pos, q=given) is given
    assert torch.equal(given, want)
    assert all(torch.equal(a, b) for a, b in zip(*caches))


@pytest.mark.parametrize("page", [16, 64, 128])
def test_a_page_filled_token_by_token_against_its_values(page):
    """A scale that grows re-rounds the page's earlier codes.  A token written
    when the block's maxima were a_1 <= .. <= a_i is rounded once, and again
    at every later growth, each time by at most 2^-4 of the value at hand and
    half a subnormal step, 2^-10 of the scale then; a page written at once is
    rounded once."""
    dim = 128
    gen = torch.Generator().manual_seed(page)
    x = torch.randn(page, 4 * dim, generator=gen)
    x[:, 2 * dim:3 * dim] *= torch.linspace(0.5, 2, page)[:, None]  # keys grow in size
    x = x.bfloat16().to(DEV)
    pos = torch.arange(page, dtype=torch.int32, device=DEV)
    slow, once = fl.kv_cache(2, page, 1, dim, DEV), fl.kv_cache(2, page, 1, dim, DEV)
    for t in range(page):
        fl.fp8_qk_norm_rope_append(x[t:t + 1], slow, pos[t:t + 1], pos[t:t + 1] + page)
    fl.fp8_qk_norm_rope_append(x, once, pos, pos + page)
    values = {"k": x[:, 2 * dim:3 * dim], "v": x[:, 3 * dim:]}
    for name in ("k", "v"):
        v = values[name].double().cpu().numpy()
        top = np.maximum.accumulate(np.abs(v).max(1))  # the block's maximum after each token
        decoded = []
        for cache, by_token in ((slow, True), (once, False)):
            s = getattr(cache, name + "_scale")[1, 0].double().item()
            assert abs(s - top[-1] / 448) <= 2.0 ** -22 * s
            got = kv_ref.TABLE[kv_ref.pages_view(getattr(cache, name))[1, 0]] * s
            decoded.append(got)
            for t in range(page):
                scales = np.unique(top[t:]) / 448 if by_token else top[-1:] / 448
                bound, size = 0.0, np.abs(v[t])
                for s_i in scales * 1.0001:
                    step = 2.0 ** -4 * (size + bound) * 1.0001 + 2.0 ** -10 * s_i
                    bound = bound + step
                assert np.all(np.abs(got[t] - v[t]) <= bound), (name, t)
        slow_rms, once_rms = (np.sqrt(((d - v) ** 2).mean()) for d in decoded)
        assert slow_rms >= once_rms * 0.99
