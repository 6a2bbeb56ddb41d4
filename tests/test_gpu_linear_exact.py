"""The linear layers on numbers whose sums float32 holds exactly, through every
kernel and every way that it divides the work, so that results are equal and
not only near; W8A16 tokens against the E4M3 parts that the definition gives
them; the same bits on every call."""
import itertools

import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import linear_ref as ref
from gpu_util import DEV, assert_status_ok
from test_gpu_linear import ACTS, BF, HF, U8, check_linear, exact_operands, normal_codes, operands

pytestmark = pytest.mark.gpu


# tokens and weight rows past a tile's end, ragged K, tail tiles (20480), K split
# over clusters of two pairs of SMs (24 tiles) and of four, and over CTAs
@pytest.mark.parametrize("kernel,M,N,K", [
    ("stream", 3, 1056, 656), ("stream", 8, 96, 4112), ("stream", 16, 160, 1040), ("stream", 37, 64, 272),
    ("swapped", 1, 4096, 4096), ("swapped", 17, 1056, 656), ("swapped", 40, 32, 4112),
    ("swapped", 100, 288, 14336), ("swapped", 300, 2080, 400), ("swapped", 1000, 96, 144),
    ("tiled", 1, 32, 16), ("tiled", 130, 1056, 656), ("tiled", 300, 512, 4096), ("tiled", 257, 544, 4112),
    ("tiled", 513, 2048, 2048), ("tiled", 520, 1888, 1040), ("tiled", 700, 20480, 144),
    ("tiled", 1021, 9728, 272), ("tiled", 4097, 512, 528)])
@pytest.mark.parametrize("gated", [False, True])
def test_whole_numbers(kernel, M, N, K, gated):
    """Sums of whole numbers up to 9 K, times powers of two by row and by
    column, plus quarters: exact before the output's rounding (with a gate the
    product of the two is rounded once, to float32)."""
    gen, a, w = exact_operands(M, M, N, K)
    sa = torch.exp2(torch.randint(-3, 3, (M,), generator=gen, device=DEV).float())
    sw = torch.exp2(torch.randint(-3, 3, (N,), generator=gen, device=DEV).float())
    b = torch.randint(-8, 8, (N,), generator=gen, device=DEV).to(BF) / 4
    width = N // 2 if gated else N
    r = None if gated else torch.randint(-64, 64, (M, width), generator=gen, device=DEV) / 8
    z = (ref.e4m3_values(a) @ ref.e4m3_values(w).T) * sa.double()[:, None] * sw.double() + b.double()
    t = (z[:, :width].clamp(min=0) * z[:, width:]).float().double() if gated else z + r.double()
    for out in (HF, BF):
        for stable in (False, True):
            y = fl.fp8_linear(a, w, sa, sw, bias=b, residual=None if gated else r.to(out), out_dtype=out,
                              per_token=True, gated=gated, activation="relu" if gated else None,
                              kernel=kernel, stable_weights=stable)
            assert torch.equal(y, t.to(out))
    if not gated:
        t = t - r.double()
    os = torch.full((1,), 8.0, device=DEV)
    y = fl.fp8_linear(a, w, sa, sw, bias=b, out_dtype=U8, out_scale=os, per_token=True, gated=gated,
                      activation="relu" if gated else None, kernel=kernel)
    assert torch.equal(ref.e4m3_values(y), ref.e4m3_round(t / 8))
    assert_status_ok()


@pytest.mark.parametrize("M", [140, 300])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_every_epilogue_on_pairs(M, act, gated):
    """Every epilogue through the 256 x 256 tiles, K whole and split."""
    n = 0
    for out, bias, residual, per_token, per_channel in itertools.product(
            (BF, HF, U8), (None, BF, HF, torch.float32), (False, True), (False, True), (False, True)):
        if residual and out is U8:
            continue
        n += 1
        check_linear(n, M, 544, 160 if n % 3 else 1168, out, bias, act, gated, residual, per_token,
                     per_channel, kernel="tiled", stable_weights=n % 2 == 0)


# ------------------------------------------------------------------ W8A16

def held(x):
    """The value that a sum of E4M3 parts holds for a 16-bit token: the row's
    largest magnitude brought to [2^7, 2^8) by 2^e (e within +-126), two parts
    of bf16, three of fp16, each 16 times finer than the one before."""
    v = x.double()
    amax = v.abs().amax(1, keepdim=True)
    # (frexp: exact, where a logarithm may fall below a power of two; amax = m 2^k, m in [1/2, 1))
    e = torch.where(amax > 0, 8.0 - torch.frexp(amax).exponent, 0.0).clamp(-126, 126)
    f = v * torch.exp2(e)
    total = torch.zeros_like(f)
    for q in range(2 if x.dtype is BF else 3):
        p = ref.e4m3_round(f)
        total += p * 16.0 ** -q
        f = (f - p) * 16
    return total * torch.exp2(-e)


def w8a16(x, w, sw, **kw):
    packed = kw.get("packed", False)
    return fl.fp8_w8a16_linear(x, fl.fp8_pack_w8a16_weights(w) if packed else w, sw, **kw)


# (bf16: whole numbers of 8 bits, two parts; fp16: of 11 bits, three)
@pytest.mark.parametrize("dtype,most,K", [(BF, 255, 4096), (BF, 255, 656), (BF, 255, 14336), (HF, 2047, 2048),
                                          (HF, 2047, 272), (HF, 2047, 1040)])
@pytest.mark.parametrize("M", [1, 8, 9, 47, 48, 49, 64, 65, 130])
@pytest.mark.parametrize("packed", [False, True])
def test_w8a16_whole_numbers(dtype, most, K, M, packed):
    """Tokens that fill their type's significand, whole-number weights (zeros
    but for a few, so that sums stay below 2^24): exact before the rounding."""
    N = 160
    gen, _, w = exact_operands(M + K, 1, N, K)
    w[torch.rand(N, K, generator=gen, device=DEV) < 1 - 1024 / max(K, 1024)] = 0
    w[:, 40:] = torch.where(torch.arange(K - 40, device=DEV) % 2 == 0, w[:, 40:], 0)
    x = torch.randint(-most, most + 1, (M, K), generator=gen, device=DEV).to(dtype)
    x[:, 3] = most  # (every row's largest)
    sw = torch.exp2(torch.randint(-12, -6, (N,), generator=gen, device=DEV).float())
    z = x.double() @ ref.e4m3_values(w).T
    assert (x.double().abs() @ ref.e4m3_values(w).abs().T).max() < 2 ** 24
    assert torch.equal(held(x), x.double())
    t = z * sw.double()
    for kernel in ("stream", "swapped"):
        y = w8a16(x, w, sw, activation="relu", packed=packed, kernel=kernel)
        assert torch.equal(y, t.clamp(min=0).to(dtype)), kernel
        g = w8a16(x, w, sw, activation="relu", gated=True, packed=packed, kernel=kernel)
        gate = t[:, : N // 2].clamp(min=0) * t[:, N // 2:]
        assert torch.equal(g, gate.float().to(dtype)), kernel
    assert_status_ok()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("ratio", [2.0 ** 6, 2.0 ** 10, 1e4])
@pytest.mark.parametrize("M", [4, 12, 60])
def test_w8a16_rows_with_an_outlier(dtype, ratio, M):
    """One value `ratio` times the rest, met by weights that are zero: what is
    left of the others is what the parts hold, and the parts hold them to 2^-21
    (bf16) or 2^-25 (fp16) of the outlier.  The streaming kernel takes the
    values whole."""
    N, K = 96, 64
    gen = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, K, generator=gen, device=DEV)
    x[:, 11] = ratio * 4
    x = x.to(dtype)
    w = normal_codes(gen, N, K)
    w[:, 11] = 0
    sw = torch.full((N,), 2.0 ** -9, device=DEV)
    v = ref.e4m3_values(w)
    assert ((held(x) - x.double()).abs() <= ref.parts_error(x)).all()
    for act in (None, "silu"):
        y = w8a16(x, w, sw, activation=act, residual=torch.zeros(M, N, dtype=dtype, device=DEV),
                  kernel="swapped")
        ref.check16(y, *ref.linear(held(x), v, sw.double().view(1, -1), activation=act))
        ref.check16(y, *ref.linear(x.double(), v, sw.double().view(1, -1), activation=act,
                                   x_error=ref.parts_error(x)))
        y = w8a16(x, w, sw, activation=act, kernel="stream")
        ref.check16(y, *ref.linear(x.double(), v, sw.double().view(1, -1), activation=act))
    assert_status_ok()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("packed", [False, True])
def test_w8a16_every_value_alone(dtype, packed):
    """Rows of two values, the largest against zero weights, the other against
    one: the result is what the parts hold of it, the value itself down to 2^-13
    of the largest."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    M, K = 4000, 32
    at, size = torch.arange(M, device=DEV) % (K - 1) + 1, torch.exp2(-24.0 * torch.arange(M, device=DEV) / M)
    x = torch.zeros(M, K, dtype=dtype, device=DEV)
    x[:, 0] = (1 + 30 * torch.rand(M, generator=gen, device=DEV)).to(dtype)
    value = (x[:, 0].float() * size * (0.5 + 0.5 * torch.rand(M, generator=gen, device=DEV))).to(dtype)
    x[torch.arange(M, device=DEV), at] = value
    w = torch.full((32, K), 0x38, dtype=U8, device=DEV)
    w[:, 0] = 0
    y = w8a16(x, w, torch.ones(32, device=DEV), residual=torch.zeros(M, 32, dtype=dtype, device=DEV),
              packed=packed, kernel="swapped")
    want = held(x)[torch.arange(M, device=DEV), at]
    assert torch.equal(y, want.to(dtype)[:, None].expand(M, 32))
    whole = value.double() >= x[:, 0].double() * 2.0 ** -13
    assert whole.sum() > M // 3 and torch.equal(want[whole], value.double()[whole])
    assert (want != value.double()).any()
    assert_status_ok()


@pytest.mark.parametrize("dtype,size", [(BF, 2.0 ** -126), (BF, 2.0 ** -120), (BF, 2.0 ** -112), (BF, 2.0 ** -100),
                                        (BF, 2.0 ** 100), (HF, 2.0 ** -20), (HF, 2.0 ** -15), (HF, 2.0 ** 12)])
@pytest.mark.parametrize("kernel", ["stream", "swapped"])
def test_w8a16_rows_near_the_types_ends(dtype, size, kernel):
    """Rows of the smallest and the largest values, with scales that bring the
    results back into the middle: the parts' own scale loses nothing."""
    M, N, K = 20, 96, 64
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = (size * torch.randn(M, K, generator=gen, device=DEV)).to(dtype)
    x[7] = 0
    w = normal_codes(gen, N, K)
    for s in (2.0 ** -9, 2.0 ** -16, 2.0 ** 20):
        if size * s * 2.0 ** 12 > (2.0 ** 120 if dtype is BF else 2.0 ** 14):
            continue
        sw = s * (0.5 + torch.rand(N, generator=gen, device=DEV))
        t, d = ref.linear(held(x) if kernel == "swapped" else x.double(), ref.e4m3_values(w),
                          sw.double().view(1, -1), activation="relu")
        # (a float32 result below 2^-126 is rounded to a multiple of 2^-149)
        ref.check16(w8a16(x, w, sw, activation="relu", kernel=kernel), t, d + 2.0 ** -148, (size, s))
        amax = x.double().abs().amax(1, keepdim=True).clamp(min=2.0 ** -119 if dtype is BF else 0.0)
        assert ((held(x) - x.double()).abs() <= amax * (2.0 ** -21 if dtype is BF else 2.0 ** -25)).all()
    assert_status_ok()


@pytest.mark.parametrize("kernel", ["stream", "swapped"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [3, 20, 100])
def test_w8a16_scales_whose_product_is_subnormal(kernel, gated, M):
    """Sums of zeros and ones times 2^-119, and weight scales of about 2^-16: a
    token's own scale times a weight's is below 2^-126, the result above it,
    and exact before its rounding but for the product with the weight's scale,
    which is rounded once to float32."""
    N, K = 96, 16384
    gen = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randint(0, 2, (M, K), generator=gen, device=DEV).to(BF) * 2.0 ** -119
    w = torch.randint(0, 2, (N, K), generator=gen, device=DEV, dtype=U8) * 0x38
    sw = (0.5 + torch.rand(N, generator=gen, device=DEV)) * 2.0 ** -16
    bias = None
    if gated:  # (up: one, from its bias; its sums are far below one's last place)
        bias = torch.zeros(N, device=DEV)
        bias[N // 2:] = 1.0
    t = ((x.double() @ ref.e4m3_values(w).T) * sw.double()).float()
    if gated:
        t = t[:, : N // 2]
    assert (t > 2.0 ** -125).all()
    y = w8a16(x, w, sw, bias=bias, activation="relu", gated=gated, kernel=kernel)
    assert torch.equal(y, t.to(BF))
    assert_status_ok()


# ------------------------------------------------------------------ repeats

def test_the_same_bits_on_every_call():
    """Norms and gated products of the sizes of a decode step and of a prompt:
    repeated calls agree bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    for M, K in ((16, 4096), (1021, 4096)):
        x, res = (torch.randn(M, K, generator=gen, device=DEV).to(BF) for _ in range(2))
        gamma = torch.ones(K, dtype=BF, device=DEV)
        for mode in ("per_token", "dynamic", "norm_only"):
            first = fl.fp8_add_rmsnorm_quant(x, res, gamma, mode=mode, want_h=True)
            for _ in range(5):
                for u, v in zip(fl.fp8_add_rmsnorm_quant(x, res, gamma, mode=mode, want_h=True), first):
                    assert u is v or torch.equal(u, v)
    os = torch.full((1,), 0.01, device=DEV)
    for M in (16, 333, 1021):
        gen, a, w, sa, sw = operands(M, M, 11008, 4096)
        first = fl.fp8_linear(a, w, sa, sw, activation="silu", gated=True, out_dtype=U8, out_scale=os)
        for _ in range(5):
            assert torch.equal(fl.fp8_linear(a, w, sa, sw, activation="silu", gated=True, out_dtype=U8,
                                             out_scale=os), first)
