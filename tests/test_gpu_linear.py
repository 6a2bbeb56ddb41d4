"""GPU parity of the linear layers with bias, activation, gate and residual in
the epilogue (fp8_linear, fp8_w8a16_linear) against a 64-bit computation, with
the bounds derived in linear_ref."""
import itertools

import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import linear_ref as ref
from gpu_util import DEV, assert_status_ok

pytestmark = pytest.mark.gpu

BF, HF, U8 = torch.bfloat16, torch.float16, torch.uint8
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def codes(gen, *shape, low=0, high=0x7F):
    """Random E4M3 codes of both signs, no NaN."""
    c = torch.randint(low, high, shape, generator=gen, device=DEV, dtype=torch.int32)
    s = torch.randint(0, 2, shape, generator=gen, device=DEV, dtype=torch.int32)
    return (c + 128 * s).to(U8)


def normal_codes(gen, *shape):
    x = 60 * torch.randn(*shape, generator=gen, device=DEV)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(U8)


def operands(seed, M, N, K, per_token=False, per_channel=True, spread=2.0):
    """a, w, a_scale, w_scale with outputs of standard deviation ~ spread."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    a, w = normal_codes(gen, M, K), normal_codes(gen, N, K)
    s = (spread / (3600 * K ** 0.5)) ** 0.5
    sa = s * (0.5 + torch.rand(M if per_token else 1, generator=gen, device=DEV))
    sw = s * (0.5 + torch.rand(N if per_channel else 1, generator=gen, device=DEV))
    return gen, a, w, sa, sw


def check_linear(seed, M, N, K, out=BF, bias=None, activation=None, gated=False, residual=False,
                 per_token=False, per_channel=True, inplace=False, **kw):
    gen, a, w, sa, sw = operands(seed, M, N, K, per_token, per_channel)
    width = N // 2 if gated else N
    b = None if bias is None else torch.randn(N, generator=gen, device=DEV).to(bias)
    r = torch.randn(M, width, generator=gen, device=DEV).to(out) if residual else None
    os = torch.full((1,), 0.013, device=DEV) if out is U8 else None
    t, d = ref.linear(ref.e4m3_values(a), ref.e4m3_values(w),
                      sa.double().view(-1, 1) * sw.double().view(1, -1), b, activation, gated, r)
    y = r if inplace else None
    got = fl.fp8_linear(a, w, sa, sw, bias=b, activation=activation, gated=gated, residual=r,
                        out_dtype=out, out_scale=os, y=y, per_token=per_token, **kw)
    assert got.shape == (M, width) and got.dtype is out
    assert not inplace or got is r
    what = (seed, M, N, K, out, bias, activation, gated, residual)
    if out is U8:
        ref.check8(got, t, d, os, what)
    else:
        ref.check16(got, t, d, what)
    assert_status_ok()
    return got


# tokens on both sides of every rule's bounds
TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 48, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300, 513]


@pytest.mark.parametrize("M", TOKENS)
def test_plain_tokens(M):
    check_linear(M, M, 528, 272, bias=BF, activation="silu", residual=True, per_token=True)


@pytest.mark.parametrize("M", TOKENS)
def test_gated_tokens(M):
    check_linear(M, M, 2 * 336, 400, activation="silu", gated=True, out=U8)
    check_linear(M + 1, M, 2 * 80, 144, bias=HF, activation="gelu_tanh", gated=True, out=HF,
                 residual=True, per_token=True, per_channel=False)


@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 1008, 4112])
@pytest.mark.parametrize("N", [32, 64, 96, 160, 544])
def test_ragged_sizes(N, K):
    for M in (3, 40, 130):
        check_linear(N + K, M, N, K, bias=torch.float32, activation="gelu", out=HF)
        check_linear(N + K, M, N, K, activation="relu", gated=True, out=BF, residual=True)


@pytest.mark.parametrize("M", [5, 33, 140])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [BF, HF, U8])
@pytest.mark.parametrize("gated", [False, True])
def test_every_epilogue(M, act, out, gated):
    n = 0
    for bias, residual, per_token, per_channel in itertools.product(
            (None, BF, HF, torch.float32), (False, True), (False, True), (False, True)):
        if residual and out is U8:
            continue
        n += 1
        check_linear(n, M, 192, 160, out, bias, act, gated, residual, per_token, per_channel)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 4096, 4096), (16, 6144, 4096), (16, 28672, 1024),
                                   (64, 10240, 2048), (100, 4096, 14336), (300, 2048, 4096),
                                   (333, 11008, 4112), (700, 4096, 4096), (1021, 8192, 1024),
                                   (2048, 12288, 512), (4097, 512, 512), (3, 65536, 256)])
def test_large(M, N, K):
    check_linear(M, M, N, K, bias=BF, residual=True, per_token=True, stable_weights=True)
    if N % 32 == 0:
        check_linear(M, M, N, K, activation="silu", gated=True, out=U8, stable_weights=True)


# sizes on both sides of each change of kernel
@pytest.mark.parametrize("M,N,K", [(8, 4096, 12288), (8, 4128, 8192), (8, 512, 16384), (8, 512, 16368),
                                   (16, 512, 4096), (16, 512, 4112), (16, 4160, 4096), (128, 12288, 128),
                                   (129, 12288, 128), (333, 11008, 256), (333, 11008, 272),
                                   (400, 11008, 256), (260, 9728, 128), (260, 9760, 128), (256, 4096, 256),
                                   (257, 4096, 256)])
def test_changes_of_kernel(M, N, K):
    check_linear(M, M, N, K, bias=BF, residual=True, per_token=True, stable_weights=True)
    check_linear(M, M, N, K, activation="silu", gated=True, out=U8, stable_weights=True)


# every kernel over sizes on both sides of its own choices: token tiles, K split
# over clusters of CTAs and of pairs (few tiles, long K), tail tiles
@pytest.mark.parametrize("kernel", ["stream", "swapped", "tiled"])
@pytest.mark.parametrize("M,N,K", [(1, 32, 16), (5, 160, 4096), (40, 2080, 272), (130, 256, 4112),
                                   (260, 1024, 2064), (300, 512, 1040), (600, 4096, 528),
                                   (513, 288, 8192), (1030, 4096, 1024), (700, 20480, 144)])
def test_forced_kernels(kernel, M, N, K):
    check_linear(M, M, N, K, HF, BF, "gelu_tanh", residual=True, per_token=True, kernel=kernel)
    check_linear(M, M, N, K, U8, None, "silu", gated=True, kernel=kernel, stable_weights=True)
    check_linear(M, M, N, K, BF, torch.float32, "relu", gated=True, residual=True, kernel=kernel,
                 per_channel=False, inplace=True)
    check_linear(M, M, N, K, U8, HF, "gelu", kernel=kernel, per_token=True)


@pytest.mark.parametrize("kernel", ["swapped", "tiled"])
@pytest.mark.parametrize("M,N,K", [(20, 512, 4096), (300, 512, 4096), (513, 1024, 2048)])
def test_same_bits_every_time(kernel, M, N, K):
    """Partial sums are added in one order: repeated calls agree bit for bit."""
    first = check_linear(M, M, N, K, activation="silu", kernel=kernel)
    for _ in range(5):
        assert torch.equal(check_linear(M, M, N, K, activation="silu", kernel=kernel), first)


def test_residual_in_place():
    for M in (1, 20, 140, 600):
        check_linear(M, M, 512, 512, residual=True, inplace=True)
        check_linear(M, M, 512, 512, residual=True, inplace=True, gated=True, activation="silu")


def exact_operands(seed, M, N, K):
    """Codes of small whole numbers: every sum is exact in float32."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.tensor([-3.0, -2, -1, 0, 1, 2, 3], device=DEV).to(torch.float8_e4m3fn).view(U8)
    a = table[torch.randint(0, 7, (M, K), generator=gen, device=DEV)]
    w = table[torch.randint(0, 7, (N, K), generator=gen, device=DEV)]
    return gen, a, w


@pytest.mark.parametrize("M", [1, 16, 17, 64, 100, 129, 300, 700])
@pytest.mark.parametrize("gated", [False, True])
def test_exact_numbers(M, gated):
    """Whole-number sums, scales that are powers of two by row and by column:
    every value before the output's rounding is exact, and so is the result."""
    N, K = 1056, 656
    gen, a, w = exact_operands(M, M, N, K)
    sa = torch.exp2(torch.randint(-3, 3, (M,), generator=gen, device=DEV).float())
    sw = torch.exp2(torch.randint(-3, 3, (N,), generator=gen, device=DEV).float())
    b = torch.randint(-8, 8, (N,), generator=gen, device=DEV).to(BF) / 4
    width = N // 2 if gated else N
    r = None if gated else (torch.randint(-64, 64, (M, width), generator=gen, device=DEV) / 8).to(HF)
    z = (ref.e4m3_values(a) @ ref.e4m3_values(w).T) * sa.double()[:, None] * sw.double() + b.double()
    if gated:  # the product of two sums has 25 bits or more: one rounding in float32 before HF's
        t = (z[:, :width].clamp(min=0) * z[:, width:]).float()
    else:
        t = z + r.double()
    y = fl.fp8_linear(a, w, sa, sw, bias=b, residual=r, out_dtype=HF, per_token=True, gated=gated,
                      activation="relu" if gated else None)
    assert torch.equal(y, t.to(HF))


def test_plain_call_is_the_product():
    """Without bias, activation and residual: fp8_scaled_mm, bit for bit."""
    for M, N, K in ((1, 512, 256), (40, 512, 1024), (200, 512, 384), (600, 8192, 512)):
        _, a, w, sa, sw = operands(M, M, N, K, per_token=True)
        y = fl.fp8_linear(a, w, sa, sw, per_token=True)
        assert torch.equal(y, fl.fp8_scaled_mm(a, w, sa, sw, per_token=True))


def test_saturation_and_zero_rows():
    gen, a, w, sa, sw = operands(3, 40, 64, 128, per_token=True)
    a[7] = 0
    a[9] = 0x80
    b = torch.zeros(64, dtype=BF, device=DEV)
    b[3] = -2.5
    os = torch.full((1,), 1e-4, device=DEV)
    y = fl.fp8_linear(a, w, sa, sw, bias=b, out_dtype=U8, out_scale=os, per_token=True)
    v = ref.e4m3_values(y)
    assert (v[7] == torch.where(b.double() == 0, 0.0, -448.0)).all() and (v[9] == v[7]).all()
    assert (v.abs().amax(1)[:7] == 448).all()
    t, d = ref.linear(ref.e4m3_values(a), ref.e4m3_values(w), sa.double()[:, None] * sw.double(), b)
    ref.check8(y, t, d, os)


def test_far_negative_gates():
    """Activations of very negative values go to zero, none to NaN."""
    gen, a, w = exact_operands(1, 24, 64, 64)
    one = torch.ones(1, device=DEV)
    bias = torch.cat([torch.linspace(-1000, 0, 32, device=DEV), torch.ones(32, device=DEV)])
    for act in ACTS[1:]:
        for M in (3, 24):
            y = fl.fp8_linear(a[:M], w, one, one, bias=bias, activation=act, gated=True)
            t, d = ref.linear(ref.e4m3_values(a[:M]), ref.e4m3_values(w), one.double().view(1, 1),
                              bias, act, True)
            assert torch.isfinite(y).all()
            ref.check16(y, t, d, act)


# ------------------------------------------------------------------ W8A16

def check_w8a16(seed, M, N, K, dtype=BF, bias=None, activation=None, gated=False, residual=False,
                packed=False, inplace=False, **kw):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=gen, device=DEV).to(dtype)
    w = normal_codes(gen, N, K)
    sw = (0.5 + torch.rand(N, generator=gen, device=DEV)) / (30 * K ** 0.5)
    width = N // 2 if gated else N
    b = None if bias is None else torch.randn(N, generator=gen, device=DEV).to(bias)
    r = torch.randn(M, width, generator=gen, device=DEV).to(dtype) if residual else None
    t, d = ref.linear(x.double(), ref.e4m3_values(w), sw.double().view(1, -1), b, activation, gated,
                      r, x_error=ref.parts_error(x))
    y = fl.fp8_w8a16_linear(x, fl.fp8_pack_w8a16_weights(w) if packed else w, sw, bias=b,
                            activation=activation, gated=gated, residual=r, y=r if inplace else None,
                            packed=packed, **kw)
    assert y.shape == (M, width) and y.dtype is dtype
    ref.check16(y, t, d, (seed, M, N, K, dtype, bias, activation, gated, residual, packed))
    assert_status_ok()
    return y


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 15, 16, 17, 32, 33, 48, 64, 65, 100])
def test_w8a16_tokens(M, packed):
    check_w8a16(M, M, 528, 272, HF, bias=HF, activation="gelu", residual=True, packed=packed)
    check_w8a16(M, M, 2 * 336, 400, BF, activation="silu", gated=True, packed=packed)


@pytest.mark.parametrize("kernel", ["stream", "swapped"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 32, 16), (3, 96, 4112), (16, 2080, 1040), (49, 256, 528),
                                   (150, 1056, 80)])
def test_w8a16_forced_kernels(kernel, packed, M, N, K):
    for dtype in (BF, HF):
        check_w8a16(M, M, N, K, dtype, torch.float32, "gelu", residual=True, packed=packed,
                    kernel=kernel)
        if N % 32 == 0:
            check_w8a16(M, M, N, K, dtype, HF, "silu", gated=True, packed=packed, kernel=kernel,
                        stable_weights=True)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("N,K", [(32, 16), (64, 48), (96, 64), (160, 80), (1056, 1040), (32, 4112)])
def test_w8a16_ragged(N, K, packed):
    for M in (1, 12, 40):
        check_w8a16(N + K, M, N, K, BF, bias=torch.float32, activation="gelu_tanh", packed=packed)
        check_w8a16(N + K, M, N, K, HF, bias=BF, activation="relu", gated=True, residual=True,
                    packed=packed)


@pytest.mark.parametrize("M", [4, 11, 50])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_w8a16_every_epilogue(M, act, gated):
    n = 0
    for dtype, bias, residual, packed in itertools.product(
            (BF, HF), (None, BF, HF, torch.float32), (False, True), (False, True)):
        n += 1
        check_w8a16(n, M, 192, 160, dtype, bias, act, gated, residual, packed, inplace=residual)


@pytest.mark.parametrize("M,N,K", [(1, 22016, 4096), (16, 4096, 11008), (5, 12288, 4096),
                                   (47, 11008, 4096), (64, 4096, 1024)])
def test_w8a16_large(M, N, K):
    for packed in (False, True):
        check_w8a16(M, M, N, K, HF, residual=True, packed=packed, stable_weights=True)
        check_w8a16(M, M, N, K, BF, activation="silu", gated=True, packed=packed,
                    stable_weights=True)


@pytest.mark.parametrize("M,N,K", [(8, 512, 22016), (9, 4096, 8192), (9, 4128, 8192), (16, 512, 8192),
                                   (16, 512, 8208), (17, 512, 4096)])
def test_w8a16_changes_of_kernel(M, N, K):
    check_w8a16(M, M, N, K, HF, residual=True, packed=True, stable_weights=True)
    check_w8a16(M, M, N, K, BF, activation="silu", gated=True, stable_weights=True)


def test_w8a16_packed_is_the_same():
    for M in (1, 16, 30):
        for gated in (False, True):
            kw = dict(activation="silu", gated=gated, bias=BF)
            assert torch.equal(check_w8a16(M, M, 480, 336, packed=True, **kw),
                               check_w8a16(M, M, 480, 336, packed=False, **kw))


def test_w8a16_plain_call_is_the_product():
    for M, dtype in ((1, HF), (16, HF), (40, HF), (64, HF), (1, BF), (16, BF)):
        gen = torch.Generator(device=DEV).manual_seed(M)
        x = torch.randn(M, 400, generator=gen, device=DEV).to(dtype)
        w, sw = normal_codes(gen, 96, 400), torch.rand(96, generator=gen, device=DEV) / 100
        assert torch.equal(fl.fp8_w8a16_linear(x, w, sw), fl.fp8_w8a16_mm(x, w, sw))


def test_w8a16_plain_calls_of_more_tokens():
    for packed in (False, True):
        check_w8a16(1, 65, 1024, 4096, HF, packed=packed, stable_weights=True)
        check_w8a16(2, 700, 96, 400, HF, packed=packed)
        check_w8a16(3, 17, 96, 400, BF, packed=packed)
        check_w8a16(4, 130, 1024, 4096, BF, packed=packed, stable_weights=True)
