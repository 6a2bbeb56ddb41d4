"""The linear layers and their norm at the largest extents: operands and results
whose offsets pass 32 bits, the longest rows and the most channels.  Codes are
zeros and ones and scales powers of two, so sums are exact; far rows and
columns are compared with 64 bits, rows of a norm with the same rows alone."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import linear_ref as ref
from gpu_util import DEV, assert_status_ok
from test_gpu_linear import BF, HF, U8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def ones(gen, *shape):
    """Codes of 0 and 1."""
    c = torch.randint(0, 2, shape, generator=gen, device=DEV, dtype=U8)
    return c.mul_(0x38)


def some(n):
    """A few indexes of n, the first and the last among them."""
    return sorted({0, 1, n // 3, n // 2 + 1, n - 17, n - 1} & set(range(n)))


def check(call, x, w, out, gated, residual, M, N):
    """call(residual) of E4M3 (or 16-bit) x, rows of w; scales 1/8 and 1/2."""
    width = N // 2 if gated else N
    r = None
    if residual:
        r = torch.empty(M, width, dtype=out, device=DEV)
        r.copy_(torch.arange(width, device=DEV) % 7)
    y = call(r)
    rows, cols = some(M), some(width)
    xs = ref.e4m3_values(x[rows]) if x.dtype is U8 else x[rows].double()

    def z(n):
        return xs @ ref.e4m3_values(w[n]).T / 16

    t = z(cols)
    if gated:
        t = (t.clamp(min=0) * z([width + n for n in cols])).float().double()
    if residual:
        t = t + (torch.tensor(cols, device=DEV) % 7).double()
    got = y[rows][:, cols]
    if out is U8:
        assert torch.equal(ref.e4m3_values(got), ref.e4m3_round(t / 64))
    else:
        assert torch.equal(got, t.to(out))
    assert_status_ok()


def w8a8(M, N, K, kernel, out, gated, residual):
    gen = torch.Generator(device=DEV).manual_seed(M)
    a, w = ones(gen, M, K), ones(gen, N, K)
    sa, sw = torch.full((1,), 0.125, device=DEV), torch.full((1,), 0.5, device=DEV)
    os = torch.full((1,), 64.0, device=DEV) if out is U8 else None
    check(lambda r: fl.fp8_linear(a, w, sa, sw, activation="relu" if gated else None, gated=gated, residual=r,
                                  y=r, out_dtype=out, out_scale=os, kernel=kernel, stable_weights=True),
          a, w, out, gated, residual, M, N)


KERNELS = ["stream", "swapped", "tiled"]


@pytest.mark.parametrize("kernel", KERNELS)
def test_results_past_32_bits(kernel):
    w8a8(66000, 32800, 32, kernel, BF, False, True)
    w8a8(66000, 65600, 32, kernel, U8, True, False)


@pytest.mark.parametrize("kernel", KERNELS)
def test_tokens_past_32_bits(kernel):
    w8a8(140000, 64, 32768, kernel, HF, False, False)


@pytest.mark.parametrize("kernel,M", [("stream", 5), ("stream", 12), ("swapped", 20), ("tiled", 140)])
@pytest.mark.parametrize("gated", [False, True])
def test_weights_past_32_bits(kernel, M, gated):
    w8a8(M, 140000, 32768, kernel, BF, gated, True)


@pytest.mark.parametrize("kernel,M", [("stream", 5), ("swapped", 20), ("swapped", 200), ("tiled", 140)])
def test_longest_rows_and_most_channels(kernel, M):
    w8a8(M, 64, 1 << 20, kernel, BF, False, True)
    w8a8(M, 64, 1 << 20, kernel, U8, True, False)
    w8a8(M, 1 << 20, 16, kernel, BF, False, True)
    w8a8(M, 1 << 20, 48, kernel, U8, True, False)


@pytest.mark.parametrize("kernel,M", [("stream", 5), ("swapped", 20)])
@pytest.mark.parametrize("packed", [False, True])
def test_w8a16_weights_past_32_bits(kernel, M, packed):
    N, K = 140000, 32768
    gen = torch.Generator(device=DEV).manual_seed(M)
    w = ones(gen, N, K)
    wp = fl.fp8_pack_w8a16_weights(w) if packed else w
    sw = torch.full((N,), 0.0625, device=DEV)
    x = torch.randint(0, 2, (M, K), generator=gen, device=DEV).to(BF)
    for gated in (False, True):
        check(lambda r: fl.fp8_w8a16_linear(x, wp, sw, activation="relu" if gated else None, gated=gated,
                                            residual=r, y=r, packed=packed, kernel=kernel,
                                            stable_weights=True), x, w, BF, gated, True, M, N)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kernel", ["stream", "swapped"])
def test_w8a16_tokens_past_32_bits(dtype, kernel):
    """(tokens in parts: 9 to 14 GB of them)"""
    M, N, K = 140000, 64, 32768
    gen = torch.Generator(device=DEV).manual_seed(M)
    w, sw = ones(gen, N, K), torch.full((N,), 0.0625, device=DEV)
    x = torch.empty(M, K, dtype=dtype, device=DEV)
    for m in range(0, M, 10000):
        x[m:m + 10000] = torch.randint(0, 2, (10000, K), generator=gen, device=DEV, dtype=U8)
    check(lambda r: fl.fp8_w8a16_linear(x, w, sw, residual=r, y=r, kernel=kernel), x, w, dtype, False, True, M, N)


@pytest.mark.parametrize("M,K", [(140000, 16384), (9000000, 256)])
def test_norms_past_32_bits(M, K):
    gen = torch.Generator(device=DEV).manual_seed(K)
    part = torch.randn(M // 8, K, generator=gen, device=DEV, dtype=BF)
    x, res = part.repeat(8, 1), part.flip(0).repeat(8, 1)
    for i in range(8):
        x[i * (M // 8):(i + 1) * (M // 8)] *= i + 1
    x[M - 3, K - 1] = 900.0  # the largest, in the last rows
    gamma = (1 + 0.2 * torch.randn(K, generator=gen, device=DEV)).to(BF)
    del part
    ends = [slice(0, 40), slice(M // 2 - 7, M // 2 + 40), slice(M - 40, M)]
    for mode in ("per_token", "dynamic"):
        q, s, total, h = fl.fp8_add_rmsnorm_quant(x, res, gamma, mode=mode)
        for i in ends:
            if mode == "per_token":
                want = fl.fp8_add_rmsnorm_quant(x[i], res[i], gamma, mode=mode)
                assert torch.equal(s[i], want[1])
            else:  # one scale, of a row behind 2^31 elements
                want = fl.fp8_add_rmsnorm_quant(x[i], res[i], gamma, mode="static", scale=s)
            assert torch.equal(q[i], want[0]) and torch.equal(total[i], want[2])
        if mode == "dynamic":
            top = fl.fp8_add_rmsnorm_quant(x[M - 3:M - 2], res[M - 3:M - 2], gamma, mode=mode)[1]
            assert torch.equal(s, top)
    del q, total
    _, _, total, h = fl.fp8_add_rmsnorm_quant(x, res, gamma, mode="norm_only", total=res)
    assert total is res
    for i in ends:
        # (the stream's rows as they stand: nothing added to them)
        want = fl.fp8_add_rmsnorm_quant(torch.zeros_like(total[i]), total[i].clone(), gamma, mode="norm_only")
        assert torch.equal(h[i], want[3])
    assert_status_ok()
