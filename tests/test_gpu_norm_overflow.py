"""fp8_add_rmsnorm_quant of rows whose float32 mean square is infinite: a
factor r of zero, as fp8_rmsnorm_quant has it, so finite elements become zeros
and the other rows (and a scale that they share) are what they are."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from gpu_util import DEV, assert_status_ok

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
EPS = 1e-5
MODES = ["dynamic", "static", "per_token", "norm_only"]


def same(u, v):
    """Equal values, NaN where the other has NaN."""
    u, v = u.float(), v.float()
    return torch.equal(torch.isnan(u), torch.isnan(v)) and \
        torch.equal(torch.nan_to_num(u, nan=0.0), torch.nan_to_num(v, nan=0.0))


def both(x, res, gamma, mode):
    s = torch.full((1,), 0.0123, device=DEV) if mode == "static" else None
    q, scale, total, h = fl.fp8_add_rmsnorm_quant(x, res, gamma, EPS, mode=mode, scale=s, want_h=True)
    q2, scale2, _, h2 = fl.fp8_add_rmsnorm_quant(x, res, gamma, EPS, mode=mode, scale=s) \
        if mode != "norm_only" else (q, scale, total, h)
    assert q is None or torch.equal(q, q2) and same(scale, scale2)
    return (q, scale, h), fl.fp8_rmsnorm_quant(total, gamma, EPS, mode=mode, scale=s, want_h=True), total


# one cluster of CTAs, a warp or a block a row, two kernels (dynamic)
SIZES = [(5, 512), (40, 4096), (700, 256), (700, 4096), (300, 16384)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("mode", MODES)
def test_finite_rows_of_large_values(mode, M, K):
    """bf16 rows of 1e20 to 1e38: squares beyond float32."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    x, res = (torch.randn(M, K, generator=gen, device=DEV).to(BF) for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(K, generator=gen, device=DEV)).to(BF)
    bad = [1, M // 2, M - 1]
    for row, size in zip(bad, (1e20, 1e30, 1e37)):
        x[row] = (size * torch.randn(K, generator=gen, device=DEV)).to(BF)
    (q, scale, h), (q_n, scale_n, h_n), total = both(x, res, gamma, mode)
    assert torch.isfinite(total.float()).all()
    assert (h[bad] == 0).all() and same(h[bad], h_n[bad])
    assert torch.isfinite(h.float()).all()
    # elsewhere the two differ by a rounding next to a border at most
    assert (h.float() - h_n.float()).abs().max() <= h_n.float().abs().max() * 2.0 ** -7
    if mode != "norm_only":
        assert torch.equal(q[bad], q_n[bad]) and (q[bad] & 0x7F == 0).all()
        assert torch.isfinite(scale).all()
        torch.testing.assert_close(scale, scale_n, rtol=2.0 ** -7, atol=0)
    if mode == "per_token":
        assert (scale[bad] == 1).all()
    assert_status_ok()


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("mode", MODES)
def test_sums_beyond_fp16(mode, M, K):
    """fp16 rows with one sum that overflows: NaN for that element (infinity
    times zero), zeros beside it, as the norm alone gives."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    x, res = (torch.randn(M, K, generator=gen, device=DEV).to(HF) for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(K, generator=gen, device=DEV)).to(HF)
    bad = [0, M // 2]
    x[bad, K - 3] = res[bad, K - 3] = 60000.0
    (q, scale, h), (q_n, scale_n, h_n), total = both(x, res, gamma, mode)
    assert torch.isinf(total[bad, K - 3].float()).all()
    assert same(h[bad], h_n[bad])
    assert torch.isnan(h[bad, K - 3].float()).all() and (h[bad, :K - 3] == 0).all()
    if mode == "per_token":
        assert same(scale[bad], scale_n[bad])
        assert torch.equal(q[bad], q_n[bad])
    elif mode == "static":
        assert torch.equal(q[bad], q_n[bad])
    elif mode == "dynamic":
        assert same(scale, scale_n)


def test_large_rows_below_the_overflow():
    """bf16 rows of 1e17: the mean square is finite, and h is the formula's."""
    for M in (3, 700):
        gen = torch.Generator(device=DEV).manual_seed(M)
        x = (1e17 * torch.randn(M, 1024, generator=gen, device=DEV)).to(BF)
        gamma = (1 + 0.2 * torch.randn(1024, generator=gen, device=DEV)).to(BF)
        _, _, total, h = fl.fp8_add_rmsnorm_quant(x, x, gamma, EPS, mode="norm_only")
        t = total.double()
        h64 = t / (t.pow(2).mean(1, keepdim=True) + EPS).sqrt() * gamma.double()
        d = h64.abs() * 2.0 ** -17
        assert ((h >= (h64 - d).to(BF)) & (h <= (h64 + d).to(BF))).all()
