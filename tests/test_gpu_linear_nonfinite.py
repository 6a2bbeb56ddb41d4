"""Activations of the linear layers at infinity and at NaN, brought in by a
bias: each as the formula has it (an infinite gate is infinite, NaN for minus
infinity where the formula multiplies it by zero), and no other column
changes."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import linear_ref as ref
from gpu_util import DEV, assert_status_ok
from test_gpu_linear import ACTS, BF, HF, U8, normal_codes, operands

pytestmark = pytest.mark.gpu

VALUES = [float("inf"), float("-inf"), float("nan")]
AT = [5, 17, 40]


def check(call, act, gated, N, out):
    gen = torch.Generator(device=DEV).manual_seed(1)
    bias = torch.randn(N, generator=gen, device=DEV)
    if gated:
        bias[N // 2:] = 300.0  # (up products of one sign)
    bad = bias.clone()
    bad[AT] = torch.tensor(VALUES, device=DEV)
    want, got = call(bias), call(bad)
    width = N // 2 if gated else N
    rest = [n for n in range(width) if n not in AT]
    assert torch.equal(got[:, rest], want[:, rest])
    v = ref.act(act, torch.tensor(VALUES, dtype=torch.float64))
    for n, t in zip(AT, v.tolist()):
        c = got[:, n]
        if out is U8:
            code = 0x7E if t == float("inf") else 0xFE if t == float("-inf") else 0 if t == 0 else 0x7F
            assert (c == code).all() if code != 0x7F else (c & 0x7F == 0x7F).all(), (n, t, c)
        elif t != t:
            assert torch.isnan(c.float()).all(), (n, t, c)
        else:
            assert (c.double() == t).all(), (n, t, c)
    assert_status_ok()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [BF, HF, U8])
@pytest.mark.parametrize("gated", [False, True])
def test_w8a8(act, out, gated):
    for kernel, M in (("stream", 5), ("swapped", 3), ("swapped", 100), ("tiled", 140)):
        gen, a, w, sa, sw = operands(3, M, 128, 64)
        os = torch.ones(1, device=DEV) if out is U8 else None
        check(lambda b: fl.fp8_linear(a, w, sa, sw, bias=b, activation=act, gated=gated, out_dtype=out,
                                      out_scale=os, kernel=kernel), act, gated, 128, out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gated", [False, True])
def test_w8a16(act, dtype, gated):
    gen = torch.Generator(device=DEV).manual_seed(2)
    for kernel, M in (("stream", 5), ("swapped", 3), ("swapped", 60)):
        x = torch.randn(M, 64, generator=gen, device=DEV).to(dtype)
        w, sw = normal_codes(gen, 128, 64), torch.full((128,), 2.0 ** -9, device=DEV)
        check(lambda b: fl.fp8_w8a16_linear(x, w, sw, bias=b, activation=act, gated=gated,
                                            kernel=kernel), act, gated, 128, dtype)
