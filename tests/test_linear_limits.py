"""Sizes and memory that the linear layers' entry points refuse before any CUDA
call (fake, never dereferenced addresses).  No kernel is launched."""
import pytest

import fp8_quantized_linear_gb300 as fl
import fp8_quantized_linear_gb300._binding as b
from test_linear_refusals import at


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_linear_gb300 import build
    build.build()
    return fl.load()


def w8a16(lib, **kw):
    ok = dict(x=at(0), dt=b.BF16, w=at(1), sw=at(2), M=17, N=32, K=16, bias=None, bdt=b.F32, act=1,
              res=None, y=at(4), ws=at(6), flags=0, st=None)
    return lib.fp8_w8a16_linear(*dict(ok, **kw).values())


def test_more_parts_than_the_tensor_map_counts(lib):
    """Tokens in parts are rows of one TMA map, at most 2^31 - 1 of them: a call
    with more is refused before its tokens are split."""
    for dt, most in ((b.BF16, (1 << 30) - 64), (b.F16, (1 << 31) // 3 - 64)):
        for M in (most + 200, (1 << 31) - 1):
            for flags in (0, 32):
                assert w8a16(lib, dt=dt, M=M, flags=flags) == b.ESHAPE, (dt, M)
    assert w8a16(lib, M=65535 * 16 + 1, flags=16) == b.ESHAPE


def test_norm_workspace_over_an_input(lib):
    """The dynamic mode writes into its workspace."""
    ok = dict(x=at(0), res=at(1), dt=b.BF16, g=at(2), eps=1e-5, M=9, K=64, total=at(3), q=at(4),
              s=at(5), mode=0, h=at(6), ws=at(7), st=None)
    for name in ("x", "res", "g"):
        assert lib.fp8_add_rmsnorm_quant(*dict(ok, ws=ok[name]).values()) == b.EINVAL, name
        assert lib.fp8_add_rmsnorm_quant(*dict(ok, ws=ok[name] + 64).values()) == b.EINVAL, name
