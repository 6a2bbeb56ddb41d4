"""Refusals of the linear layers with fused neighbours: argument errors are
found on the host before any CUDA call (fake, never dereferenced addresses),
and the binding refuses tensors it cannot pass on.  No kernel is launched."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import fp8_quantized_linear_gb300._binding as b

A = 0x100000000  # a fake, 16-byte aligned address; buffers sit far apart
STEP = 1 << 36


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_linear_gb300 import build
    build.build()
    return fl.load()


def at(i):
    return A + i * STEP


def linear(lib, **kw):
    ok = dict(a=at(0), w=at(1), M=9, N=256, K=64, sa=at(2), sw=at(3), pc=1, bias=at(4), bdt=b.BF16,
              act=2, res=at(5), os=None, y=at(6), out=b.BF16, ws=at(7), flags=0, st=None)
    return lib.fp8_linear(*dict(ok, **kw).values())


def test_linear_argument_errors(lib):
    def call(**kw):
        return linear(lib, **kw)
    for kw in (dict(out=b.F32), dict(out=-1), dict(act=5), dict(act=-1), dict(act=16 + 5),
               dict(act=32), dict(bdt=b.E4M3), dict(bdt=9), dict(flags=2), dict(flags=8),
               dict(flags=64), dict(out=b.E4M3, res=None), dict(out=b.E4M3, os=at(8))):
        assert call(**kw) == b.EINVAL, kw
    for name in ("a", "w", "sa", "sw", "y"):
        assert call(**{name: None}) == b.EINVAL, name
    for kw in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=8), dict(N=-16), dict(K=0), dict(K=8),
               dict(N=(1 << 20) + 16), dict(K=(1 << 20) + 16), dict(N=48, act=16 + 2)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("a", "w", "y", "res", "ws"):
        assert call(**{name: at(0) + 8}) == b.EALIGN, name
    for name in ("sa", "sw"):
        assert call(**{name: at(2) + 2}) == b.EALIGN, name
    assert call(bias=at(4) + 1) == b.EALIGN
    assert call(bias=at(4) + 2, bdt=b.F32) == b.EALIGN
    assert call(out=b.E4M3, res=None, os=at(8) + 1) == b.EALIGN


def test_linear_output_over_inputs(lib):
    y, size = at(6), 9 * 256 * 2
    for name in ("a", "w", "sa", "sw", "bias", "res"):
        assert linear(lib, **{name: y + size - 16}) == b.EINVAL, name
    for name in ("a", "w", "sa", "sw", "bias"):
        assert linear(lib, **{name: y}) == b.EINVAL, name
    assert linear(lib, res=y - 16) == b.EINVAL
    assert linear(lib, ws=y + 32) == b.EINVAL
    assert linear(lib, res=None, out=b.E4M3, os=y + 4) == b.EINVAL
    # (adjacent buffers and the residual itself pass on to the device check)
    past = (b.ECUDA, b.EUNSUPPORTED)
    if torch.cuda.is_available():
        return
    assert linear(lib, res=y) in past
    assert linear(lib, bias=y + size) in past
    assert linear(lib, M=0, y=None, a=None) in past


def test_w8a16_argument_errors(lib):
    ok = dict(x=at(0), dt=b.F16, w=at(1), sw=at(2), M=17, N=256, K=64, bias=at(3), bdt=b.F16, act=1,
              res=at(4), y=at(5), ws=at(6), flags=0, st=None)

    def call(**kw):
        return lib.fp8_w8a16_linear(*dict(ok, **kw).values())
    for kw in (dict(dt=b.E4M3), dict(dt=b.F32), dict(act=7), dict(bdt=b.E4M3), dict(flags=4),
               dict(flags=8), dict(x=None), dict(w=None), dict(sw=None), dict(y=None),
               dict(ws=None), dict(flags=48)):
        assert call(**kw) == b.EINVAL, kw
    for kw in (dict(M=-1), dict(M=1 << 31), dict(N=24), dict(K=24), dict(N=0), dict(K=-16),
               dict(N=272, act=16 + 1)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("x", "w", "y", "res", "ws"):
        assert call(**{name: at(0) + 4}) == b.EALIGN, name
    assert call(sw=at(2) + 2) == b.EALIGN and call(bias=at(3) + 1) == b.EALIGN
    y = at(5)
    for name in ("x", "w", "sw", "bias", "res", "y"):
        assert call(**{"ws": ok[name] + 16}) == b.EINVAL, name
    for kw in (dict(x=y), dict(w=y + 512), dict(sw=y + 16), dict(bias=y + 16), dict(res=y + 16)):
        assert call(**kw) == b.EINVAL, kw


def test_add_norm_argument_errors(lib):
    ok = dict(x=at(0), res=at(1), dt=b.BF16, g=at(2), eps=1e-5, M=9, K=64, total=at(3), q=at(4),
              s=at(5), mode=0, h=at(6), ws=at(7), st=None)

    def call(**kw):
        return lib.fp8_add_rmsnorm_quant(*dict(ok, **kw).values())
    for kw in (dict(dt=b.E4M3), dict(dt=b.F32), dict(mode=4), dict(mode=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(g=None), dict(s=None),
               dict(x=None), dict(res=None), dict(total=None), dict(q=None), dict(ws=None),
               dict(mode=3, h=None)):
        assert call(**kw) == b.EINVAL, kw
    for kw in (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=24), dict(K=32784), dict(K=-16)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("x", "res", "g", "total", "q", "h", "ws"):
        assert call(**{name: at(0) + 8}) == b.EALIGN, name
    assert call(s=at(5) + 2) == b.EALIGN
    n = 9 * 64
    for kw in (dict(total=at(0) + 16), dict(total=at(1) + 2 * n - 16), dict(q=at(0)), dict(h=at(1)),
               dict(q=at(3) + 2 * n - 16), dict(h=at(3)), dict(h=at(4)), dict(s=at(3)),
               dict(s=at(7) + 16), dict(total=at(2)), dict(q=at(2)), dict(s=at(2)),
               dict(mode=2, s=at(4) - 32), dict(mode=1, s=at(4)), dict(total=at(7))):
        assert call(**kw) == b.EINVAL, kw
    if torch.cuda.is_available():
        return
    past = (b.ECUDA, b.EUNSUPPORTED)
    for kw in (dict(total=at(0)), dict(total=at(1)), dict(q=at(3) + 2 * n), dict(h=None),
               dict(mode=3, q=None, s=None), dict(x=at(1))):
        assert call(**kw) in past, kw


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 64, dtype=torch.uint8)
    s = torch.ones(1)
    with pytest.raises(TypeError):
        fl.fp8_linear(c, c, s, s)
    with pytest.raises(TypeError):
        fl.fp8_w8a16_linear(t, c, s)
    with pytest.raises(TypeError):
        fl.fp8_add_rmsnorm_quant(t, t, t[0])
    with pytest.raises(TypeError):
        fl.fp8_add_rmsnorm_quant(None, t, t[0])
