"""GPU parity of the residual addition fused with RMSNorm and E4M3 quantization
(fp8_add_rmsnorm_quant).

The new residual stream is one float32 addition rounded to 16 bits: exact.  h
is computed in float32 from the stream as written: its factor r has a relative
error below 2^-18 (a sum of at most 32768 exact squares, added in pieces of at
most 16 and then in a tree: 40 roundings of 2^-24, halved by the root; a
division, a root, a reciprocal), the two products 2^-23, so h lies between the
roundings of its 64-bit value times 1 -+ 2^-17.  Given h, codes and scales are
the quantizer's, bit for bit."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import oracle
from gpu_util import DEV, assert_status_ok, host

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
EPS = 1e-5


def inputs(seed, M, K, dtype):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    size = 1 + 30 * (torch.rand(K, generator=gen, device=DEV) < 0.02)
    x = (torch.randn(M, K, generator=gen, device=DEV) * size).to(dtype)
    res = (3 * torch.randn(M, K, generator=gen, device=DEV) * size).to(dtype)
    gamma = (1 + 0.3 * torch.randn(K, generator=gen, device=DEV)).to(dtype)
    return x, res, gamma


def check(x, res, gamma, mode, q, scale, total, h, static=None, eps=EPS):
    want = (x.float() + res.float()).to(x.dtype)
    assert torch.equal(total, want)
    t = want.double()
    h64 = t / (t.pow(2).mean(1, keepdim=True) + eps).sqrt() * gamma.double()
    if h is not None:
        d = h64.abs() * 2.0 ** -17
        assert ((h >= (h64 - d).to(h.dtype)) & (h <= (h64 + d).to(h.dtype))).all()
    if mode == "norm_only":
        assert q is None and scale is None
        return
    hh = host(h).astype(np.float32)
    if mode == "per_token":
        q_o, s_o = oracle.quant_per_row(hh)
    elif mode == "static":
        q_o, s_o = oracle.quant_per_tensor(hh, scale=np.float32(static))
    else:
        q_o, s_o = oracle.quant_per_tensor(hh)
    assert np.array_equal(host(q), q_o)
    assert np.array_equal(host(scale).reshape(-1).view(np.uint32),
                          np.asarray(s_o, np.float32).reshape(-1).view(np.uint32))


def run(x, res, gamma, mode, want_h=True, **kw):
    s = torch.full((1,), 0.0123, device=DEV) if mode == "static" else None
    return fl.fp8_add_rmsnorm_quant(x, res, gamma, EPS, mode=mode, scale=s, want_h=want_h, **kw)


MODES = ["dynamic", "static", "per_token", "norm_only"]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 80), (9, 256), (33, 272), (17, 1024), (5, 1040),
                                 (7, 2064), (40, 4096), (9, 6160), (160, 8192), (21, 14336),
                                 (6, 16400), (3, 32768)])
@pytest.mark.parametrize("mode", MODES)
def test_modes(mode, M, K, dtype):
    x, res, gamma = inputs(M + K, M, K, dtype)
    q, s, total, h = run(x, res, gamma, mode)
    check(x, res, gamma, mode, q, s, total, h, 0.0123)
    if mode != "norm_only":  # the same when h is not written
        q2, s2, total2, h2 = run(x, res, gamma, mode, want_h=False)
        assert h2 is None
        assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(total2, total)
    assert_status_ok()


@pytest.mark.parametrize("M,K", [(1024, 4096), (5000, 272), (3001, 8192), (1300, 16384)])
@pytest.mark.parametrize("mode", ["dynamic", "per_token"])
def test_many_rows(mode, M, K):
    """More rows than the GPU holds at once; dynamic: more than fit shared memory."""
    x, res, gamma = inputs(M + K, M, K, BF)
    q, s, total, h = run(x, res, gamma, mode)
    check(x, res, gamma, mode, q, s, total, h)
    assert_status_ok()


# rows and lengths on both sides of what one cluster of CTAs takes; the rows
# behind the batch stay
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("K", [256, 272, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400])
def test_few_rows_with_one_scale(K, dtype):
    for M in (1, 15, 16, 17, 32, 33, 63, 64, 65, 128, 129, 512, 513):
        if M > 130 and K > 1024:
            continue
        x, res, gamma = inputs(M + K, M, K, dtype)
        x[M // 2, K - 1] = 300.0  # the maximum in any CTA
        q, s, total, h = run(x, res, gamma, "dynamic")
        check(x, res, gamma, "dynamic", q, s, total, h)
        big_q = torch.full((M + 3, K), 7, dtype=torch.uint8, device=DEV)
        big_t = torch.full((M + 3, K), 7, dtype=dtype, device=DEV)
        q2, s2, _, _ = run(x, res, gamma, "dynamic", False, q=big_q[:M], total=big_t[:M])
        assert torch.equal(big_q[:M], q) and torch.equal(s2, s) and torch.equal(big_t[:M], total)
        assert (big_q[M:] == 7).all() and (big_t[M:] == 7).all()


def test_few_rows_that_are_not_finite():
    """A NaN or an infinity in one CTA's row shows in the scale as it does for
    many rows."""
    for bad in (float("nan"), float("inf")):
        x, res, gamma = inputs(3, 600, 256, HF)
        x[5, 9] = bad
        many = run(x, res, gamma, "dynamic")
        few = run(x[:20].contiguous(), res[:20].contiguous(), gamma, "dynamic")
        assert torch.equal(many[1].view(torch.int32), few[1].view(torch.int32))
        assert torch.equal(many[0][:20], few[0])


@pytest.mark.parametrize("mode", MODES)
def test_in_place(mode):
    """The stream updated in its own tensor, or in x's."""
    for M, K in ((5, 512), (700, 4096), (3000, 8192)):
        x, res, gamma = inputs(M, M, K, BF)
        want = run(x, res, gamma, mode)
        for which in (0, 1):
            pair = [x.clone(), res.clone()]
            got = run(*pair, gamma, mode, total=pair[which])
            assert got[2] is pair[which]
            for u, v in zip(got, want):
                assert (u is None and v is None) or torch.equal(u, v)


def test_zero_and_cancelling_rows():
    """Rows whose sum is zero: h and the codes are zeros, the scale 1."""
    for mode in ("dynamic", "per_token"):
        x, res, gamma = inputs(1, 6, 512, HF)
        res[2], x[4], res[4] = -x[2], 0, 0
        q, s, total, h = run(x, res, gamma, mode)
        check(x, res, gamma, mode, q, s, total, h)
        assert (h[[2, 4]] == 0).all()
        if mode == "per_token":
            assert (s[[2, 4]] == 1).all()
        q, s, total, h = run(torch.zeros_like(x), torch.zeros_like(x), gamma, mode)
        assert (s == 1).all() and (q & 0x7F == 0).all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device=DEV)
    g = torch.ones(64, dtype=BF, device=DEV)
    for mode in MODES:
        q, s, total, h = run(x, x, g, mode)
        if mode == "dynamic":
            assert s.item() == 1
        assert total.shape == (0, 64)


def test_bytes_of_large_and_small_values():
    """Sums past the type's largest value, and subnormal ones, as they round."""
    x = torch.tensor([[60000.0, -60000, 1e-7, 3e-8] * 8], device=DEV).to(HF)
    g = torch.ones(32, dtype=HF, device=DEV)
    _, _, total, _ = fl.fp8_add_rmsnorm_quant(x[:, 2:].repeat(1, 2)[:, :32], x, g, mode="norm_only")
    assert torch.equal(total, (x[:, 2:].repeat(1, 2)[:, :32].float() + x.float()).to(HF))


def test_graph_beside_eager_calls():
    """Two captured graphs and eager calls on another stream, dynamic mode: none
    shares barrier words with another."""
    args = [inputs(i, 300 + i, 4096, BF) for i in range(3)]
    want = [run(*a, "dynamic") for a in args]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([run(*a, "dynamic") for _ in range(3)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = run(*args[2], "dynamic")
    torch.cuda.synchronize()
    for got, w in zip(outs + [[eager]], want):
        for one in got:
            for u, v in zip(one, w):
                assert torch.equal(u, v)
    assert_status_ok()


def test_few_rows_in_graphs_and_streams():
    """Dynamic calls of one cluster among calls of two kernels: captured, on
    three streams at once, and each call's stream read by the next."""
    sizes = [(1, 4096), (20, 8192), (300, 2048), (16, 16384), (400, 128)]
    args = [inputs(i, M, K, BF if i & 1 else HF) for i, (M, K) in enumerate(sizes)]

    def chain():
        out = []
        for x, res, gamma in args:
            first = run(x, res, gamma, "dynamic")
            out += [first, run(first[2], res, gamma, "dynamic", False)]
        return out

    want = chain()
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(chain())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = chain()
    torch.cuda.synchronize()
    for one in got + [eager]:
        for u, v in zip(one, want):
            assert all(torch.equal(a, b) for a, b in zip(u, v) if a is not None)
    assert_status_ok()
