"""Calls of the linear layers that a program makes around the numbers: waits
that give up, graphs beside eager calls, streams, no tokens, views, refusals of
the binding."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from fp8_quantized_linear_gb300 import _binding as b
from gpu_util import DEV, assert_status_ok
from test_gpu_linear import BF, HF, U8, check_linear, check_w8a16, normal_codes, operands

pytestmark = pytest.mark.gpu


# swapped operands with and without a cluster, pairs of SMs, pairs splitting K
@pytest.mark.parametrize("kernel,M,N,K", [("swapped", 20, 512, 1024), ("swapped", 20, 512, 64),
                                          ("tiled", 300, 512, 256), ("tiled", 300, 512, 4096)])
@pytest.mark.parametrize("given", [False, True])
def test_stalled_products_time_out(kernel, M, N, K, given):
    kw = dict(activation="silu", gated=True, residual=True, kernel=kernel)
    check_linear(1, M, N, K, **kw)
    ws = fl.workspace(DEV)
    assert fl.fp8l_read_status(ws) == b.OK
    gen, a, w, sa, sw = operands(1, M, N, K)
    r = torch.zeros(M, N // 2, dtype=BF, device=DEV)
    fl.fp8l_debug_waits(wait_cycles=1 << 20, stall_mask=b.STALL_MMA)
    try:
        fl.fp8_linear(a, w, sa, sw, activation="silu", gated=True, residual=r, kernel=kernel,
                      ws=ws if given else None)
        assert fl.fp8l_read_status(ws) == b.ETIMEOUT
        assert fl.fp8l_read_status(ws) == b.OK
    finally:
        fl.fp8l_debug_waits()
    check_linear(1, M, N, K, **kw)


def test_stalled_w8a16_times_out():
    ws = fl.workspace(DEV)
    check_w8a16(1, 30, 512, 1024, activation="silu")
    x = torch.zeros(30, 1024, dtype=BF, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    w, sw = normal_codes(gen, 512, 1024), torch.ones(512, device=DEV)
    fl.fp8l_debug_waits(wait_cycles=1 << 20, stall_mask=b.STALL_MMA)
    try:
        fl.fp8_w8a16_linear(x, w, sw, activation="silu")
        assert fl.fp8l_read_status(ws) == b.ETIMEOUT
    finally:
        fl.fp8l_debug_waits()
    check_w8a16(1, 30, 512, 1024, activation="silu")


@pytest.mark.parametrize("M", [3, 40, 300])
def test_graphs_and_eager_calls_at_once(M):
    """Two graphs and eager calls on three streams, over and over: each its own
    results."""
    cases = []
    for i in range(3):
        gen, a, w, sa, sw = operands(10 + i, M, 1024, 2048, per_token=True)
        x = torch.randn(M, 2048, generator=gen, device=DEV).to(HF)
        r = torch.randn(M, 1024, generator=gen, device=DEV).to(HF)
        cases.append((a, w, sa, sw, x, r))

    def call(c):
        a, w, sa, sw, x, r = c
        y = fl.fp8_linear(a, w, sa, sw, activation="gelu", residual=r, per_token=True,
                          stable_weights=True)
        return y, fl.fp8_w8a16_linear(x, w, sw, activation="silu", gated=True, stable_weights=True)

    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([call(c) for _ in range(3)][-1])
        graphs.append(g)
    streams = [torch.cuda.Stream(DEV) for _ in range(3)]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [call(cases[2]) for _ in range(2)][-1]
    torch.cuda.synchronize()
    for got, one in zip(outs + [eager], want):
        assert all(torch.equal(u, v) for u, v in zip(got, one))
    assert_status_ok()


def test_chained_calls_see_each_other():
    """Programmatic dependents: a chain in which every call reads what the call
    before wrote, replayed with the intermediates cleared, is the eager one."""
    M, K = 24, 1024
    gen, a, w, sa, sw = operands(3, M, 2 * K, K, per_token=True)
    w2 = normal_codes(gen, K, K)
    s2 = torch.full((K,), 2.0 ** -13, device=DEV)
    os = torch.full((1,), 0.02, device=DEV)
    gamma = torch.ones(K, dtype=BF, device=DEV)
    bufs = dict(act=torch.empty(M, K, dtype=U8, device=DEV),
                stream=torch.empty(M, K, dtype=BF, device=DEV),
                total=torch.empty(M, K, dtype=BF, device=DEV),
                q=torch.empty(M, K, dtype=U8, device=DEV), s=torch.empty(M, device=DEV),
                h=torch.empty(M, K, dtype=BF, device=DEV), y=torch.empty(M, K, dtype=BF, device=DEV))

    def chain():
        fl.fp8_linear(a, w, sa, sw, activation="silu", gated=True, out_dtype=U8, out_scale=os,
                      y=bufs["act"], per_token=True, stable_weights=True)
        fl.fp8_linear(bufs["act"], w2, os, s2, bias=gamma, y=bufs["stream"], stable_weights=True)
        fl.fp8_add_rmsnorm_quant(bufs["stream"], bufs["stream"], gamma, mode="per_token",
                                 total=bufs["total"], q=bufs["q"], scale=bufs["s"], h=bufs["h"])
        fl.fp8_w8a16_linear(bufs["h"], w2, s2, activation="gelu", residual=bufs["total"],
                            y=bufs["y"], stable_weights=True)

    chain()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in bufs.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            chain()
    for _ in range(5):
        for v in bufs.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for k, v in bufs.items():
            assert torch.equal(v, want[k]), k


def test_no_tokens():
    gen, a, w, sa, sw = operands(1, 4, 64, 64)
    y = fl.fp8_linear(a[:0], w, sa, sw, activation="relu", gated=True)
    assert y.shape == (0, 32)
    assert fl.fp8_linear(a[:0], w, sa, sw).shape == (0, 64)
    assert fl.fp8_linear(a[:0], w, sa[:0], sw, activation="relu").shape == (0, 64)
    assert fl.fp8_linear(a[:0], w, sa[:0], sw, activation="relu", per_token=True).shape == (0, 64)
    x = torch.empty(0, 64, dtype=HF, device=DEV)
    assert fl.fp8_w8a16_linear(x, w, sw, activation="relu").shape == (0, 64)


def test_rows_behind_the_batch_stay():
    """Outputs into the first rows of a larger buffer leave the rest alone."""
    for M in (1, 9, 40, 200, 300):
        gen, a, w, sa, sw = operands(M, M, 256, 512)
        big = torch.full((M + 64, 256), 7.0, dtype=BF, device=DEV)
        fl.fp8_linear(a, w, sa, sw, activation="silu", y=big[:M])
        assert (big[M:] == 7).all()
        x = torch.randn(M, 512, generator=gen, device=DEV).to(BF)
        fl.fp8_w8a16_linear(x, w, sw, activation="silu", y=big[:M])
        assert (big[M:] == 7).all()
        rows = torch.full((M + 32, 512), 7.0, dtype=BF, device=DEV)
        fl.fp8_add_rmsnorm_quant(x, x, torch.ones(512, dtype=BF, device=DEV), mode="norm_only",
                                 h=rows[:M])
        assert (rows[M:] == 7).all()


@pytest.mark.parametrize("kernel", ["stream", "swapped", "tiled"])
def test_rows_behind_the_batch_stay_in_every_kernel(kernel):
    os = torch.ones(1, device=DEV)
    for M in (1, 37, 300):
        gen, a, w, sa, sw = operands(M, M, 320, 512)
        r = torch.randn(M, 320, generator=gen, device=DEV).to(BF)
        for dtype, kw in ((BF, dict(residual=r)), (U8, dict(out_scale=os))):
            big = torch.full((M + 300, 320), 7, dtype=dtype, device=DEV)
            fl.fp8_linear(a, w, sa, sw, bias=r[0].contiguous(), y=big[:M], kernel=kernel, **kw)
            assert (big[M:] == 7).all()


def test_values_that_are_not_finite_show():
    """W8A16: a token with an infinity or a NaN has no finite result, whatever
    the kernel, and the others are what they are without it."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    w = normal_codes(gen, 96, 256)
    sw = torch.full((96,), 2.0 ** -12, device=DEV)
    for dtype in (BF, HF):
        x = torch.randn(24, 256, generator=gen, device=DEV).to(dtype)
        bad = x.clone()
        bad[3, 7], bad[11, 200], bad[20, 0] = float("inf"), float("nan"), float("-inf")
        rows = [i for i in range(24) if i not in (3, 11, 20)]
        for kernel in ("stream", "swapped"):
            want = fl.fp8_w8a16_linear(x, w, sw, activation="silu", kernel=kernel)
            got = fl.fp8_w8a16_linear(bad, w, sw, activation="silu", kernel=kernel)
            assert torch.equal(got[rows], want[rows])
            # (silu of minus infinity is 0 times infinity, of infinity infinity)
            assert not torch.isfinite(got[[3, 11, 20]]).any()


def test_a_long_call_before_is_no_time_out():
    """A dependent that is resident early does not count the preceding kernel's
    time: the waits limited to 0.13 ms, behind a call of about half a millisecond
    that leaves SMs free."""
    K = 1 << 20
    long_a = torch.zeros(1, K, dtype=U8, device=DEV)
    long_w = torch.zeros(2048, K, dtype=U8, device=DEV)
    one = torch.ones(1, device=DEV)
    gen, a, w, sa, sw = operands(5, 40, 512, 256)
    want = {k: fl.fp8_linear(a, w, sa, sw, activation="silu", kernel=k) for k in ("swapped", "tiled")}
    fl.fp8l_debug_waits(wait_cycles=1 << 18)
    try:
        for k in ("swapped", "tiled"):
            fl.fp8_linear(long_a, long_w, one, one, activation="relu", kernel="stream",
                          stable_weights=True)
            got = fl.fp8_linear(a, w, sa, sw, activation="silu", kernel=k, stable_weights=True)
            assert torch.equal(got, want[k])
            assert_status_ok()
    finally:
        fl.fp8l_debug_waits()


def test_codes_as_float8_and_offsets():
    """E4M3 tensors as float8, bias views at odd offsets, rows of a larger tensor."""
    gen, a, w, sa, sw = operands(2, 12, 96, 128)
    bias = torch.randn(97, generator=gen, device=DEV).to(HF)[1:]
    y = fl.fp8_linear(a, w, sa, sw, bias=bias, out_dtype=HF)
    f8 = torch.float8_e4m3fn
    assert torch.equal(fl.fp8_linear(a.view(f8), w.view(f8), sa, sw, bias=bias, out_dtype=HF), y)
    os = torch.ones(1, device=DEV)
    z = fl.fp8_linear(a, w, sa, sw, bias=bias, out_dtype=f8, out_scale=os)
    assert z.dtype is U8
    out = torch.empty(12, 96, dtype=f8, device=DEV)
    assert fl.fp8_linear(a, w, sa, sw, bias=bias, out_scale=os, y=out) is out
    assert torch.equal(out.view(U8), z)


def test_binding_refusals():
    gen, a, w, sa, sw = operands(2, 12, 96, 128)
    x = torch.randn(12, 128, generator=gen, device=DEV).to(HF)
    r = torch.zeros(12, 96, dtype=BF, device=DEV)
    g = torch.ones(128, dtype=HF, device=DEV)
    os = torch.ones(1, device=DEV)
    L, W, N = fl.fp8_linear, fl.fp8_w8a16_linear, fl.fp8_add_rmsnorm_quant
    for call in (
            lambda: L(a, w, sa, sw, activation="swish"), lambda: L(a, w, sa, sw, kernel="fast"),
            lambda: L(a, w[:, :112].contiguous(), sa, sw), lambda: L(a, w, sa, sw[:50].contiguous()),
            lambda: L(a, w, torch.ones(5, device=DEV), sw), lambda: L(a, w, sa.double(), sw),
            lambda: L(a, w, sa, sw.half()), lambda: L(a.int(), w, sa, sw),
            lambda: L(a, w, sa, sw, bias=torch.ones(95, device=DEV)),
            lambda: L(a, w, sa, sw, bias=torch.ones(96, dtype=torch.double, device=DEV)),
            lambda: L(a, w, sa, sw, residual=r[:, :48].contiguous()),
            lambda: L(a, w, sa, sw, residual=r, gated=True),
            lambda: L(a, w, sa, sw, residual=r, out_dtype=HF),
            lambda: L(a, w, sa, sw, residual=r, out_dtype=U8, out_scale=os),
            lambda: L(a, w, sa, sw, out_dtype=U8), lambda: L(a, w, sa, sw, out_dtype=torch.float32),
            lambda: L(a, w, sa, sw, y=r, out_dtype=HF), lambda: L(a, w, sa, sw, y=r[:11]),
            lambda: L(a, w, sa, sw, ws=torch.zeros(8, dtype=U8, device=DEV)),
            lambda: L(a, w.t(), sa, sw), lambda: L(a[:, ::2], w, sa, sw),
            lambda: W(x.float(), w, sw), lambda: W(x, w, sw[:80].contiguous()),
            lambda: W(x, w.view(-1)[:-16], sw, packed=True), lambda: W(x, w, sw, residual=r),
            lambda: W(x, w, sw, y=r), lambda: W(x[0], w, sw),
            lambda: N(x, x[:5], g), lambda: N(x, x, g.float()), lambda: N(x, x, g, mode="none"),
            lambda: N(x, x.to(BF), g), lambda: N(x, x, g, total=r), lambda: N(x, x, g, mode="static"),
            lambda: N(x, x, g, mode="per_token", scale=os), lambda: N(x, x, g, q=a[:3]),
            lambda: N(x, x, g, h=x.float()), lambda: N(x, x, g, ws=os)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: L(a, w, sa, None), lambda: L(a, w.cpu(), sa, sw), lambda: W(x, None, sw),
                 lambda: W(x.cpu(), w, sw), lambda: N(x, None, g), lambda: N(x, x, g.cpu()),
                 lambda: L(a, w, sa, sw, out_dtype="bf16")):
        with pytest.raises(TypeError):
            call()
    # overlaps and what the library refuses
    for call in (lambda: L(a, w[:40], sa, sw[:40].contiguous(), activation="relu"),
                 lambda: L(a, w[:48], sa, sw[:48].contiguous(), gated=True),
                 lambda: N(x, x, g, total=x, h=x, mode="norm_only"),
                 lambda: W(x, w, sw, y=x[:, :96].contiguous().copy_(x[:, :96]), kernel="tiled",
                           activation="relu")):
        with pytest.raises(fl.Fp8LinearError):
            call()
    assert_status_ok()


def test_a_fresh_process_captures_first(tmp_path):
    """The first calls of a process inside a graph capture."""
    import subprocess
    import sys
    code = """
import torch, sys
sys.path.insert(0, %r)
import fp8_quantized_linear_gb300 as fl
g = torch.Generator(device="cuda").manual_seed(1)
c = lambda *s: (60 * torch.randn(*s, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
a, w = c(300, 256), c(512, 256)
s = torch.full((1,), 0.01, device="cuda")
x = torch.randn(20, 256, generator=g, device="cuda").bfloat16()
sw = torch.full((512,), 0.01, device="cuda")
gam = torch.ones(256, dtype=torch.bfloat16, device="cuda")
def calls():
    return [fl.fp8_linear(a, w, s, s, activation="silu"), fl.fp8_linear(a[:20], w, s, s, activation="silu"),
            fl.fp8_linear(a[:1], w, s, s, activation="silu"),
            fl.fp8_w8a16_linear(x, w, sw, activation="silu"),
            *[t for t in fl.fp8_add_rmsnorm_quant(x, x, gam) if t is not None]]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
want = calls()
assert all(torch.equal(u, v) for u, v in zip(got, want))
print("same")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code % root], capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stderr[-2000:]
