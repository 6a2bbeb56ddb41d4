"""The linear layers' calls beside other Python threads: a call that waits in
the driver (its launch queue is full) lets the others run, and two threads that
share a stream do not get into each other's scales."""
import threading
import time

import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from gpu_util import DEV, assert_status_ok
from test_gpu_linear import BF, normal_codes, operands

pytestmark = pytest.mark.gpu


def calls(name):
    gen, a, w, sa, sw = operands(1, 2, 32, 32)
    x = torch.randn(600, 32, generator=gen, device=DEV).to(BF)
    y = torch.empty(2, 32, dtype=BF, device=DEV)
    if name == "linear":
        return lambda: fl.fp8_linear(a, w, sa, sw, activation="relu", y=y)
    if name == "w8a16":
        swc = torch.ones(32, device=DEV)
        return lambda: fl.fp8_w8a16_linear(x[:2], w, swc, activation="relu", y=y, kernel="swapped")
    out = dict(total=torch.empty_like(x), q=torch.empty(600, 32, dtype=torch.uint8, device=DEV),
               scale=torch.empty(1, device=DEV))
    return lambda: fl.fp8_add_rmsnorm_quant(x, x, x[0].contiguous(), mode="dynamic", **out)


@pytest.mark.parametrize("name", ["linear", "w8a16", "norm"])
def test_other_threads_run_while_a_launch_waits(name):
    call = calls(name)
    call()
    torch.cuda.synchronize()
    done = threading.Event()
    gap = [0.0]

    def observe():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0] = max(gap[0], now - last)
            last = now

    observer = threading.Thread(target=observe)
    torch.cuda._sleep(2 << 30)  # about a second that the stream stands still
    observer.start()
    start = time.perf_counter()
    for _ in range(4000):  # more launches than the queue holds
        call()
    waited = time.perf_counter() - start
    done.set()
    observer.join()
    torch.cuda.synchronize()
    assert waited > 0.4, "the launch queue was never full"
    assert gap[0] < waited / 4, (gap, waited)
    assert_status_ok()


def test_two_threads_on_one_stream():
    """Dynamic norms of two kernels each, whose maximum passes through the
    stream's workspace; products of both kinds beside them."""
    cases = []
    for i, M in enumerate((300, 140)):
        gen = torch.Generator(device=DEV).manual_seed(i)
        x, res = ((i + 1) * torch.randn(M, 2048, generator=gen, device=DEV) for _ in range(2))
        gamma = torch.ones(2048, device=DEV).to(BF)
        w, sw = normal_codes(gen, 64, 2048), torch.full((64,), 2.0 ** -12, device=DEV)
        cases.append((x.to(BF), res.to(BF), gamma, w, sw))

    def step(x, res, gamma, w, sw):
        q, s, total, h = fl.fp8_add_rmsnorm_quant(x, res, gamma, want_h=True)
        return q, s, total, fl.fp8_linear(q, w, s, sw, activation="silu"), \
            fl.fp8_w8a16_linear(h, w, sw, activation="silu")

    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    wrong, begin = [], threading.Barrier(2)

    def work(i):
        begin.wait()
        for _ in range(10):
            got = [step(*cases[i]) for _ in range(20)]
            wrong.extend(k for g in got for k, (u, v) in enumerate(zip(g, want[i])) if not torch.equal(u, v))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]
    assert_status_ok()
