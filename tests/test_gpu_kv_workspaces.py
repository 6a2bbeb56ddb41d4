"""Workspaces of fp8_kv_attention: one per stream for eager calls, one per
capture for graphs, so that calls that may overlap share neither partials nor
merge counters."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from fp8_quantized_linear_gb300 import _binding as b
from gpu_util import DEV
from test_gpu_kv_attention import check, i32, make, run

pytestmark = pytest.mark.gpu


def test_a_capture_takes_a_workspace_of_its_own():
    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        eager = fl.fp8_kv_attention_workspace(DEV)
        assert fl.fp8_kv_attention_workspace(DEV) is eager
    seen = [eager]
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            ws = fl.fp8_kv_attention_workspace(DEV)
            assert fl.fp8_kv_attention_workspace(DEV) is ws
        seen.append(ws)
    assert len({ws.data_ptr() for ws in seen}) == 3
    with torch.cuda.stream(side):
        assert fl.fp8_kv_attention_workspace(DEV) is eager


@pytest.mark.parametrize("n", [1, 4, 90])
def test_graphs_of_one_stream_replay_beside_each_other_and_eager_calls(n):
    # requests that span blocks, so that every call merges partials
    cases = [make(torch.bfloat16, 64, 8, 2, 128, [n] * 3, [5000, 3000, 900 + i], seed=20 + i)
             for i in range(3)]
    lens = [(i32(s["off"]), i32(s["kv"])) for s in cases]

    def call(i):
        s, (off, kv) = cases[i], lens[i]
        return fl.fp8_kv_attention(s["q"], s["cache"], s["table"], off, kv, s["n"])[0]

    want = [call(i) for i in range(3)]
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        call(0)  # the stream has a workspace before it is captured
    side.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = torch.empty_like(want[i])
            for _ in range(4):
                out.copy_(call(i))
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(side):
            eager = [call(2) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(torch.equal(e, want[2]) for e in eager)


def test_one_capture_over_two_streams():
    s = make(torch.bfloat16, 64, 8, 2, 128, [1] * 3, [5000, 3000, 900], seed=23)
    off, kv = i32(s["off"]), i32(s["kv"])

    def call():
        return fl.fp8_kv_attention(s["q"], s["cache"], s["table"], off, kv, s["n"])[0]

    want, _ = run(s)
    main, side = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        first = call()
        with torch.cuda.stream(side):
            second = call()
        main.wait_stream(side)
    for _ in range(10):
        first.zero_(), second.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, want) and torch.equal(second, want)


@pytest.mark.parametrize("q_lens,kv", [([1, 1], [3000, 129]), ([200, 40], [1500, 40])])
def test_a_time_out_in_a_replayed_graph_is_reported(q_lens, kv):
    # the graph's workspace is its own: any status read reports it
    s = make(torch.bfloat16, 64, 8, 2, 128, q_lens, kv, seed=1)
    off, lens = i32(s["off"]), i32(s["kv"])
    check(s)
    ws = fl.workspace(s["q"].device)
    assert fl.fp8l_read_status(ws) == b.OK
    graphs = []
    for stall in (b.STALL_MMA, 0):
        g = torch.cuda.CUDAGraph()
        fl.fp8l_debug_waits(wait_cycles=1 << 20 if stall else 0, stall_mask=stall)
        try:
            with torch.cuda.graph(g):
                out, _ = fl.fp8_kv_attention(s["q"], s["cache"], s["table"], off, lens, s["n"])
        finally:
            fl.fp8l_debug_waits()
        graphs.append((g, out))
    for _ in range(2):
        graphs[0][0].replay()
        graphs[0][0].replay()
        assert fl.fp8l_read_status(ws) == b.ETIMEOUT
        assert fl.fp8l_read_status(ws) == b.OK
    graphs[1][0].replay()
    assert fl.fp8l_read_status(ws) == b.OK
    assert torch.equal(graphs[1][1], run(s)[0])


FIRST_CALL = """
import torch
import fp8_quantized_linear_gb300 as fl
dev = torch.device("cuda:0")
cache = fl.kv_cache(4, 16, 2, 64, dev)
q = torch.ones(1, 4, 64, dtype=torch.half, device=dev)
table = torch.zeros(1, 1, dtype=torch.int32, device=dev)
off = torch.tensor([0, 1], dtype=torch.int32, device=dev)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = fl.fp8_kv_attention(q, cache, table, off, off[1:], 1, want_lse=True)
g.replay()
torch.cuda.synchronize()
# lse = ln 1; the hardware logarithm of the smallest block scale is within 3
# units of 2^-17, that is 2^-16 in lse
assert bool((out == 0).all()) and bool((lse.abs() <= 2.0 ** -16 * 1.05).all()), (out, lse)
assert fl.fp8l_read_status(fl.workspace(dev)) == 0
"""


def test_the_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    root = b._PKG.rsplit("/", 1)[0]
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True,
                          text=True, timeout=300)
    assert done.returncode == 0, done.stderr


FAILED_LAUNCH = """
import torch
import fp8_quantized_linear_gb300 as fl
dev = torch.device("cuda:0")
cache = fl.kv_cache(4, 16, 2, 64, dev)
q = torch.ones(1, 4, 64, dtype=torch.half, device=dev)
x = torch.ones(1, 8 * 64, dtype=torch.half, device=dev)
i = torch.zeros(1, dtype=torch.int32, device=dev)
off = torch.tensor([0, 1], dtype=torch.int32, device=dev)
table, ws = torch.zeros_like(i).view(1, 1), fl.fp8_kv_attention_workspace(dev)
calls = (lambda: fl.fp8_kv_attention(q, cache, i.view(1, 1), off, off[1:], 1, ws=ws),
         lambda: fl.fp8_qk_norm_rope_append(x, cache, i, i, q=q),
         lambda: fl.fp8_kv_plan(i, i, table, off, 0, 16))
for call in calls:
    call()
    fl.fp8_quant_per_tensor(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(g):
            try:
                torch.cuda.synchronize()  # not allowed here: the capture is lost
            except RuntimeError:
                pass
            try:
                call()
            except fl.Fp8LinearError as e:
                assert e.status == 4, e
            else:
                raise AssertionError("launched into a lost capture")
    except RuntimeError:
        pass
    fl.fp8_quant_per_tensor(x)  # raises if it finds the other call's error
"""


def test_a_launch_that_failed_is_not_reported_by_the_next_call():
    # a lost graph capture refuses launches on its stream, on the host
    import subprocess
    import sys
    root = b._PKG.rsplit("/", 1)[0]
    done = subprocess.run([sys.executable, "-c", FAILED_LAUNCH], cwd=root, capture_output=True,
                          text=True, timeout=300)
    assert done.returncode == 0, done.stderr


def test_two_host_threads_on_streams_of_their_own():
    import threading
    cases = [make(torch.bfloat16, 64, 8, 2, 128, [n] * 3, [5000, 3000, 900], seed=50 + n)
             for n in (1, 4, 90)]
    want = [run(s)[0] for s in cases]
    torch.cuda.synchronize()
    errors = []

    def work(s, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream(DEV)):
                for _ in range(50):
                    assert torch.equal(run(s)[0], w)
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
