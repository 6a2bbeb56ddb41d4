"""Bounded waits of the attention kernels: a wait that nothing completes gives
up after a short limit, the call returns a context that stays usable, the
status is read from the call's workspace, and the next call is right again."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from fp8_quantized_linear_gb300 import _binding as b
from test_gpu_kv_attention import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,kv", [([1, 1], [3000, 129]), ([5, 5], [700, 900]),
                                       ([200, 40], [1500, 40])])
def test_stalled_products_time_out(q_lens, kv):
    s = make(torch.bfloat16, 64, 8, 2, 128, q_lens, kv, seed=1)
    ws = fl.fp8_kv_attention_workspace(s["q"].device)
    check(s)
    assert fl.fp8l_read_status(ws) == b.OK
    fl.fp8l_debug_waits(wait_cycles=1 << 20, stall_mask=b.STALL_MMA)
    try:
        run(s)
        assert fl.fp8l_read_status(ws) == b.ETIMEOUT
    finally:
        fl.fp8l_debug_waits()
    check(s)
    assert fl.fp8l_read_status(ws) == b.OK
