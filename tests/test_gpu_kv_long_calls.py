"""A call of the attention kernels that takes longer than any of its waits may."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import kv_ref
from fp8_quantized_linear_gb300 import _binding as b

pytestmark = pytest.mark.gpu


def test_a_call_longer_than_a_wait_may_be_is_no_time_out():
    # 720 thousand tokens of one prompt: about three seconds, longer than the
    # two that any single wait is given
    T, page, hq, hkv, dim = 720_000, 128, 32, 8, 128
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    q = torch.empty(T, hq, dim, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    pages = T // page
    shape = (pages, hkv, page // 8, dim // 16, 8, 16)
    codes = [torch.randint(0x20, 0x48, shape, dtype=torch.uint8, device=dev, generator=gen)
             | (torch.randint(0, 2, shape, dtype=torch.uint8, device=dev, generator=gen) << 7)
             for _ in range(2)]
    scales = [torch.full((pages, hkv), s, device=dev) for s in (0.5, 1.0)]
    cache = fl.KvCache(*codes, *scales)
    table = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)[None].contiguous()
    off = torch.tensor([0, T], dtype=torch.int32, device=dev)
    ws = fl.fp8_kv_attention_workspace(dev)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    out, _ = fl.fp8_kv_attention(q, cache, table, off, off[1:], T)
    end.record()
    assert fl.fp8l_read_status(ws) == b.OK
    assert begin.elapsed_time(end) > 2300
    # rows of the first, a middle and the last tile
    value = torch.from_numpy(kv_ref.TABLE).to(dev)

    def rows(c, s, g):
        x = value[c[table[0].long(), g].long()].transpose(2, 3) * s
        return x.reshape(-1, dim)

    for g in (0, 5):
        k, v = rows(codes[0], 0.5, g), rows(codes[1], 1.0, g)
        for t in (0, 200, 360_001, T - 1):
            h = g * (hq // hkv) + t % 4
            p = torch.softmax(k[:t + 1] @ q[t, h].double() * dim ** -0.5, 0)
            want, spread = p @ v[:t + 1], p @ v[:t + 1].abs()
            err = (out[t, h].double() - want).abs()
            assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * spread).all()), (t, h, err.max())
