"""The attention layer over the paged FP8 cache (PagedAttentionBlock): a
prompt, decode steps, drafted tokens and a second request chained through one
cache, each stage compared with a 64-bit computation from the values that the
stage itself was given, and a captured step replayed."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import kv_ref
import oracle
import synthetic
from fp8_quantized_linear_gb300 import _binding as b
from fp8_quantized_linear_gb300.block import SHAPES
from fp8_quantized_linear_gb300.paged_block import (HEAD_DIM, HEADS, KV_HEADS, PagedAttentionBlock,
                                                    rotation_table)
from gpu_util import DEV, assert_gemm_close, assert_status_ok, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def weights():
    return {n: synthetic.weight(*SHAPES[n], torch.bfloat16, seed=50 + i)
            for i, n in enumerate(("qkv", "o"))}


def make(weights, **kw):
    gen = torch.Generator().manual_seed(1)
    gammas = {n: (1 + 0.1 * torch.randn(HEAD_DIM, generator=gen)).bfloat16().to(DEV)
              for n in ("q_gamma", "k_gamma")}
    return PagedAttentionBlock({k: v.to(DEV) for k, v in weights.items()}, num_pages=40, requests=3,
                               max_tokens=600, page_size=32, **gammas, **kw)


def values(cache, table, length):
    """64-bit keys and values [kv_heads, length, dim] of one request."""
    out = []
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        v = kv_ref.TABLE[kv_ref.pages_view(codes)] * scale.double().cpu().numpy()[:, :, None, None]
        pages = table[: -(-length // cache.page_size)]
        v = v[pages].transpose(1, 0, 2, 3).reshape(KV_HEADS, -1, HEAD_DIM)[:, :length]
        out.append(torch.from_numpy(np.ascontiguousarray(v)))
    return out


def test_steps_of_mixed_requests(weights):
    blk = make(weights)
    rng_lens = [[70, 0, 33], [1, 5, 1], [1, 1, 1], [40, 1, 3]]
    past = np.zeros(3, int)
    qw_o, sw_o = oracle.quant_per_row(weights["o"])
    for n, q_lens in enumerate(rng_lens):
        x = synthetic.activation(sum(q_lens), 4096, torch.bfloat16, seed=n).to(DEV)
        plan = blk.plan(torch.tensor(q_lens, dtype=torch.int32, device=DEV), sum(q_lens))
        y = blk.forward(x, plan, max(q_lens))
        past += q_lens
        assert plan.kv_lens.tolist() == list(past) and plan.used.tolist()[1] == 0
        # what the stages were given and gave, stage by stage
        codes, scale, _ = fl.fp8_rmsnorm_quant(x, blk.gamma, blk.eps)
        qkv = fl.fp8_scaled_mm(codes, blk.w["qkv"], scale, blk.sw["qkv"])
        heads = qkv.double().cpu().numpy().reshape(len(x), -1, HEAD_DIM)
        cs = rotation_table(600).double().numpy()
        pos = plan.positions.cpu().numpy()
        q = kv_ref.norm_rotate(heads[:, :HEADS], blk.q_gamma.double().cpu().numpy(), blk.eps, cs,
                               pos, False)
        q = torch.from_numpy(q).bfloat16().double()
        table = blk.table.cpu().numpy()
        kv = [values(blk.cache, table[r], past[r]) for r in range(3)]
        off = np.concatenate([[0], np.cumsum(q_lens)])
        att, _, spread, reach = kv_ref.attention(q, [a for a, _ in kv], [v for _, v in kv], off,
                                                 past, HEAD_DIM ** -0.5, 0)
        # the o product of the attention's E4M3 codes: a code may differ where
        # the value is near a rounding border (q itself is one bf16 rounding
        # away), so its input is checked and the product recomputed from it
        got, _ = fl.fp8_kv_attention(fl.fp8_qk_norm_rope_append(
            qkv, fl.KvCache(*[t.clone() for t in blk.cache]), plan.positions, plan.slots,
            blk.cos_sin, blk.q_gamma, blk.k_gamma, eps=blk.eps), blk.cache, blk.table,
            plan.q_offsets, plan.kv_lens, max(q_lens), out_dtype=torch.uint8,
            out_scale=blk.out_scale)
        s = blk.out_scale.item()
        # a query one rounding off moves each score by 2^-8 of sum |q_d k_d|
        slack = (spread * (2.0 ** -10 + 2 * 2.0 ** -8 * reach[:, :, None])).numpy() / s
        assert kv_ref.nearest_code_ok(att.numpy() / s, kv_ref.TABLE[host(got)], slack).all()
        want = oracle.scaled_mm_ref(host(got).reshape(len(x), -1), qw_o, np.float32(s), sw_o)
        assert_gemm_close(host(y), want, n)
        blk.commit(plan, int(plan.used[0]))
    assert_status_ok()
    assert fl.fp8l_read_status(fl.fp8_kv_attention_workspace(DEV)) == b.OK


def test_step_equals_its_parts_and_runs_out_of_pages(weights):
    one, two = make(weights), make(weights)
    for n, q_lens in enumerate(([20, 3, 0], [1, 1, 64])):
        x = synthetic.activation(sum(q_lens), 4096, torch.bfloat16, seed=n).to(DEV)
        y = one.step(x, q_lens)
        plan = two.plan(torch.tensor(q_lens, dtype=torch.int32, device=DEV), sum(q_lens))
        assert torch.equal(y, two.forward(x, plan, max(q_lens)))
        two.commit(plan, int(plan.used[0]))
        assert torch.equal(one.kv_lens, two.kv_lens) and torch.equal(one.free, two.free)
    one.free = one.free[:1].contiguous()
    plan = one.plan(torch.tensor([100, 1, 1], dtype=torch.int32, device=DEV), 102)
    assert plan.used.tolist()[1] > 0 and bool((plan.slots == -1).any())


def test_captured_decode_step(weights):
    blk = make(weights)
    x = synthetic.activation(150, 4096, torch.bfloat16, seed=7).to(DEV)
    blk.step(x, [100, 20, 30])
    q_lens = torch.ones(3, dtype=torch.int32, device=DEV)
    xs = synthetic.activation(3, 4096, torch.bfloat16, seed=8).to(DEV)

    def decode():
        plan = blk.plan(q_lens, 3)
        return plan, blk.forward(xs, plan, 1)

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        _, eager = decode()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        plan, y = decode()
    for seed in (9, 10):
        xs.copy_(synthetic.activation(3, 4096, torch.bfloat16, seed=seed).to(DEV))
        saved = [t.clone() for t in blk.cache]
        g.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        for t, s in zip(blk.cache, saved):
            t.copy_(s)
        _, eager = decode()
        assert torch.equal(replayed, eager)
        blk.commit(plan, int(plan.used[0]))


@pytest.mark.parametrize("why", ["pages", "width"])
def test_a_step_whose_tokens_find_no_page_is_refused(weights, why):
    blk, fresh = make(weights), make(weights)
    x = synthetic.activation(23, 4096, torch.bfloat16, seed=1).to(DEV)
    for one in (blk, fresh):
        one.step(x, [20, 3, 0])
    held = blk.free
    if why == "pages":
        blk.free, lens = held[:1].contiguous(), [100, 1, 1]
    else:
        lens = [1, 640, 1]  # 643 tokens, the table's 19 pages hold 608
    before = [t.clone() for t in (*blk.cache, blk.kv_lens, blk.free)]
    with pytest.raises(RuntimeError, match="page"):
        blk.step(synthetic.activation(sum(lens), 4096, torch.bfloat16, seed=2).to(DEV), lens)
    for a, t in zip(before, (*blk.cache, blk.kv_lens, blk.free)):
        assert torch.equal(a, t)
    # with pages again it goes on as if nothing had been tried
    blk.free = held
    x = synthetic.activation(42, 4096, torch.bfloat16, seed=3).to(DEV)
    assert torch.equal(blk.step(x, [40, 1, 1]), fresh.step(x, [40, 1, 1]))
    assert torch.equal(blk.kv_lens, fresh.kv_lens) and torch.equal(blk.free, fresh.free)


def test_the_last_page_of_a_request_is_rotated_by_its_positions(weights):
    # 600 tokens at most are 19 pages of 32: the table takes 608
    blk, wide = make(weights), make(weights)
    wide.cos_sin = rotation_table(608, device=DEV)
    x = synthetic.activation(608, 4096, torch.bfloat16, seed=5).to(DEV)
    assert torch.equal(blk.step(x, [0, 608, 0]), wide.step(x, [0, 608, 0]))
    assert torch.equal(blk.cache.k, wide.cache.k)


def test_a_finished_request_gives_its_pages_back(weights):
    blk, fresh = make(weights), make(weights)
    first = synthetic.activation(230, 4096, torch.bfloat16, seed=1).to(DEV)
    blk.step(first, [130, 0, 100])
    fresh.step(first[130:].contiguous(), [0, 0, 100])
    blk.free = blk.free[:0].contiguous()
    blk.release(0)
    assert blk.free.numel() == 5 and blk.kv_lens.tolist() == [0, 0, 100]
    # another request in its place, on the same pages: five, and no more
    for n, lens in enumerate(([157, 0, 1], [1, 0, 1], [2, 0, 0])):
        x = synthetic.activation(sum(lens), 4096, torch.bfloat16, seed=2 + n).to(DEV)
        assert torch.equal(blk.step(x, lens), fresh.step(x, lens))
    assert blk.free.numel() == 0 and blk.kv_lens.tolist() == [160, 0, 102]
    with pytest.raises(RuntimeError, match="page"):
        blk.step(first[:1], [1, 0, 0])
    blk.release(1)  # a request without tokens has nothing to give
    assert blk.free.numel() == 0


def test_a_step_with_more_tokens_than_rows_is_refused(weights):
    blk = make(weights)
    x = synthetic.activation(12, 4096, torch.bfloat16, seed=1).to(DEV)
    with pytest.raises(ValueError, match="rows"):
        blk.step(x, [10, 3, 0])
    assert blk.kv_lens.tolist() == [0, 0, 0] and blk.free.numel() == 40
    assert blk.step(x, [9, 3, 0]).shape == (12, 4096)
