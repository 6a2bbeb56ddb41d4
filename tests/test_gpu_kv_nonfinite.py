"""Values that are not finite in the paged FP8 cache: outside the contract, but
never turned into what looks like a result (a row without keys, a page of
ordinary values)."""
import math

import pytest
import torch

import fp8_quantized_linear_gb300 as fl
from gpu_util import DEV
from test_gpu_kv_attention import make, run

pytestmark = pytest.mark.gpu

# rows per kv head 4, 12, 28 (decode kernel) and 240 (prompt kernel); 5000 keys
# are shared by several blocks, whose partials are merged
LENGTHS = [1, 3, 7, 60]


def poisoned(s, spoil):
    """(clean out, spoiled out, spoiled lse) with `spoil` applied to copies."""
    clean, _ = run(s)
    t = dict(s, q=s["q"].clone(), cache=fl.KvCache(*[x.clone() for x in s["cache"]]))
    spoil(t)
    out, lse = run(t, want_lse=True)
    return clean.float(), out.float(), lse


def same_rows(clean, out, lse, rows):
    """Rows that met nothing bad: within the rounding of two computations
    (2^-8 of bf16 outputs and 2^-10 of the largest each)."""
    assert bool(torch.isfinite(lse[rows]).all())
    assert bool(((out - clean)[rows].abs() <= 2.0 ** -6 * clean.abs().max()).all())


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_gives_a_row_of_nan(n, bad):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [5000, 300], seed=31)

    def spoil(t):
        t["q"][n - 1, 5, 17] = bad

    clean, out, lse = poisoned(s, spoil)
    hit = torch.zeros(2 * n, 8, dtype=torch.bool, device=DEV)
    hit[n - 1, 5] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    same_rows(clean, out, lse, ~hit)


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("what", ["k", "k_scale", "v_scale"])
def test_a_key_or_scale_that_is_not_finite_gives_rows_of_nan(n, what):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [5000, 300], seed=32)
    page = int(s["table"][0, 0])

    def spoil(t):
        if what == "k":
            t["cache"].k[page, 1, 0, 2, 3, 5] = 0x7F  # token 3, dimension 37
        else:
            getattr(t["cache"], what)[page, 1] = math.nan

    clean, out, lse = poisoned(s, spoil)
    hit = torch.zeros(2 * n, 8, dtype=torch.bool, device=DEV)
    hit[:n, 4:] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    same_rows(clean, out, lse, ~hit)


@pytest.mark.parametrize("n", LENGTHS)
def test_codes_of_a_row_that_met_a_nan_are_nan(n):
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [5000, 300], seed=34)
    s["q"][0, 6, 0] = math.nan
    scale = torch.full((1,), 0.02, device=DEV)
    out, _ = run(s, out_dtype=torch.uint8, out_scale=scale)
    hit = torch.zeros(2 * n, 8, dtype=torch.bool, device=DEV)
    hit[0, 6] = True
    assert bool(((out[hit] & 0x7F) == 0x7F).all()) and not bool(((out[~hit] & 0x7F) == 0x7F).any())
    # a NaN in one dimension of a value
    s = make(torch.bfloat16, 64, 8, 2, 128, [n, n], [5000, 300], seed=35)
    s["cache"].v[int(s["table"][0, 0]), 0, 0, 4, 2, 1] = 0x7F  # token 2, dimension 65
    for out in (run(s, out_dtype=torch.uint8, out_scale=scale)[0], run(s)[0]):
        nan = (out & 0x7F) == 0x7F if out.dtype == torch.uint8 else out.isnan()
        want = torch.zeros_like(nan)
        want[:n, :4, 65] = True
        assert torch.equal(nan, want)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("count", [1, 2, 40])  # runs of one or two tokens, and longer ones
def test_a_page_that_is_given_a_value_that_is_not_finite_says_so(count, bad):
    page, hkv, dim = 64, 2, 128
    gen = torch.Generator().manual_seed(count)
    x = torch.randn(count, 4 * dim + 2 * hkv * dim, generator=gen).bfloat16().to(DEV)
    x[count - 1, 4 * dim + 3] = bad           # key head 0
    x[0, 4 * dim + (hkv + 1) * dim + 9] = bad  # value head 1
    cache = fl.kv_cache(3, page, hkv, dim, DEV)
    pos = torch.arange(count, dtype=torch.int32, device=DEV)
    slots = pos + 5 + page
    cache.k_scale[1], cache.v_scale[1] = 0.01, 0.01
    fl.fp8_qk_norm_rope_append(x, cache, pos, slots)
    after = fl.fp8_qk_norm_rope_append(torch.ones_like(x[:1]), cache, pos[:1], slots[-1:] + 1)
    assert bool(torch.isfinite(after).all())
    for name, head in (("k_scale", 0), ("v_scale", 1)):
        scale = getattr(cache, name)[1]
        assert not math.isfinite(scale[head].item()) and math.isfinite(scale[1 - head].item())
    # a request that takes the page over starts it anew
    fl.fp8_qk_norm_rope_append(torch.ones_like(x[:1]), cache, pos[:1], pos[:1] + page)
    assert bool(torch.isfinite(cache.k_scale[1]).all()) and bool(torch.isfinite(cache.v_scale[1]).all())
