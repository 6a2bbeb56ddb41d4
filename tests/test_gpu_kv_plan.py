"""fp8_kv_plan against a loop over requests: block tables, slots, positions,
offsets and lengths are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import kv_ref
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def check(q, kv, page, tokens=None, width=None, free=None, seed=0):
    rng = np.random.default_rng(seed)
    q, kv = np.asarray(q), np.asarray(kv)
    tokens = int(np.maximum(q, 0).sum()) if tokens is None else tokens
    old = -(-np.maximum(kv, 0) // page)
    total = -(-(np.maximum(kv, 0) + np.maximum(q, 0)) // page)
    width = max(1, int(total.max())) if width is None else width
    ids = rng.permutation(int(total.sum()) + 9)
    table = np.full((len(q), width), -1)
    at = 0
    for r in range(len(q)):
        n = min(int(old[r]), width)
        table[r, :n] = ids[at:at + n]
        at += n
    pages = ids[at:] if free is None else ids[at:at + free]
    want = kv_ref.plan(q, kv, table, pages, tokens, page)
    t = i32(table)
    for _ in range(2):  # a repeated call gives the same
        p = fl.fp8_kv_plan(i32(q), i32(kv), t, i32(pages), tokens, page)
        for name in ("q_offsets", "kv_lens", "positions", "slots", "used"):
            assert np.array_equal(getattr(p, name).cpu().numpy(), want[name]), name
        assert np.array_equal(t.cpu().numpy(), want["table"])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R", [1, 2, 63, 513, 1500])
def test_random_lengths(R, page):
    rng = np.random.default_rng(R * page)
    check(rng.integers(0, 40, R), rng.integers(0, 700, R), page, seed=R)


def test_decode_step_and_page_boundaries():
    check(np.ones(130, int), np.arange(130), 16)
    check(np.ones(5, int), [0, 15, 16, 17, 32], 16)


def test_long_prompts():
    check([20001, 0, 3, 9999], [5, 100, 0, 64], 64)


def test_empty_requests_and_negative_lengths():
    check([0, 0, 0], [0, 5, 16], 16)
    check([0, -4, 7, 0], [0, 3, -2, 0], 32)


def test_padded_and_cut_rows():
    check([3, 2], [10, 0], 16, tokens=11)   # rows past the last request
    check([3, 9, 4], [10, 0, 20], 16, tokens=7)  # the last tokens do not fit


def test_pages_run_out():
    check([30, 40, 50], [3, 16, 31], 16, free=4)
    check([30, 40], [3, 16], 16, free=0)


def test_table_width_limits_a_request():
    check([100, 20], [10, 0], 16, width=4)


def test_most_requests():
    rng = np.random.default_rng(5)
    check(rng.integers(0, 3, 8192), rng.integers(0, 50, 8192), 16, seed=2)


@pytest.mark.parametrize("R,most", [(3, 9), (40, 300), (1500, 40)])
def test_a_plan_reused_step_after_step(R, most):
    # the lengths updated in place and all tensors reused; up to 30000 rows
    # (several blocks, if the lengths were not shared)
    rng = np.random.default_rng(R)
    page, width = 16, 200
    table, pages = np.full((R, width), -1), rng.permutation(R * width)
    lens, tokens = np.zeros(R, int), R * most
    dev_table, dev_lens = i32(table), i32(lens)
    plan = None
    for _ in range(4):
        q = rng.integers(0, most + 1, R)
        want = kv_ref.plan(q, lens, table, pages, tokens, page)
        given = None if plan is None else plan._replace(kv_lens=dev_lens)
        plan = fl.fp8_kv_plan(i32(q), dev_lens, dev_table, i32(pages), tokens, page, plan=given)
        for name in ("q_offsets", "kv_lens", "positions", "slots", "used"):
            assert np.array_equal(getattr(plan, name).cpu().numpy(), want[name]), name
        assert np.array_equal(dev_table.cpu().numpy(), want["table"])
        table, lens, pages = want["table"], want["kv_lens"], pages[want["used"][0]:]
        dev_lens = plan.kv_lens


def test_outputs_over_inputs_are_refused():
    q, kv, table, free = i32([3, 2]), i32([4, 5]), i32(np.full((2, 4), -1)), i32(np.arange(9))
    plan = fl.fp8_kv_plan(q, kv, table, free, 5, 16)
    for given in (plan._replace(kv_lens=q), plan._replace(positions=free[:5]),
                  plan._replace(slots=plan.positions), plan._replace(used=kv)):
        with pytest.raises(fl.Fp8LinearError) as e:
            fl.fp8_kv_plan(q, kv, table, free, 5, 16, plan=given)
        assert e.value.status == 1


def test_threads_that_plan_different_numbers_of_requests():
    # both need more shared memory than a launch gets by default
    import threading
    errors = []

    def work(R):
        try:
            rng = np.random.default_rng(R)
            q, kv = rng.integers(0, 3, R), rng.integers(0, 50, R)
            table, pages = np.full((R, 4), 7), np.arange(2 * R)
            want = kv_ref.plan(q, kv, table, pages, 100, 16)
            args = i32(q), i32(kv), i32(table), i32(pages), 100, 16
            with torch.cuda.stream(torch.cuda.Stream(DEV)):
                for _ in range(500):
                    plan = fl.fp8_kv_plan(*args)
                assert np.array_equal(plan.kv_lens.cpu().numpy(), want["kv_lens"])
                assert np.array_equal(plan.slots.cpu().numpy(), want["slots"])
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(R,)) for R in (8192, 4100, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("kv", [2 ** 31 - 1, 2 ** 31 - 60, 2 ** 31 - 200])
@pytest.mark.parametrize("page", [16, 128])
def test_lengths_up_to_32_bits(page, kv):
    t = i32([[3, 3, 3], [7, 7, 7]])
    plan = fl.fp8_kv_plan(i32([0, 5]), i32([kv, 3]), t, i32([4, 5]), 5, page)
    assert plan.kv_lens.tolist() == [kv, 8] and plan.used.tolist() == [0, 0]
    assert plan.slots.tolist() == [7 * page + 3 + i for i in range(5)]
    # new tokens beyond the table have no page
    plan = fl.fp8_kv_plan(i32([0, 5]), i32([3, kv - 200]), t, i32([4, 5]), 5, page)
    full = -(-(kv - 200) // page) * page
    assert plan.kv_lens.tolist() == [3, min(kv - 195, full)]
    assert plan.used.tolist() == [0, max(kv - 195 - full, 0)] and plan.slots.tolist() == [-1] * 5
