"""Host side of the paged FP8 cache entry points and their binding, without a
GPU: no kernel is launched and no address dereferenced."""
import ctypes

import pytest

import fp8_quantized_linear_gb300 as fl
import fp8_quantized_linear_gb300._binding as b


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_linear_gb300 import build
    build.build()
    return fl.load()


def test_capture_id_arguments(lib):
    got = ctypes.c_ulonglong(7)
    assert lib.fp8l_capture_id(None, None) == b.EINVAL
    assert lib.fp8l_capture_id(None, got) == b.OK and got.value == 0


def test_plan_outputs_may_not_share_memory(lib):
    ok = dict(q=0x1000, kv=0x2000, R=4, T=9, page=64, table=0x3000, W=3, free=0x4000, F=5, off=0x5000,
              out=0x6000, pos=0x7000, slots=0x8000, used=0x9000, st=None)
    size = dict(q=4, kv=4, table=12, free=5, off=5, out=4, pos=9, slots=9, used=2)

    def call(**kw):
        return lib.fp8_kv_plan(*dict(ok, **kw).values())
    outputs = ("table", "off", "out", "pos", "slots", "used")
    for o in outputs:
        for other in size:
            if other == o:
                continue
            first, last = ok[other] - 4 * (size[o] - 1), ok[other] + 4 * (size[other] - 1)
            for at in (first, last, ok[other]):
                if (o, other) == ("out", "kv") and at == ok["kv"]:
                    continue  # the lengths in place
                assert call(**{o: at}) == b.EINVAL, (o, other, at)
