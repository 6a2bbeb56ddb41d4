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
