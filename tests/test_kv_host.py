"""Host side of the paged FP8 cache entry points and their binding, without a
GPU: no kernel is launched and no address dereferenced."""
import contextlib
import ctypes
import subprocess

import pytest
import torch

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


BIG = 2 ** 57  # times 128 wraps around to 0


def test_sizes_whose_products_wrap_around(lib):
    A = 0x10000
    plan = dict(q=A, kv=A, R=4, T=9, page=64, table=A, W=3, free=A, F=5, off=A, out=A, pos=A, slots=A,
                used=A, st=None)
    append = dict(x=A, dt=b.BF16, T=9, ld=48 * 128, hq=32, hkv=8, dim=128, qg=A, kg=A, eps=1e-6,
                  cs=A, mp=100, rot=128, il=0, pos=A, slots=A, q=A, k=A, v=A, ks=A, vs=A, pages=7,
                  page=64, st=None)
    attention = dict(q=A, dt=b.F16, T=9, ld=32 * 128, hq=32, hkv=8, dim=128, k=A, v=A, ks=A, vs=A,
                     pages=7, page=64, table=A, W=3, off=A, kv=A, R=4, n=3, scale=0.1, window=0,
                     os=A, out=A, od=b.F16, lse=None, ws=A, st=None)
    for f, ok, bad in ((lib.fp8_kv_plan, plan, (dict(F=BIG, page=128), dict(F=2 ** 58 + 1),
                                                dict(F=2 ** 62))),
                       (lib.fp8_qk_norm_rope_append, append,
                        (dict(hq=BIG), dict(hq=BIG, hkv=BIG), dict(hq=BIG, hkv=2 ** 56),
                         dict(hq=2 ** 62, hkv=2 ** 61))),
                       (lib.fp8_kv_attention, attention,
                        (dict(hq=BIG), dict(hq=BIG, hkv=BIG), dict(hq=2 ** 62, hkv=2 ** 61),
                         # rows of a tile past the last are numbered too
                         dict(T=2 ** 31 - 1, hq=1, hkv=1, ld=128),
                         dict(T=2 ** 24, hq=128, ld=128 * 128)))):
        for kw in bad:
            assert f(*dict(ok, **kw).values()) == b.ESHAPE, (f.__name__, kw)


class FakeLibrary:
    """The entry points that fp8l_read_status uses, after a time-out."""
    asked = None

    def fp8l_read_status(self, ws, stream):
        return b.ETIMEOUT

    def fp8_kv_attention_workspace_bytes(self):
        return 4096

    def fp8_kv_attention_workspace_zero_bytes(self):
        return 1024


@pytest.mark.parametrize("extra", [0, 16, 5000])
def test_counters_are_zeroed_after_a_time_out_whatever_the_workspace_has_beyond(monkeypatch, extra):
    monkeypatch.setattr(b, "load", lambda: FakeLibrary())
    monkeypatch.setattr(b, "_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    ws = torch.ones(4096 + extra, dtype=torch.uint8)
    assert fl.fp8l_read_status(ws) == b.ETIMEOUT
    assert bool((ws[:1024] == 0).all()) and bool((ws[1024:] == 1).all())
    small = torch.ones(512, dtype=torch.uint8)  # no attention workspace
    assert fl.fp8l_read_status(small) == b.ETIMEOUT and bool((small == 1).all())


@pytest.mark.parametrize("current", [0, 1])
def test_a_device_without_an_index_is_the_current_one(monkeypatch, current):
    def on(index):
        return torch.device("cuda", index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(b, "_stream_handle", lambda index: 0)
    monkeypatch.setattr(b, "_workspaces", {on(i): ("workspace", i) for i in range(3)})
    monkeypatch.setattr(b, "_attention_workspaces", {(i, 0): ("attention", i) for i in range(3)})
    for get, name in ((fl.workspace, "workspace"), (fl.fp8_kv_attention_workspace, "attention")):
        for device in (None, "cuda", torch.device("cuda")):
            assert get(device) == (name, current)
        for device in ("cuda:2", torch.device("cuda", 2)):
            assert get(device) == (name, 2)
        assert get("cuda:0") == (name, 0)


def test_a_stale_library_is_refused_by_name(monkeypatch, tmp_path):
    # right version, but built before the paged cache's entry points
    src, so = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text("int fp8l_abi_version(void) { return %d; }\n" % b.ABI_VERSION)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(b, "LIB_PATH", str(so))
    monkeypatch.setattr(b, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild"):
        b.load()
    assert b._lib is None
