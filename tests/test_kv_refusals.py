"""Refusals of the paged FP8 cache entry points: argument errors are found on
the host before any CUDA call (fake, never dereferenced addresses), and the
binding refuses tensors it cannot pass on.  No kernel is launched here."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import fp8_quantized_linear_gb300._binding as b

A = 0x10000  # a fake, 16-byte aligned address


@pytest.fixture(scope="module")
def lib():
    from fp8_quantized_linear_gb300 import build
    build.build()
    return fl.load()


def test_plan_argument_errors(lib):
    ok = dict(q=A, kv=A, R=4, T=9, page=64, table=A, W=3, free=A, F=5, off=A, out=A, pos=A, slots=A,
              used=A, st=None)

    def call(**kw):
        return lib.fp8_kv_plan(*dict(ok, **kw).values())
    for page in (0, 8, 48, 256, -16):
        assert call(page=page) == b.ESHAPE
    for kw in (dict(R=0), dict(R=8193), dict(T=-1), dict(T=1 << 31), dict(W=0), dict(F=-1),
               dict(F=1 << 26), dict(W=1 << 31)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("q", "kv", "table", "free", "off", "out", "pos", "slots", "used"):
        assert call(**{name: None}) == b.EINVAL, name
        assert call(**{name: A + 2}) == b.EALIGN, name


def test_append_argument_errors(lib):
    ok = dict(x=A, dt=b.BF16, T=9, ld=48 * 128, hq=32, hkv=8, dim=128, qg=A, kg=A, eps=1e-6, cs=A,
              mp=100, rot=128, il=0, pos=A, slots=A, q=A, k=A, v=A, ks=A, vs=A, pages=7, page=64,
              st=None)

    def call(**kw):
        return lib.fp8_qk_norm_rope_append(*dict(ok, **kw).values())
    for kw in (dict(dt=b.F32), dict(dt=b.E4M3), dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf"))):
        assert call(**kw) == b.EINVAL, kw
    for kw in (dict(T=-1), dict(T=1 << 31), dict(ld=48 * 128 - 8), dict(ld=48 * 128 + 4), dict(hq=30),
               dict(hq=4), dict(hkv=0), dict(dim=96), dict(dim=256), dict(rot=136), dict(rot=24),
               dict(rot=-16), dict(mp=0), dict(pages=0), dict(pages=1 << 25), dict(page=24),
               dict(hq=1 << 14, hkv=1 << 13, ld=1 << 30)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("x", "cs", "pos", "slots", "q", "k", "v", "ks", "vs"):
        assert call(**{name: None}) == b.EINVAL, name
    for name in ("x", "cs", "q", "k", "v", "qg", "kg"):
        assert call(**{name: A + 8}) == b.EALIGN, name
    for name in ("ks", "vs", "pos", "slots"):
        assert call(**{name: A + 1}) == b.EALIGN, name


def test_attention_argument_errors(lib):
    ok = dict(q=A, dt=b.F16, T=9, ld=32 * 128, hq=32, hkv=8, dim=128, k=A, v=A, ks=A, vs=A, pages=7,
              page=64, table=A, W=3, off=A, kv=A, R=4, n=3, scale=0.1, window=0, os=A, out=A,
              od=b.F16, lse=None, ws=A, st=None)

    def call(**kw):
        return lib.fp8_kv_attention(*dict(ok, **kw).values())
    for kw in (dict(dt=b.F32), dict(od=b.BF16), dict(od=b.F32), dict(od=7), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(od=b.E4M3, os=None)):
        assert call(**kw) == b.EINVAL, kw
    for kw in (dict(T=-1), dict(ld=32 * 128 - 8), dict(ld=32 * 128 + 4), dict(hq=20), dict(hkv=0),
               dict(dim=80), dict(pages=0), dict(pages=1 << 25), dict(page=12), dict(W=0), dict(R=0),
               dict(R=8193), dict(n=-1), dict(window=-1)):
        assert call(**kw) == b.ESHAPE, kw
    for name in ("q", "k", "v", "ks", "vs", "table", "off", "kv", "out", "ws"):
        assert call(**{name: None}) == b.EINVAL, name
    for name in ("q", "k", "v", "out", "ws"):
        assert call(**{name: A + 8}) == b.EALIGN, name
    for name in ("ks", "vs", "table", "off", "kv", "os", "lse"):
        assert call(**{name: A + 2}) == b.EALIGN, name


def test_workspace_sizes(lib):
    size, zero = (lib.fp8_kv_attention_workspace_bytes(),
                  lib.fp8_kv_attention_workspace_zero_bytes())
    assert 32 <= zero <= size and size % 16 == 0


def test_cpu_tensors_and_bad_caches_are_refused():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        fl.fp8_kv_plan(i, i, i.view(4, 1), i, 4, 16)
    cache = fl.kv_cache(3, 16, 2, 64, device="cpu")
    assert (cache.page_size, cache.head_dim, cache.kv_heads, cache.num_pages) == (16, 64, 2, 3)
    with pytest.raises(TypeError, match="CUDA"):
        fl.fp8_qk_norm_rope_append(torch.zeros(4, 6 * 64).half(), cache, i, i)
    with pytest.raises(TypeError, match="CUDA"):
        fl.fp8_kv_attention(torch.zeros(4, 2, 64).half(), cache, i.view(4, 1), i, i, 1)
    for bad in (dict(page_size=24), dict(head_dim=96)):
        with pytest.raises(ValueError):
            fl.kv_cache(**dict(dict(num_pages=3, page_size=16, kv_heads=2, head_dim=64, device="cpu"),
                               **bad))


@pytest.mark.gpu
def test_shapes_and_types_are_checked():
    dev = torch.device("cuda:0")
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    cache = fl.kv_cache(3, 16, 2, 64, device=dev)
    q = torch.zeros(4, 2, 64, dtype=torch.half, device=dev)
    x = torch.zeros(4, 6 * 64, dtype=torch.half, device=dev)
    off, table = torch.zeros(5, dtype=torch.int32, device=dev), i.view(4, 1)
    with pytest.raises(ValueError, match="int32"):
        fl.fp8_kv_plan(i.long(), i, table, i, 4, 16)
    with pytest.raises(ValueError):
        fl.fp8_kv_plan(i[:3], i, table, i, 4, 16)
    with pytest.raises(fl.Fp8LinearError):
        fl.fp8_kv_plan(i, i, table, i, 4, 24)
    for bad in (lambda: fl.fp8_qk_norm_rope_append(x, cache, i[:3], i),
                lambda: fl.fp8_qk_norm_rope_append(x[:, :-1], cache, i, i),
                lambda: fl.fp8_qk_norm_rope_append(x, cache, i, i, q_gamma=x[0, :64].float()),
                lambda: fl.fp8_qk_norm_rope_append(x.t(), cache, i, i),
                lambda: fl.fp8_qk_norm_rope_append(x, cache, i, i, q=q[:2]),
                lambda: fl.fp8_qk_norm_rope_append(x, cache._replace(v=cache.v[:2]), i, i),
                lambda: fl.fp8_kv_attention(q, cache, table, off[:4], i, 1),
                lambda: fl.fp8_kv_attention(q[:, :, :32], cache, table, off, i, 1),
                lambda: fl.fp8_kv_attention(q, cache, table.float(), off, i, 1),
                lambda: fl.fp8_kv_attention(q, cache, table, off, i, 1, out=q[:3]),
                lambda: fl.fp8_kv_attention(q.transpose(1, 2).contiguous().transpose(1, 2), cache,
                                            table, off, i, 1)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fl.fp8_qk_norm_rope_append(x.float(), cache, i, i),
                lambda: fl.fp8_kv_attention(q.float(), cache, table, off, i, 1),
                lambda: fl.fp8_kv_attention(q, cache, table, off, i, 1, out_dtype=torch.bfloat16),
                lambda: fl.fp8_kv_attention(q, cache, table, off, i, 1, out_dtype=torch.uint8),
                lambda: fl.fp8_kv_attention(q, cache, table, off, i, 1, sm_scale=0.0)):
        with pytest.raises(fl.Fp8LinearError):
            bad()
