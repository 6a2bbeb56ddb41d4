"""ctypes binding of libfp8linear.so: argument marshalling only.

Every function has the name of the C entry point it calls.  Tensors are torch
CUDA tensors (torch supplies device memory and the current stream); E4M3
tensors are uint8 code tensors (a torch.float8_e4m3fn tensor is accepted and
viewed as uint8).  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8linear.so")

ABI_VERSION = 7  # the library version this binding is written for
F16, BF16, E4M3, F32 = 0, 1, 2, 3
WEIGHTS_STABLE = 1
WEIGHTS_PACKED = 2
A_PER_TOKEN = 4
SINGLE_SM_TILES = 8
KERNELS = {"auto": 0, "stream": 16, "swapped": 32, "tiled": 48}  # FP8L_KERNEL_*
FUSED_DYNAMIC_MAX_BYTES = 65536  # FP8L_FUSED_DYNAMIC_MAX_BYTES
OK, EINVAL, ESHAPE, EALIGN, ECUDA, ETIMEOUT, EUNSUPPORTED = range(7)

_DTYPE_CODE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32,
               torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}
_CODE_DTYPE = {F16: torch.float16, BF16: torch.bfloat16, E4M3: torch.uint8}

_lock = threading.Lock()
_lib = None
_workspaces = {}


class Fp8LinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def load():
    """The loaded library (ctypes.CDLL); raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                f"g.build()\"` (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        lib.fp8l_abi_version.restype = I
        lib.fp8l_abi_version.argtypes = []
        version = lib.fp8l_abi_version()
        if version != ABI_VERSION:
            raise RuntimeError(
                f"{LIB_PATH} has ABI version {version}, this binding needs {ABI_VERSION}: "
                f"rebuild it with `python -c \"import __graft_entry__ as g; g.build()\"`")
        # additions that kept the version: their symbols tell
        missing = [name for name in ("fp8_kv_plan", "fp8_qk_norm_rope_append", "fp8_kv_attention",
                                     "fp8l_capture_id", "fp8_linear", "fp8_w8a16_linear",
                                     "fp8_add_rmsnorm_quant") if not hasattr(lib, name)]
        if missing:
            raise RuntimeError(
                f"{LIB_PATH} lacks {', '.join(missing)}: "
                f"rebuild it with `python -c \"import __graft_entry__ as g; g.build()\"`")
        lib.fp8l_workspace_bytes.restype = ctypes.c_size_t
        lib.fp8l_workspace_bytes.argtypes = []
        lib.fp8l_strerror.restype = ctypes.c_char_p
        lib.fp8l_strerror.argtypes = [I]
        lib.fp8l_read_status.restype = I
        lib.fp8l_read_status.argtypes = [P, P]
        lib.fp8l_debug_waits.restype = I
        lib.fp8l_debug_waits.argtypes = [ctypes.c_longlong, ctypes.c_uint]
        lib.fp8_quant_per_tensor.restype = I
        lib.fp8_quant_per_tensor.argtypes = [P, I, I64, I64, P, P, I, P, P]
        lib.fp8_quant_per_row.restype = I
        lib.fp8_quant_per_row.argtypes = [P, I, I64, I64, P, P, P]
        lib.fp8_scaled_mm.restype = I
        lib.fp8_scaled_mm.argtypes = [P, P, I64, I64, I64, P, P, I, P, P, I, P, ctypes.c_uint, P]
        lib.fp8_quant_scaled_mm.restype = I
        lib.fp8_quant_scaled_mm.argtypes = [P, I, P, I64, I64, I64, P, I, P, I, P, P, I, P,
                                            ctypes.c_uint, P]
        lib.fp8_quant_scaled_mm_preferred.restype = I
        lib.fp8_quant_scaled_mm_preferred.argtypes = [I64, I64, I64, I]
        lib.fp8_w8a16_mm_kernel.restype = ctypes.c_uint
        lib.fp8_w8a16_mm_kernel.argtypes = [I64, I64, I64, ctypes.c_uint]
        lib.fp8_scaled_mm_kernel.restype = ctypes.c_uint
        lib.fp8_scaled_mm_kernel.argtypes = [I64, I64, I64, ctypes.c_uint]
        lib.fp8_w8a16_mm.restype = I
        lib.fp8_w8a16_mm.argtypes = [P, I, P, P, I64, I64, I64, P, ctypes.c_uint, P]
        lib.fp8_packed_weight_bytes.restype = ctypes.c_size_t
        lib.fp8_packed_weight_bytes.argtypes = [I64, I64]
        lib.fp8_pack_w8a16_weights.restype = I
        lib.fp8_pack_w8a16_weights.argtypes = [P, I64, I64, P, P]
        lib.fp8_grouped_mm.restype = I
        lib.fp8_grouped_mm.argtypes = [P, P, P, I64, I64, I64, I64, P, P, I, P, P, I, P,
                                       ctypes.c_uint, P]
        lib.fp8_rmsnorm_quant.restype = I
        lib.fp8_rmsnorm_quant.argtypes = [P, I, P, ctypes.c_float, I64, I64, P, P, I, P, P, P]
        U = ctypes.c_uint
        lib.fp8_add_rmsnorm_quant.restype = I
        lib.fp8_add_rmsnorm_quant.argtypes = [P, P, I, P, ctypes.c_float, I64, I64, P, P, P, I, P,
                                              P, P]
        lib.fp8_linear.restype = I
        lib.fp8_linear.argtypes = [P, P, I64, I64, I64, P, P, I, P, I, I, P, P, P, I, P, U, P]
        lib.fp8_w8a16_linear.restype = I
        lib.fp8_w8a16_linear.argtypes = [P, I, P, P, I64, I64, I64, P, I, I, P, P, P, U, P]
        lib.fp8_w8a16_linear_workspace_bytes.restype = ctypes.c_size_t
        lib.fp8_w8a16_linear_workspace_bytes.argtypes = [I, I64, I64, I64, U]
        lib.fp8_kv_plan.restype = I
        lib.fp8_kv_plan.argtypes = [P, P, I64, I64, I64, P, I64, P, I64, P, P, P, P, P, P]
        lib.fp8_qk_norm_rope_append.restype = I
        lib.fp8_qk_norm_rope_append.argtypes = [P, I, I64, I64, I64, I64, I64, P, P,
                                                ctypes.c_float, P, I64, I64, I, P, P, P, P, P, P,
                                                P, I64, I64, P]
        lib.fp8l_capture_id.restype = I
        lib.fp8l_capture_id.argtypes = [P, ctypes.POINTER(ctypes.c_ulonglong)]
        lib.fp8_kv_attention_workspace_bytes.restype = ctypes.c_size_t
        lib.fp8_kv_attention_workspace_bytes.argtypes = []
        lib.fp8_kv_attention_workspace_zero_bytes.restype = ctypes.c_size_t
        lib.fp8_kv_attention_workspace_zero_bytes.argtypes = []
        lib.fp8_kv_attention.restype = I
        lib.fp8_kv_attention.argtypes = [P, I, I64, I64, I64, I64, I64, P, P, P, P, I64, I64, P,
                                         I64, P, P, I64, I64, ctypes.c_float, I64, P, P, I, P, P,
                                         P]
        _lib = lib
        return lib


def strerror(status: int) -> str:
    return load().fp8l_strerror(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise Fp8LinearError(status, where)


def _codes(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not isinstance(t, torch.Tensor) or not t.is_cuda):
            raise TypeError("expected CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("expected contiguous tensors")


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def fp8l_workspace_bytes() -> int:
    return int(load().fp8l_workspace_bytes())


def _device_index(device) -> int:
    """Index of a CUDA device; the current one's when it names none."""
    index = None if device is None else torch.device(device).index
    return torch.cuda.current_device() if index is None else index


def workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for `device`, allocated once and reused."""
    device = torch.device("cuda", _device_index(device))
    ws = _workspaces.get(device)
    if ws is None:
        ws = torch.zeros(fp8l_workspace_bytes(), dtype=torch.uint8, device=device)
        _workspaces[device] = ws
    return ws


def fp8l_read_status(ws: torch.Tensor) -> int:
    lib = load()
    with torch.cuda.device(ws.device):
        st = int(lib.fp8l_read_status(ws.data_ptr(), _stream(ws.device)))
        if st == ETIMEOUT and ws.numel() >= lib.fp8_kv_attention_workspace_bytes():
            # an attention call that gave up may leave its merge counters mid-way
            ws[: lib.fp8_kv_attention_workspace_zero_bytes()].zero_()
    return st


STALL_MMA = 1
STALL_GRID = 2


def fp8l_debug_waits(wait_cycles: int = 0, stall_mask: int = 0) -> None:
    """Testing hook: shorten the device-side wait limit (cycles; 0 = default)
    and make the given waits target a barrier that nothing completes
    (STALL_MMA, STALL_GRID).  Process-wide; fp8l_debug_waits() restores the
    defaults."""
    _check(load().fp8l_debug_waits(int(wait_cycles), int(stall_mask)), "fp8l_debug_waits")


def fp8_quant_per_tensor(x: torch.Tensor, q: torch.Tensor | None = None,
                         scale: torch.Tensor | None = None, dynamic: bool = True,
                         ws: torch.Tensor | None = None):
    """Per-tensor E4M3 quantization of x.  Returns (q uint8, scale float32[1]).
    dynamic=False reads the given `scale` (static input scale)."""
    _need_cuda(x, q, scale, ws)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        if not dynamic:
            raise ValueError("static quantization needs a scale tensor")
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if dynamic and ws is None:
        ws = workspace(x.device)
    rows = x.shape[0] if x.dim() > 1 else 1
    cols = x.numel() // rows if rows else 0
    with torch.cuda.device(x.device):
        st = load().fp8_quant_per_tensor(
            x.data_ptr(), _DTYPE_CODE[x.dtype], rows, cols, _codes(q).data_ptr(),
            scale.data_ptr(), 1 if dynamic else 0, ws.data_ptr() if ws is not None else None,
            _stream(x.device))
    _check(st, "fp8_quant_per_tensor")
    return q, scale


NQ_MODES = {"dynamic": 0, "static": 1, "per_token": 2, "norm_only": 3}


def fp8_rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                      mode: str = "dynamic", q: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None, h: torch.Tensor | None = None,
                      want_h: bool = False, ws: torch.Tensor | None = None):
    """RMSNorm of x [M, K] (fp16/bf16) with gamma [K], fused with its E4M3
    quantization.  mode: "dynamic" (per-tensor scale written), "static"
    (scale given), "per_token" (M scales written) or "norm_only" (h only).
    Returns (q uint8 or None, scale or None, h or None); h is written when
    given, when want_h, or in norm_only mode."""
    _need_cuda(x, gamma, q, scale, h, ws)
    if x.dim() != 2 or gamma.shape != (x.shape[1],) or gamma.dtype != x.dtype:
        raise ValueError("expected x [M, K] and gamma [K] of the same dtype")
    M, K = x.shape
    m = NQ_MODES[mode]
    if (want_h or mode == "norm_only") and h is None:
        h = torch.empty_like(x)
    if mode != "norm_only":
        if q is None:
            q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if scale is None:
            if mode == "static":
                raise ValueError("static mode needs a scale tensor")
            scale = torch.empty(M if mode == "per_token" else 1, dtype=torch.float32,
                                device=x.device)
    if mode == "dynamic" and ws is None:
        ws = workspace(x.device)
    with torch.cuda.device(x.device):
        st = load().fp8_rmsnorm_quant(
            x.data_ptr(), _DTYPE_CODE[x.dtype], gamma.data_ptr(), float(eps), M, K,
            _codes(q).data_ptr() if q is not None else None,
            scale.data_ptr() if scale is not None else None, m,
            h.data_ptr() if h is not None else None,
            ws.data_ptr() if ws is not None else None, _stream(x.device))
    _check(st, "fp8_rmsnorm_quant")
    return q, scale, h


def fp8_quant_per_row(x: torch.Tensor, q: torch.Tensor | None = None,
                      row_scale: torch.Tensor | None = None):
    """One dynamic scale per row of a 2-D tensor.  Returns (q uint8, scales float32[rows])."""
    _need_cuda(x, q, row_scale)
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if row_scale is None:
        row_scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        st = load().fp8_quant_per_row(x.data_ptr(), _DTYPE_CODE[x.dtype], rows, cols,
                                      _codes(q).data_ptr(), row_scale.data_ptr(),
                                      _stream(x.device))
    _check(st, "fp8_quant_per_row")
    return q, row_scale


def scaled_mm_kernel(M: int, N: int, K: int, kernel: str = "auto") -> str:
    """Name ("stream", "swapped" or "tiled") of the kernel fp8_scaled_mm runs
    for this shape and kernel choice (fp8_scaled_mm_kernel; no GPU needed)."""
    code = load().fp8_scaled_mm_kernel(M, N, K, KERNELS[kernel])
    return {v: k for k, v in KERNELS.items()}[code]


def quant_scaled_mm_preferred(M: int, N: int, K: int, dynamic: bool = True) -> bool:
    """Whether fp8_quant_scaled_mm takes this shape and is the faster way to
    run it (fp8_quant_scaled_mm_preferred; no GPU needed)."""
    return bool(load().fp8_quant_scaled_mm_preferred(M, N, K, 1 if dynamic else 0))


def fp8_quant_scaled_mm(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                        a_scale: torch.Tensor | None = None, dynamic: bool = True,
                        out_dtype=torch.bfloat16, out_scale: torch.Tensor | None = None,
                        y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                        stable_weights: bool = False, kernel: str = "auto"):
    """W8A8 product of 16-bit x [M <= 128, K] and E4M3 w [N, K] with the
    per-tensor activation quantization fused into it (fp8_quant_scaled_mm):
    dynamic writes a_scale (a new [1] tensor when None), static reads it.
    kernel: "auto" (the one fp8_scaled_mm would run, tiles excepted),
    "stream" (up to 16 tokens) or "swapped".  Returns (y, a_scale)."""
    _need_cuda(x, w, w_scale, a_scale, out_scale, y, ws)
    w = _codes(w)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("inner dimensions differ")
    if a_scale is None:
        if not dynamic:
            raise ValueError("a static scale must be given")
        a_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if out_dtype == torch.float8_e4m3fn:
        out_dtype = torch.uint8
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = workspace(x.device)
    if w_scale.numel() not in (1, N):
        raise ValueError("w_scale must have 1 or N entries")
    per_channel = 1 if w_scale.numel() == N and N != 1 else 0
    with torch.cuda.device(x.device):
        st = load().fp8_quant_scaled_mm(
            x.data_ptr(), _DTYPE_CODE[x.dtype], w.data_ptr(), M, N, K, a_scale.data_ptr(),
            1 if dynamic else 0, w_scale.data_ptr(), per_channel,
            out_scale.data_ptr() if out_scale is not None else None, _codes(y).data_ptr(),
            _DTYPE_CODE[y.dtype], ws.data_ptr(),
            (WEIGHTS_STABLE if stable_weights else 0) | KERNELS[kernel], _stream(x.device))
    _check(st, "fp8_quant_scaled_mm")
    return y, a_scale


def w8a16_mm_kernel(M: int, N: int, K: int, kernel: str = "auto") -> str:
    """Name ("stream" or "swapped") of the kernel fp8_w8a16_mm runs for this
    shape and kernel choice (fp8_w8a16_mm_kernel; no GPU needed)."""
    code = load().fp8_w8a16_mm_kernel(M, N, K, KERNELS[kernel])
    return {v: k for k, v in KERNELS.items()}[code]


def fp8_scaled_mm(a: torch.Tensor, w: torch.Tensor, a_scale: torch.Tensor,
                  w_scale: torch.Tensor, out_dtype=torch.bfloat16,
                  out_scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stable_weights: bool = False,
                  per_token: bool | None = None, single_sm: bool = False,
                  kernel: str = "auto") -> torch.Tensor:
    """W8A8 product of E4M3 a [M, K] and w [N, K] with a per-tensor ([1]) or
    per-token ([M]) a_scale and a per-tensor ([1]) or per-channel ([N])
    w_scale.  out_dtype bf16 / fp16, or uint8 (E4M3 codes, needs out_scale).
    stable_weights sets FP8L_WEIGHTS_STABLE (no work in flight on the stream
    writes w or w_scale); per_token (default: a_scale has M > 1 entries) sets
    FP8L_A_PER_TOKEN; single_sm sets FP8L_SINGLE_SM_TILES; kernel ("auto",
    "stream", "swapped" or "tiled") sets the FP8L_KERNEL_* choice."""
    _need_cuda(a, w, a_scale, w_scale, out_scale, y, ws)
    a, w = _codes(a), _codes(w)
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("inner dimensions differ")
    if out_dtype == torch.float8_e4m3fn:
        out_dtype = torch.uint8
    code = _DTYPE_CODE[out_dtype]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if ws is None:
        ws = workspace(a.device)
    per_channel = 1 if w_scale.numel() == N and N != 1 else 0
    if w_scale.numel() not in (1, N):
        raise ValueError("w_scale must have 1 or N entries")
    if per_token is None:
        per_token = a_scale.numel() == M and M > 1
    if a_scale.numel() != (M if per_token else 1):
        raise ValueError("a_scale must have 1 entry, or M with per_token")
    flags = ((WEIGHTS_STABLE if stable_weights else 0) | (A_PER_TOKEN if per_token else 0) |
             (SINGLE_SM_TILES if single_sm else 0) | KERNELS[kernel])
    with torch.cuda.device(a.device):
        st = load().fp8_scaled_mm(
            a.data_ptr(), w.data_ptr(), M, N, K, a_scale.data_ptr(), w_scale.data_ptr(),
            per_channel, out_scale.data_ptr() if out_scale is not None else None,
            _codes(y).data_ptr(), code, ws.data_ptr(), flags, _stream(a.device))
    _check(st, "fp8_scaled_mm")
    return y


def fp8_grouped_mm(a: torch.Tensor, w: torch.Tensor, group_offsets: torch.Tensor,
                   a_scale: torch.Tensor, w_scale: torch.Tensor, out_dtype=torch.bfloat16,
                   out_scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, stable_weights: bool = False,
                   per_token: bool | None = None) -> torch.Tensor:
    """Grouped W8A8 product of mixture-of-experts layers: rows
    group_offsets[e] .. group_offsets[e+1]-1 of E4M3 a [M, K] times expert
    e's E4M3 weights w[e] [N, K].  group_offsets: int32 [E + 1] on the
    device; w_scale: [E] (per expert) or [E, N] (per channel); a_scale [1] or
    [M] (per token).  Rows outside the groups of a freshly allocated y are
    zero-filled first; a given y keeps them."""
    _need_cuda(a, w, group_offsets, a_scale, w_scale, out_scale, y, ws)
    a, w = _codes(a), _codes(w)
    M, K = a.shape
    E, N, K2 = w.shape
    if K2 != K or group_offsets.numel() != E + 1 or group_offsets.dtype != torch.int32:
        raise ValueError("shape mismatch")
    per_channel = w_scale.numel() == E * N and N != 1
    if w_scale.numel() not in (E, E * N):
        raise ValueError("w_scale must have E or E * N entries")
    if per_token is None:
        per_token = a_scale.numel() == M and M > 1
    if out_dtype == torch.float8_e4m3fn:
        out_dtype = torch.uint8
    if y is None:
        y = torch.zeros((M, N), dtype=out_dtype, device=a.device)
    if ws is None:
        ws = workspace(a.device)
    flags = (WEIGHTS_STABLE if stable_weights else 0) | (A_PER_TOKEN if per_token else 0)
    with torch.cuda.device(a.device):
        st = load().fp8_grouped_mm(
            a.data_ptr(), w.data_ptr(), group_offsets.data_ptr(), E, M, N, K,
            a_scale.data_ptr(), w_scale.data_ptr(), 1 if per_channel else 0,
            out_scale.data_ptr() if out_scale is not None else None, _codes(y).data_ptr(),
            _DTYPE_CODE[y.dtype], ws.data_ptr(), flags, _stream(a.device))
    _check(st, "fp8_grouped_mm")
    return y


def fp8_packed_weight_bytes(N: int, K: int) -> int:
    """Bytes of the packed layout of [N, K] E4M3 weights (0 for a bad shape)."""
    return int(load().fp8_packed_weight_bytes(N, K))


def fp8_pack_w8a16_weights(w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """The packed copy of E4M3 weight codes w [N, K] that fp8_w8a16_mm reads
    with packed=True: a 1-D uint8 tensor of fp8_packed_weight_bytes(N, K)."""
    _need_cuda(w, out)
    w = _codes(w)
    N, K = w.shape
    nbytes = fp8_packed_weight_bytes(N, K)
    if nbytes == 0:
        _check(ESHAPE, "fp8_pack_w8a16_weights")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
    elif out.dtype != torch.uint8 or out.numel() != nbytes:
        raise ValueError("out must be a uint8 tensor of fp8_packed_weight_bytes(N, K) elements")
    with torch.cuda.device(w.device):
        st = load().fp8_pack_w8a16_weights(w.data_ptr(), N, K, out.data_ptr(), _stream(w.device))
    _check(st, "fp8_pack_w8a16_weights")
    return out


def fp8_w8a16_mm(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                 y: torch.Tensor | None = None, stable_weights: bool = False,
                 packed: bool = False, kernel: str = "auto") -> torch.Tensor:
    """Weight-only product: fp16/bf16 x [M, K] times E4M3 w [N, K] with
    per-channel w_scale [N]; the output has x's dtype.  stable_weights sets
    FP8L_WEIGHTS_STABLE (no work in flight on the stream writes w or
    w_scale).  packed: w is the output of fp8_pack_w8a16_weights (N is
    taken from w_scale) and FP8L_WEIGHTS_PACKED is set.  kernel ("auto",
    "stream" or "swapped") sets the FP8L_KERNEL_* choice."""
    _need_cuda(x, w, w_scale, y)
    w = _codes(w)
    M, K = x.shape
    N = w_scale.numel()
    if packed:
        if w.dtype != torch.uint8 or w.numel() != fp8_packed_weight_bytes(N, K):
            raise ValueError("packed weights must be fp8_pack_w8a16_weights output for [N, K]")
    elif w.dim() != 2 or w.shape[0] != N or w.shape[1] != K:
        raise ValueError("shape mismatch")
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    flags = ((WEIGHTS_STABLE if stable_weights else 0) | (WEIGHTS_PACKED if packed else 0) |
             KERNELS[kernel])
    with torch.cuda.device(x.device):
        st = load().fp8_w8a16_mm(x.data_ptr(), _DTYPE_CODE[x.dtype], w.data_ptr(),
                                 w_scale.data_ptr(), M, N, K, y.data_ptr(), flags,
                                 _stream(x.device))
    _check(st, "fp8_w8a16_mm")
    return y


# The functions of the paged cache run once per layer and step in front of
# kernels of a few microseconds, so their checks are written to cost little:
# one pass of plain attribute tests, the stream's handle without a Stream
# object, no device switch when the device is current already.

KV_PAGE_SIZES = (16, 32, 64, 128)
KV_MIN_SCALE = 2.0 ** -64  # FP8L_KV_MIN_SCALE


class KvCache(NamedTuple):
    """A paged FP8 cache: codes uint8 [num_pages, kv_heads, page_size / 8,
    head_dim / 16, 8, 16] and block scales float32 [num_pages, kv_heads]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @property
    def page_size(self) -> int:
        return self.k.shape[2] * 8

    @property
    def head_dim(self) -> int:
        return self.k.shape[3] * 16

    @property
    def kv_heads(self) -> int:
        return self.k.shape[1]

    @property
    def num_pages(self) -> int:
        return self.k.shape[0]


class KvPlan(NamedTuple):
    """Outputs of fp8_kv_plan (all int32, on the device)."""
    q_offsets: torch.Tensor
    kv_lens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    used: torch.Tensor


def kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, device=None) -> KvCache:
    """A zero-filled paged FP8 cache."""
    if page_size not in KV_PAGE_SIZES or head_dim not in (64, 128):
        raise ValueError("page_size is 16, 32, 64 or 128, head_dim 64 or 128")
    device = torch.device("cuda") if device is None else torch.device(device)
    shape = (num_pages, kv_heads, page_size // 8, head_dim // 16, 8, 16)
    codes = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.full((num_pages, kv_heads), KV_MIN_SCALE, dtype=torch.float32, device=device)
              for _ in range(2)]
    return KvCache(*codes, *scales)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_handle(index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _kv_call(f, index: int, *args) -> int:
    """f(*args, current stream of device `index`) with that device current."""
    with torch.cuda.device(index):
        return f(*args, _stream_handle(index))


def _kv_refuse(index: int, *ts):
    """Says what is wrong with tensors that _kv_placed did not accept."""
    for t in ts:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("expected CUDA tensors")
        if t.get_device() != index:
            raise ValueError("tensors are on different devices")
        if not t.is_contiguous():
            raise ValueError("expected contiguous tensors")


def _kv_placed(index: int, ts) -> bool:
    """Whether the tensors (or None) are contiguous and on device `index`."""
    try:
        for t in ts:
            if t is not None and (t.get_device() != index or not t.is_contiguous()):
                return False
    except AttributeError:
        return False
    return True


def _kv_device(t) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("expected CUDA tensors")
    return t.get_device()


def _kv_cache_shape(cache: KvCache):
    """(num_pages, kv_heads, page_size, head_dim) of a well-formed cache."""
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 6 or shape[4] != 8 or shape[5] != 16 or v.shape != shape or \
            ks.shape != shape[:2] or vs.shape != shape[:2]:
        raise ValueError("cache codes are [num_pages, kv_heads, page_size / 8, head_dim / 16, 8, "
                         "16] and scales [num_pages, kv_heads]")
    if k.dtype is not _U8 or v.dtype is not _U8 or ks.dtype is not _F32 or vs.dtype is not _F32:
        raise ValueError("cache codes are uint8, scales float32")
    return shape[0], shape[1], shape[2] * 8, shape[3] * 16


def _rows(x: torch.Tensor) -> int:
    """Row stride of a token tensor whose rows are dense (any row stride)."""
    want = 1
    for d in range(x.dim() - 1, 0, -1):
        if x.shape[d] > 1 and x.stride(d) != want:
            raise ValueError("expected dense rows (only the row stride may differ)")
        want *= x.shape[d]
    return x.stride(0) if x.shape[0] > 1 else want


def fp8_kv_plan(q_lens: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                free_pages: torch.Tensor, tokens: int, page_size: int,
                plan: KvPlan | None = None) -> KvPlan:
    """Places a step's new tokens in pages (fp8_kv_plan).  q_lens, kv_lens:
    int32 [R], new and cached tokens of each request; block_table: int32 [R,
    W], new entries written in place; free_pages: int32 [F], taken from the
    front; tokens: rows of the step's token tensors.  Returns KvPlan
    (q_offsets [R + 1], kv_lens after the step [R], positions and slots
    [tokens], used [2]: pages taken, tokens without a page, which have to be 0
    for the step to go on to fp8_kv_attention), in `plan`'s tensors when given:
    none may share memory with an input or another, but plan.kv_lens may be
    the kv_lens given."""
    index = _kv_device(q_lens)
    given = (q_lens, kv_lens, block_table, free_pages)
    if not _kv_placed(index, given):
        _kv_refuse(index, *given)
    if q_lens.dtype is not _I32 or kv_lens.dtype is not _I32 or \
            block_table.dtype is not _I32 or free_pages.dtype is not _I32:
        raise ValueError("q_lens, kv_lens, block_table and free_pages must be int32")
    if block_table.dim() != 2:
        raise ValueError("block_table is [requests, table_width]")
    R, W = block_table.shape
    if q_lens.shape != (R,) or kv_lens.shape != (R,):
        raise ValueError("q_lens and kv_lens have one entry per row of block_table")
    tokens = int(tokens)
    if plan is None:
        # one allocation, 4-byte aligned parts
        n = tokens if tokens > 0 else 0
        buf = torch.empty(2 * R + 3 + 2 * n, dtype=_I32, device=q_lens.device)
        plan = KvPlan(*torch.unsafe_split_with_sizes(buf, (R + 1, R, n, n, 2)))
        at = buf.data_ptr()
        ptrs = (at, at + 4 * (R + 1), at + 4 * (2 * R + 1), at + 4 * (2 * R + 1 + n),
                at + 4 * (2 * R + 1 + 2 * n))
    else:
        if not _kv_placed(index, plan):
            _kv_refuse(index, *plan)
        if [t.shape for t in plan] != [(R + 1,), (R,), (tokens,), (tokens,), (2,)] or \
                any(t.dtype is not _I32 for t in plan):
            raise ValueError("plan tensors are int32 [R + 1], [R], [tokens], [tokens], [2]")
        ptrs = tuple(t.data_ptr() for t in plan)
    args = (q_lens.data_ptr(), kv_lens.data_ptr(), R, tokens, page_size, block_table.data_ptr(), W,
            free_pages.data_ptr(), free_pages.numel(), *ptrs)
    f = (_lib or load()).fp8_kv_plan
    st = (f(*args, _stream_handle(index)) if _current_device() == index
          else _kv_call(f, index, *args))
    if st:
        _check(st, "fp8_kv_plan")
    return plan


def fp8_qk_norm_rope_append(qkv: torch.Tensor, cache: KvCache, positions: torch.Tensor,
                            slots: torch.Tensor, cos_sin: torch.Tensor | None = None,
                            q_gamma: torch.Tensor | None = None,
                            k_gamma: torch.Tensor | None = None, eps: float = 1e-6,
                            interleaved: bool = False,
                            q: torch.Tensor | None = None) -> torch.Tensor:
    """Per-head norms of queries and keys, the position rotation, and keys and
    values quantized into the cache (fp8_qk_norm_rope_append).  qkv: [tokens,
    (q_heads + 2 kv_heads) * head_dim], fp16 or bf16, rows at any stride;
    positions, slots: int32 [tokens] (fp8_kv_plan); cos_sin: float32
    [max_positions, rot] or None (no rotation); q_gamma, k_gamma: [head_dim]
    or None (no norm).  Returns q [tokens, q_heads, head_dim]."""
    index = _kv_device(qkv)
    k, v, ks, vs = cache
    given = (k, v, ks, vs, positions, slots, cos_sin, q_gamma, k_gamma, q)
    if not _kv_placed(index, given):
        _kv_refuse(index, *given)
    pages, hkv, page, dim = _kv_cache_shape(cache)
    if qkv.dim() != 2 or qkv.shape[1] % dim != 0:
        raise ValueError("qkv is [tokens, (q_heads + 2 kv_heads) * head_dim]")
    T, width = qkv.shape
    dtype, heads = qkv.dtype, width // dim - 2 * hkv
    if positions.shape != (T,) or slots.shape != (T,) or positions.dtype is not _I32 or \
            slots.dtype is not _I32:
        raise ValueError("positions and slots are int32, one entry per token")
    angles, limit, rot = None, 0, 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype is not _F32:
            raise ValueError("cos_sin is float32 [max_positions, rot]")
        angles, (limit, rot) = cos_sin.data_ptr(), cos_sin.shape
    gammas = [None, None]
    for i, gamma in enumerate((q_gamma, k_gamma)):
        if gamma is not None:
            if gamma.shape != (dim,) or gamma.dtype is not dtype:
                raise ValueError("q_gamma and k_gamma are [head_dim] of qkv's dtype")
            gammas[i] = gamma.data_ptr()
    if q is None:
        q = torch.empty((T, heads if heads > 0 else 0, dim), dtype=dtype, device=qkv.device)
    elif q.shape != (T, heads, dim) or q.dtype is not dtype:
        raise ValueError("q is [tokens, q_heads, head_dim] of qkv's dtype")
    args = (qkv.data_ptr(), _DTYPE_CODE.get(dtype, -1), T,
            width if qkv.is_contiguous() else _rows(qkv), heads, hkv, dim, gammas[0], gammas[1],
            eps, angles, limit, rot, 1 if interleaved else 0, positions.data_ptr(),
            slots.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), ks.data_ptr(),
            vs.data_ptr(), pages, page)
    f = (_lib or load()).fp8_qk_norm_rope_append
    st = (f(*args, _stream_handle(index)) if _current_device() == index
          else _kv_call(f, index, *args))
    if st:
        _check(st, "fp8_qk_norm_rope_append")
    return q


_attention_workspaces = {}  # (device, stream): workspace of its eager calls
_capture_workspaces = {}  # (device, stream): (capture, workspace) of its last capture


def _capture_id(index: int, stream: int) -> int:
    """The stream's capture, 0 when it is not being captured."""
    if not stream:
        return 0  # the legacy default stream cannot be
    got = ctypes.c_ulonglong()
    f = (_lib or load()).fp8l_capture_id
    if _current_device() == index:
        st = f(stream, got)
    else:
        with torch.cuda.device(index):
            st = f(stream, got)
    _check(st, "fp8l_capture_id")
    return got.value


def fp8_kv_attention_workspace(device=None) -> torch.Tensor:
    """A workspace of fp8_kv_attention for the current stream of `device`:
    allocated once per stream and reused (its counters zeroed), so calls on
    different streams do not share one.  A graph capture never takes it: each
    capture gets a workspace of its own for each of its streams, from the
    graph's memory, whose counters every replay zeroes first, so a graph may
    be replayed on any stream and beside eager calls."""
    index = device if isinstance(device, int) else _device_index(device)
    key = (index, _stream_handle(index))
    capture = _capture_id(*key)
    if capture:
        kept, ws = _capture_workspaces.get(key, (0, None))
        if kept == capture:
            return ws
    else:
        ws = _attention_workspaces.get(key)
        if ws is not None:
            return ws
    lib = load()
    ws = torch.empty(lib.fp8_kv_attention_workspace_bytes(), dtype=_U8,
                     device=torch.device("cuda", index))
    ws[: lib.fp8_kv_attention_workspace_zero_bytes()].zero_()
    if capture:
        # held until the stream's next capture: the later calls of this one
        # need it, and the graph's memory outlives the tensor
        _capture_workspaces[key] = (capture, ws)
    else:
        _attention_workspaces[key] = ws
    return ws


def fp8_kv_attention(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor,
                     q_offsets: torch.Tensor, kv_lens: torch.Tensor, max_q_len: int,
                     sm_scale: float | None = None, window: int = 0, out_dtype=None,
                     out_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, want_lse: bool = False,
                     ws: torch.Tensor | None = None):
    """Causal attention of q [tokens, q_heads, head_dim] (rows at any stride)
    over the paged cache (fp8_kv_attention): decode, drafted tokens, prompt
    chunks.  block_table: int32 [R, W]; q_offsets: int32 [R + 1], kv_lens:
    int32 [R] after the step (fp8_kv_plan); max_q_len: host bound of a
    request's new tokens.  sm_scale defaults to head_dim ** -0.5; window > 0
    limits each row to its last `window` keys; out_dtype: q's (default) or
    uint8 (E4M3 codes of out / out_scale).  Returns (out, lse or None)."""
    index = _kv_device(q)
    k, v, ks, vs = cache
    if ws is None:
        ws = fp8_kv_attention_workspace(index)
    elif ws.dtype is not _U8 or ws.numel() < load().fp8_kv_attention_workspace_bytes():
        raise ValueError("ws is a uint8 tensor of fp8_kv_attention_workspace_bytes() elements")
    given = (k, v, ks, vs, block_table, q_offsets, kv_lens, out_scale, out, lse, ws)
    if not _kv_placed(index, given):
        _kv_refuse(index, *given)
    pages, hkv, page, dim = _kv_cache_shape(cache)
    if block_table.dtype is not _I32 or q_offsets.dtype is not _I32 or kv_lens.dtype is not _I32:
        raise ValueError("block_table, q_offsets and kv_lens must be int32")
    shape = q.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError("q is [tokens, q_heads, head_dim]")
    if block_table.dim() != 2:
        raise ValueError("block_table is [requests, table_width]")
    R, W = block_table.shape
    if q_offsets.shape != (R + 1,) or kv_lens.shape != (R,):
        raise ValueError("q_offsets is [requests + 1], kv_lens [requests]")
    if out_dtype is None:
        out_dtype = q.dtype if out is None else out.dtype
    if out_dtype is torch.float8_e4m3fn:
        out_dtype = _U8
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=q.device)
    elif out.shape != shape or _codes(out).dtype is not out_dtype:
        raise ValueError("out is [tokens, q_heads, head_dim] of out_dtype")
    scale_ptr = lse_ptr = None
    if out_scale is not None:
        if out_scale.dtype is not _F32 or out_scale.numel() != 1:
            raise ValueError("out_scale is one float32")
        scale_ptr = out_scale.data_ptr()
    if want_lse and lse is None:
        lse = torch.empty(shape[:2], dtype=_F32, device=q.device)
    if lse is not None:
        if lse.shape != shape[:2] or lse.dtype is not _F32:
            raise ValueError("lse is float32 [tokens, q_heads]")
        lse_ptr = lse.data_ptr()
    args = (q.data_ptr(), _DTYPE_CODE.get(q.dtype, -1), shape[0],
            shape[1] * dim if q.is_contiguous() else _rows(q), shape[1], hkv, dim, k.data_ptr(),
            v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, page, block_table.data_ptr(), W,
            q_offsets.data_ptr(), kv_lens.data_ptr(), R, max_q_len,
            dim ** -0.5 if sm_scale is None else sm_scale, window, scale_ptr, out.data_ptr(),
            _DTYPE_CODE.get(out_dtype, -1), lse_ptr, ws.data_ptr())
    f = (_lib or load()).fp8_kv_attention
    st = (f(*args, _stream_handle(index)) if _current_device() == index
          else _kv_call(f, index, *args))
    if st:
        _check(st, "fp8_kv_attention")
    return out, lse


# fp8l_activation
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# The linear layers stand in front of kernels of a few microseconds too; their
# checks, outputs and calls are C functions of the extension _calls.so
# (csrc/calls.cpp), which the build makes beside the library.
_calls = None


def _load_calls():
    global _calls
    load()  # (refuses a library that is missing or stale)
    path = os.path.join(_PKG, "_calls.so")
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
    spec = importlib.util.spec_from_file_location(f"{__package__}._calls", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.setup(Fp8LinearError)
    _calls = module
    return module


def _choice(table: dict, key, what: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{what} is one of {', '.join(repr(k) for k in table)}") from None


def fp8_linear(a: torch.Tensor, w: torch.Tensor, a_scale: torch.Tensor, w_scale: torch.Tensor,
               bias: torch.Tensor | None = None, activation: str | None = None,
               gated: bool = False, residual: torch.Tensor | None = None, out_dtype=None,
               out_scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, stable_weights: bool = False,
               per_token: bool | None = None, kernel: str = "auto") -> torch.Tensor:
    """The W8A8 linear layer (fp8_linear): fp8_scaled_mm of E4M3 a [M, K] and
    w [N, K] with bias [N] (fp16, bf16 or float32), activation (None, "relu",
    "silu", "gelu", "gelu_tanh") and residual in the epilogue.  gated: w holds
    N / 2 gate rows, then N / 2 up rows, and the result is act(gate) * up, [M,
    N / 2].  residual: [M, N] ([M, N / 2]) of the output's 16-bit type, added
    last; y may be the residual itself.  out_dtype: y's, else the residual's,
    else bf16; uint8 for E4M3 codes of the result / out_scale (no residual
    then).  ws: where a time-out is recorded (None: the library's status word;
    fp8l_read_status reports both).  Scales, stable_weights, per_token and
    kernel as for fp8_scaled_mm."""
    return (_calls or _load_calls()).linear(
        a, w, a_scale, w_scale, bias, _choice(ACTIVATIONS, activation, "activation"), gated,
        residual, out_dtype, out_scale, y, ws,
        _choice(KERNELS, kernel, "kernel") | (WEIGHTS_STABLE if stable_weights else 0), per_token)


def fp8_w8a16_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                     bias: torch.Tensor | None = None, activation: str | None = None,
                     gated: bool = False, residual: torch.Tensor | None = None,
                     y: torch.Tensor | None = None, stable_weights: bool = False,
                     packed: bool = False, kernel: str = "auto") -> torch.Tensor:
    """The W8A16 linear layer (fp8_w8a16_linear): fp8_w8a16_mm of fp16/bf16 x
    [M, K] and E4M3 w [N, K] (per-channel w_scale [N]; packed: the output of
    fp8_pack_w8a16_weights) with bias, activation, gate and residual as in
    fp8_linear; y and residual have x's dtype.  kernel: "auto", "stream" or
    "swapped" (FP8L_KERNEL_*); above 8 tokens (16 with few weights) "auto" holds
    x in E4M3 parts, cut at 2^-21 (bf16) or 2^-25 (fp16) of a row's largest
    magnitude, where "stream" takes it whole (and reads the weights once for
    every 16 tokens)."""
    return (_calls or _load_calls()).w8a16_linear(
        x, w, w_scale, bias, _choice(ACTIVATIONS, activation, "activation"), gated, residual, y,
        _choice(KERNELS, kernel, "kernel") | (WEIGHTS_STABLE if stable_weights else 0) |
        (WEIGHTS_PACKED if packed else 0))


_norm_workspaces = {}  # (device, stream): workspace of its eager calls
_norm_capture_workspaces = {}  # (device, stream): (capture, workspace) of its last capture


def _norm_workspace(index: int) -> torch.Tensor:
    """A workspace of a dynamic fp8_add_rmsnorm_quant for the current stream:
    the words through which the tensor's maximum passes belong to one call at
    a time, so streams do not share one, and a graph capture gets its own from
    the graph's memory, zeroed by every replay (a graph may run beside eager
    calls and other graphs)."""
    key = (index, _stream_handle(index))
    capture = _capture_id(*key)
    if capture:
        kept, ws = _norm_capture_workspaces.get(key, (0, None))
        if kept == capture:
            return ws
    else:
        ws = _norm_workspaces.get(key)
        if ws is not None:
            return ws
    ws = torch.zeros(fp8l_workspace_bytes(), dtype=_U8, device=torch.device("cuda", index))
    if capture:
        _norm_capture_workspaces[key] = (capture, ws)
    else:
        _norm_workspaces[key] = ws
    return ws


def fp8_add_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor,
                          eps: float = 1e-5, mode: str = "dynamic",
                          total: torch.Tensor | None = None, q: torch.Tensor | None = None,
                          scale: torch.Tensor | None = None, h: torch.Tensor | None = None,
                          want_h: bool = False, ws: torch.Tensor | None = None):
    """fp8_rmsnorm_quant of x + residual [M, K] (fp16/bf16), the sum written as
    the new residual stream (fp8_add_rmsnorm_quant).  total: the stream's
    tensor, a new one when None; it may be residual (or x) itself.  gamma, eps,
    mode, q, scale, h and want_h as for fp8_rmsnorm_quant.  Returns (q uint8 or
    None, scale or None, total, h or None).  ws: needed in dynamic mode only; without it one per
    stream and one per graph capture are kept."""
    m = _choice(NQ_MODES, mode, "mode")
    if m == 0 and ws is None:
        ws = _norm_workspace(_kv_device(x))
    return (_calls or _load_calls()).add_rmsnorm_quant(x, residual, gamma, eps, m, total, q, scale,
                                                       h, want_h, ws)
