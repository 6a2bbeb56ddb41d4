"""Measured cases of a layer's linear operators with their neighbours fused in:
the residual addition with RMSNorm and E4M3 quantization, and the W8A8 and
W8A16 products with bias, activation (gated or not) and residual addition in
the epilogue.

Each case is one call of one operator.  `own` selects between the plain form
(elementary torch operations in 32 bits) and the library's entry point.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# --------------------------------------------------------------------- cases

def listed():
    def norm(name, **kw):
        return dict(name=name, op="norm", **kw)

    def linear(name, **kw):
        return dict(name=name, op="linear", **kw)

    def w8a16(name, **kw):
        return dict(name=name, op="w8a16", **kw)

    return [
        # a decode step of a small batch, one scale per token
        norm("norm_decode_16", M=16, K=4096, mode="per_token", dtype="bf16", h=False),
        # a prompt of odd length, one dynamic scale for all of it; the 16-bit activations are
        # wanted too (for a product that stays in 16 bits)
        norm("norm_prefill_1021", M=1021, K=8192, mode="dynamic", dtype="bf16", h=True),
        # a large prefill batch with calibrated scales
        norm("norm_prefill_16k", M=16384, K=8192, mode="static", dtype="f16", h=False),
        # one token's attention output into the residual stream: latency
        linear("linear_o_1", M=1, N=4096, K=4096, bias=False, act="none", gated=False,
               residual=True, out="bf16", tokens="tensor", channels=True),
        # a decode step's gate and up products, E4M3 straight into the down product
        linear("linear_gate_up_16", M=16, N=28672, K=4096, bias=False, act="silu", gated=True,
               residual=False, out="e4m3", tokens="token", channels=True),
        # a mid-size batch with biases and GELU, a ragged K
        linear("linear_gelu_333", M=333, N=11008, K=4112, bias=True, act="gelu_tanh", gated=False,
               residual=False, out="f16", tokens="tensor", channels=False),
        # a prompt of odd length through the gated half of a feed-forward
        linear("linear_gate_up_1021", M=1021, N=28672, K=4096, bias=False, act="silu", gated=True,
               residual=False, out="e4m3", tokens="tensor", channels=True),
        # the down product of a large prefill batch, added to the residual stream
        linear("linear_down_4096", M=4096, N=8192, K=28672, bias=True, act="none", gated=False,
               residual=True, out="bf16", tokens="token", channels=True),
        # one token with 16-bit activations: gate and up, weights packed at loading
        w8a16("w8a16_gate_up_1", M=1, N=22016, K=4096, bias=False, act="silu", gated=True,
              residual=False, dtype="f16", packed=True),
        # a decode batch's down product into the residual stream
        w8a16("w8a16_down_16", M=16, N=4096, K=11008, bias=False, act="none", gated=False,
              residual=True, dtype="bf16", packed=True),
        # query/key/value with biases, rows as loaded
        w8a16("w8a16_qkv_5", M=5, N=12288, K=4096, bias=True, act="none", gated=False,
              residual=False, dtype="bf16", packed=False),
        # drafted tokens of a batch, biases and GELU
        w8a16("w8a16_gelu_47", M=47, N=11008, K=4096, bias=True, act="gelu", gated=False,
              residual=False, dtype="f16", packed=True),
    ]


_WIDTHS = [256, 512, 4096, 4096, 6144, 8192, 8192, 10240, 11008, 12288, 14336, 22016, 28672]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(step, hi=28672):
        if rng.random() < 0.5:
            return rng.choice([n for n in _WIDTHS if n <= hi])
        return step * log(1, hi // step)

    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "w8a16", "w8a16"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        K = width(16)
        M = log(1, max(1, min(32768, (1 << 27) // K)))
        return dict(op=op, M=M, K=K, mode=rng.choice(["per_token", "dynamic", "static", "norm_only"]),
                    dtype=dtype, h=rng.random() < 0.3)
    gated = rng.random() < 0.4
    act = rng.choice(["relu", "silu", "silu", "gelu", "gelu_tanh"] if gated
                     else ["none", "none", "none", "relu", "silu", "gelu", "gelu_tanh"])
    residual = rng.random() < (0.2 if gated else 0.5)
    bias = rng.random() < 0.4
    N, K = width(32), width(16)
    if op == "w8a16":
        return dict(op=op, M=log(1, 64), N=N, K=K, bias=bias, act=act, gated=gated,
                    residual=residual, dtype=dtype, packed=rng.random() < 0.5)
    M = log(1, 8192)
    M = max(1, min(M, 4096 * 8192 * 28672 // (N * K)))
    out = dtype if residual else rng.choice([dtype, "e4m3"])
    return dict(op=op, M=M, N=N, K=K, bias=bias, act=act, gated=gated, residual=residual, out=out,
                tokens=rng.choice(["tensor", "token"]), channels=rng.random() < 0.8)


# -------------------------------------------------------------------- inputs

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _codes(x, scale):
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _activations(gen, M, K):
    """Normal values, one channel in a hundred eight times as large."""
    size = 1 + 7 * (torch.rand(K, generator=gen, device=DEV) < 0.01)
    return torch.randn(M, K, generator=gen, device=DEV) * size


def _weights(gen, N, K, channels):
    """E4M3 codes and scales (per channel, or one) of normal values."""
    codes = torch.empty((N, K), dtype=torch.uint8, device=DEV)
    scale = torch.empty(N if channels else 1, device=DEV)
    if not channels:
        scale.fill_(0.02 * 6 / 448)
    step = max(1, (1 << 26) // K)
    for n in range(0, N, step):
        w = 0.02 * torch.randn(min(step, N - n), K, generator=gen, device=DEV)
        if channels:
            scale[n:n + step] = w.abs().amax(1) / 448
        codes[n:n + step] = _codes(w, scale[n:n + step, None] if channels else scale)
    return codes, scale


def _packed(w):
    """Weight codes in the order of the packed layout: blocks of 16 rows by 64
    columns, in each the 16-byte pieces of rows 0-7, then of rows 8-15."""
    N, K = w.shape
    chunks = -(-K // 64)
    w = torch.nn.functional.pad(w, (0, chunks * 64 - K))
    return w.view(N // 16, 2, 8, chunks, 4, 16).permute(0, 3, 1, 2, 4, 5).contiguous().view(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, M, K = case, case["M"], case["K"]
    s = dict(case=case, op=case["op"])
    if c["op"] == "norm":
        dtype = _DTYPES[c["dtype"]]
        # the residual stream is larger than what a layer adds to it
        s.update(x=_activations(gen, M, K).to(dtype),
                 residual=(3 * _activations(gen, M, K)).to(dtype),
                 gamma=(1 + 0.2 * torch.randn(K, generator=gen, device=DEV)).to(dtype),
                 scale=torch.full((1,), 20.0 / 448.0, device=DEV))
        return s
    N = c["N"]
    width = N // 2 if c["gated"] else N
    x = _activations(gen, M, K)
    s["w"], s["w_scale"] = _weights(gen, N, K, c["op"] == "w8a16" or c["channels"])
    spread = 0.02 * math.sqrt(K) * 1.28  # of a channel's sums
    out = _DTYPES[c["dtype"]] if c["op"] == "w8a16" else _DTYPES.get(c["out"], torch.bfloat16)
    s["bias"] = (0.5 * torch.randn(N, generator=gen, device=DEV)).to(out) if c["bias"] else None
    s["residual"] = (torch.randn(M, width, generator=gen, device=DEV) * 3).to(out) \
        if c["residual"] else None
    s["out"] = out
    if c["op"] == "w8a16":
        s["x"] = x.to(out)
        s["w_packed"] = _packed(s["w"]) if c["packed"] else None
        return s
    amax = x.abs().amax(1, keepdim=True) if c["tokens"] == "token" else x.abs().max().view(1, 1)
    s["a_scale"] = (amax / 448).view(-1)
    s["a"] = _codes(x, amax / 448)
    peak = 4.5 * spread + (1.0 if c["bias"] else 0.0)
    s["out_scale"] = torch.full((1,), (peak * peak if c["gated"] else peak) / 448, device=DEV)
    return s


# ----------------------------------------------------------------- the calls

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import fp8_quantized_linear_gb300 as fl
    c = s["case"]
    if c["op"] == "norm":
        q, scale, total, h = fl.fp8_add_rmsnorm_quant(
            s["x"], s["residual"], s["gamma"], eps=EPS, mode=c["mode"],
            scale=s["scale"] if c["mode"] == "static" else None, want_h=c["h"])
        return _norm_outputs(c, q, scale, total, h)
    act = None if c["act"] == "none" else c["act"]
    if c["op"] == "w8a16":
        return fl.fp8_w8a16_linear(s["x"], s["w_packed"] if c["packed"] else s["w"], s["w_scale"],
                                   bias=s["bias"], activation=act, gated=c["gated"],
                                   residual=s["residual"], packed=c["packed"], stable_weights=True)
    e4m3 = c["out"] == "e4m3"
    y = fl.fp8_linear(s["a"], s["w"], s["a_scale"], s["w_scale"], bias=s["bias"], activation=act,
                      gated=c["gated"], residual=s["residual"],
                      out_dtype=torch.uint8 if e4m3 else s["out"],
                      out_scale=s["out_scale"] if e4m3 else None,
                      per_token=c["tokens"] == "token", stable_weights=True)
    return y.view(torch.float8_e4m3fn) if e4m3 else y


def _norm_outputs(c, q, scale, total, h):
    res = dict(total=total)
    if c["mode"] != "norm_only":
        res["q"] = q.view(torch.float8_e4m3fn) if q.dtype == torch.uint8 else q
    if c["mode"] in ("dynamic", "per_token"):
        res["scale"] = scale
    if c["h"] or c["mode"] == "norm_only":
        res["h"] = h
    return res


def _plain_norm(s):
    c, dtype = s["case"], s["x"].dtype
    total = (s["x"].float() + s["residual"].float()).to(dtype)
    t = total.float()
    h = (t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["gamma"].float()).to(dtype)
    if c["mode"] == "norm_only":
        return _norm_outputs(c, None, None, total, h)
    f = h.float()
    if c["mode"] == "static":
        scale = s["scale"]
    else:
        scale = (f.abs().amax(1) if c["mode"] == "per_token" else f.abs().max().view(1)) / 448
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = _codes(f, scale[:, None] if c["mode"] == "per_token" else scale)
    return _norm_outputs(c, q, scale, total, h)


def _act_32(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_epilogue(s, z):
    """Bias, activation and residual on the scaled products z [M, N]."""
    c = s["case"]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if c["gated"]:
        gate, up = z.chunk(2, dim=1)
        z = _act_32(c["act"], gate) * up
    else:
        z = _act_32(c["act"], z)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z


def _plain_linear(s):
    c = s["case"]
    a = s["a"].view(torch.float8_e4m3fn).float()
    w = s["w"].view(torch.float8_e4m3fn).float()
    z = _plain_epilogue(s, (a @ w.T) * s["a_scale"][:, None] * s["w_scale"])
    if c["out"] == "e4m3":
        return (z / s["out_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return z.to(s["out"])


def _plain_w8a16(s):
    w = s["w"].view(torch.float8_e4m3fn).float()
    return _plain_epilogue(s, (s["x"].float() @ w.T) * s["w_scale"]).to(s["out"])


_PLAIN = {"norm": _plain_norm, "linear": _plain_linear, "w8a16": _plain_w8a16}


# ------------------------------------------------------------- floors, truth

def work(case):
    c, M, K = case, case["M"], case["K"]
    if c["op"] == "norm":
        codes = c["mode"] != "norm_only"
        h = c["h"] or not codes
        scales = {"per_token": M, "norm_only": 0}.get(c["mode"], 1)
        return {"bytes": M * K * (6 + codes + 2 * h) + 2 * K + 4 * scales, "flops": 8 * M * K}
    N = c["N"]
    width = N // 2 if c["gated"] else N
    if c["op"] == "w8a16":
        token, out, scales = 2 * K, 2, 4 * N
    else:
        token, out = K, 1 if c["out"] == "e4m3" else 2
        scales = 4 * (N if c["channels"] else 1) + 4 * (M if c["tokens"] == "token" else 1)
    return {"bytes": M * token + N * K + M * width * (out + 2 * c["residual"]) + scales
            + 2 * N * c["bias"], "flops": 2 * M * N * K}


def _e4m3_64(x):
    """The nearest E4M3 values (ties to even) of doubles, saturated at 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6)
    e = torch.where(a < torch.exp2(e), e - 1, e).clamp(min=-6)
    ulp = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / ulp) * ulp, x)


def _values_64(codes):
    """Doubles of codes, by the format's definition."""
    b = torch.arange(256, device=DEV)
    e, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -x, x)[codes.int()]


def _exact_norm(s):
    c, dtype, K = s["case"], s["x"].dtype, s["case"]["K"]
    rows, largest = [], 0.0
    step = max(1, (1 << 25) // K)
    for m in range(0, c["M"], step):
        # the stream is held in 16 bits, and the norm is of what is held
        total = (s["x"][m:m + step].double() + s["residual"][m:m + step].double()).to(dtype)
        t = total.double()
        h = t / (t.pow(2).sum(1, keepdim=True) / K + EPS).sqrt() * s["gamma"].double()
        held = h.to(dtype).double()  # and so are the activations that are quantized
        rows.append((total, h if c["h"] or c["mode"] == "norm_only" else None, held.to(dtype)))
        largest = max(largest, held.abs().max().item())
    res = dict(total=torch.cat([r[0] for r in rows]).double())
    if c["h"] or c["mode"] == "norm_only":
        res["h"] = torch.cat([r[1] for r in rows])
    if c["mode"] == "norm_only":
        return res
    held = torch.cat([r[2] for r in rows])
    one = torch.ones((), dtype=torch.float64, device=DEV)
    if c["mode"] == "per_token":
        scale = held.abs().amax(1).double() / 448
        scale = torch.where(scale == 0, one, scale)
    else:
        scale = one.view(1) * ((largest / 448 or 1.0) if c["mode"] == "dynamic"
                               else s["scale"].item())
    q = torch.empty(held.shape, dtype=torch.float32, device=DEV)
    for m in range(0, c["M"], step):
        part = scale[m:m + step, None] if c["mode"] == "per_token" else scale
        q[m:m + step] = _e4m3_64(held[m:m + step].double() / part).float()
    res["q"] = q
    if c["mode"] != "static":
        res["scale"] = scale
    return res


def _act_64(name, z):
    if name == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2u
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3)))
    return z


def _exact_linear(s):
    c, N = s["case"], s["case"]["N"]
    width = N // 2 if c["gated"] else N
    if c["op"] == "w8a16":
        x = s["x"].double()
    else:
        x = _values_64(s["a"]) * s["a_scale"].double()[:, None]
    out = torch.empty((c["M"], width), dtype=torch.float64, device=DEV)
    scale = s["w_scale"].double().expand(N)

    def part(lo, hi):
        z = (x @ _values_64(s["w"][lo:hi]).T) * scale[lo:hi]
        return z if s["bias"] is None else z + s["bias"][lo:hi].double()

    for n in range(0, width, 2048):
        hi = min(width, n + 2048)
        t = _act_64(c["act"], part(n, hi))
        if c["gated"]:
            t = t * part(width + n, width + hi)
        if s["residual"] is not None:
            t = t + s["residual"][:, n:hi].double()
        out[:, n:hi] = t
    if c.get("out") == "e4m3":
        out = _e4m3_64(out / s["out_scale"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_linear(s)
