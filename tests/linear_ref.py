"""Plain 64-bit forms of the linear layers with fused neighbours, and the bounds
their kernels are held to.

A result of value t, computed in float32 with an error of at most d, comes out
between the roundings of t - d and t + d (rounding is monotone), so the tests
ask for exactly that.  d adds up:
  - the product's float32 sum of K terms: at most K 2^-23 of the sum of the
    terms' magnitudes, whatever the order and if every addition truncates;
  - scale products, bias, gate and residual: a rounding of 2^-24 each, 2^-21
    of the magnitudes in all;
  - the activation: a slope of at most 1.13, and its own evaluation, 2^-22
    (16 + |z| + z^2 + |z|^3 / 8) of its value (an exponential's argument is
    rounded, the arguments being |z| for SiLU, 2 x^2 = z^2 for erfc's relative
    slope, up to 1.6 |z| + 0.072 |z|^3 for the tanh form), and 1e-35 where the
    exponential leaves float32's range.
"""
import math

import torch

def e4m3_values(codes):
    """Doubles of codes, by the format's definition."""
    b = torch.arange(256, device=codes.device)
    e, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -x, x)[codes.int()]


def e4m3_round(x):
    """The nearest E4M3 values (ties to even) of doubles, saturated at 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6)
    e = torch.where(a < torch.exp2(e), e - 1, e).clamp(min=-6)
    ulp = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / ulp) * ulp, x)


def act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def parts_error(x):
    """What a 16-bit token may differ by when it is held in E4M3 parts: the
    row's largest magnitude is brought to [2^7, 2^8); a value below E4M3's
    normal range is off by at most half its smallest step, 2^-10, in the first
    part, 2^-14 after the second (bf16), 2^-18 after the third (fp16)."""
    return x.double().abs().amax(1, keepdim=True) * (2.0 ** -21 if x.dtype == torch.bfloat16
                                                     else 2.0 ** -25)


def linear(x, w, scale, bias=None, activation=None, gated=False, residual=None, x_error=0.0):
    """(t, d): the layer in doubles and the error bound.  x [M, K], w [N, K]
    doubles; scale broadcasts to [M, N]; x_error: of every x, by row."""
    K = x.shape[1]
    z = (x @ w.T) * scale
    d = x_error * w.abs().sum(1) * scale.abs() + z.abs() * 2.0 ** -22
    d = d + (x.abs() @ w.abs().T) * scale.abs() * (K * 2.0 ** -23)
    if bias is not None:
        z = z + bias.double()
        d = d + (z.abs() + bias.double().abs()) * 2.0 ** -23
    gate, dg = (z[:, : z.shape[1] // 2], d[:, : z.shape[1] // 2]) if gated else (z, d)
    t = act(activation, gate)
    if activation is None:
        dt = dg
    else:
        g = gate.abs()
        dt = 1.13 * dg + t.abs() * (16 + g + g ** 2 + g ** 3 / 8) * 2.0 ** -22 + 1e-35
    if gated:
        up, du = z[:, z.shape[1] // 2:], d[:, z.shape[1] // 2:]
        dt = dt * up.abs() + t.abs() * du + dt * du + (t * up).abs() * 2.0 ** -22
        t = t * up
    if residual is not None:
        t = t + residual.double()
        dt = dt + (t.abs() + residual.double().abs()) * 2.0 ** -22
    return t, dt


def check16(y, t, d, what=""):
    """y between the roundings of t - d and t + d to its type."""
    lo, hi = (t - d).to(y.dtype), (t + d).to(y.dtype)
    bad = ~((y >= lo) & (y <= hi))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           y[bad][:4].tolist(), t[bad][:4].tolist(), d[bad][:4].tolist())


def check8(codes, t, d, out_scale, what=""):
    y = e4m3_values(codes)
    s = float(out_scale)
    d = d + t.abs() * 2.0 ** -23  # the quotient's own rounding
    lo, hi = e4m3_round((t - d) / s), e4m3_round((t + d) / s)
    bad = ~((y >= lo) & (y <= hi))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           y[bad][:4].tolist(), (t / s)[bad][:4].tolist(), d[bad][:4].tolist())
