"""The feed-forward half of a layer as its calls are used together: residual
addition + norm + quantization, gate/up product with its gate, down product
added to the stream, each stage against a 64-bit computation from the stage's
own inputs (bounds as derived in linear_ref and test_gpu_add_norm), eagerly,
captured in a graph, and on another stream."""
import pytest
import torch

import fp8_quantized_linear_gb300 as fl
import linear_ref as ref
from fp8_quantized_linear_gb300.block import HIDDEN, SHAPES
from fp8_quantized_linear_gb300.feed_forward import INNER, FeedForwardBlock
from gpu_util import DEV, assert_status_ok

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def weights():
    gen = torch.Generator(device=DEV).manual_seed(5)
    return {name: (0.02 * torch.randn(*SHAPES[name], generator=gen, device=DEV)).to(BF)
            for name in ("gate_up", "down")}


def inputs(M, seed=1):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, HIDDEN, generator=gen, device=DEV).to(BF)
    stream = (4 * torch.randn(M, HIDDEN, generator=gen, device=DEV)).to(BF)
    return x, stream


def codes_of(block, name, weight):
    return fl.fp8_quant_per_row(weight)[0]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 16, 70, 300])
@pytest.mark.parametrize("kind", ["w8a8", "w8a16"])
def test_stages(weights, kind, M, bias):
    gen = torch.Generator(device=DEV).manual_seed(7)
    biases = {n: torch.randn(SHAPES[n][0], generator=gen, device=DEV).to(BF)
              for n in SHAPES if n in weights} if bias else None
    gamma = (1 + 0.2 * torch.randn(HIDDEN, generator=gen, device=DEV)).to(BF)
    block = FeedForwardBlock(weights, kind, gamma, biases=biases)
    x, stream = inputs(M)
    want = (x.float() + stream.float()).to(BF)
    codes, h = block.norm(x, stream)
    assert torch.equal(stream, want)
    t = want.double()
    h64 = t / (t.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * gamma.double()
    if kind == "w8a8":
        # a code is within half a step (2^-4) of h / scale, h within 2^-8 of h64
        got = ref.e4m3_values(codes) * h.double()[:, None]
        assert ((got - h64).abs() <= h64.abs() * 2.0 ** -3.9 + h.double()[:, None] * 2.0 ** -9).all()
        operand, scale, error = ref.e4m3_values(codes), h.double()[:, None], 0.0
    else:
        ref.check16(h, h64, h64.abs() * 2.0 ** -17)
        operand, scale, error = h.double(), 1.0, ref.parts_error(h)
    inner = block.gate_up(codes, h)
    w = ref.e4m3_values(codes_of(block, "gate_up", weights["gate_up"]))
    b = block.bias.get("gate_up")
    v, d = ref.linear(operand, w, scale * block.sw["gate_up"].double(), b, "silu", True, x_error=error)
    assert inner.shape == (M, INNER)
    if kind == "w8a8":
        ref.check8(inner, v, d, block.gate_scale)
        operand, scale, error = ref.e4m3_values(inner), block.gate_scale.double(), 0.0
    else:
        ref.check16(inner, v, d)
        operand, scale, error = inner.double(), 1.0, ref.parts_error(inner)
    w = ref.e4m3_values(codes_of(block, "down", weights["down"]))
    v, d = ref.linear(operand, w, scale * block.sw["down"].double(), block.bias.get("down"),
                      residual=stream, x_error=error)
    out = block.down(inner, stream)
    assert out is stream
    ref.check16(out, v, d)
    assert_status_ok()


@pytest.mark.parametrize("kind", ["w8a8", "w8a16"])
@pytest.mark.parametrize("M", [1, 24, 200])
def test_graph_and_streams(weights, kind, M):
    """Two layers in a row, captured and replayed, and issued on another stream:
    the eager result, bit for bit."""
    block = FeedForwardBlock(weights, kind)
    x, first = inputs(M)
    eager = first.clone()
    block.forward(x, eager)
    block.forward(x, eager)

    stream = first.clone()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        block.forward(x, stream)
        block.forward(x, stream)
    for _ in range(4):
        stream.copy_(first)
        g.replay()
        assert torch.equal(stream, eager)

    other = first.clone()
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        for _ in range(3):
            other.copy_(first)
            block.forward(x, other)
            block.forward(x, other)
    torch.cuda.current_stream(DEV).wait_stream(side)
    assert torch.equal(other, eager)
    assert_status_ok()


def test_after_the_attention_block(weights):
    """The two halves of a layer over one residual stream: a step of a prompt and
    a decoded token through the paged attention, then the feed-forward."""
    from fp8_quantized_linear_gb300.paged_block import PagedAttentionBlock
    gen = torch.Generator(device=DEV).manual_seed(9)
    half = {name: (0.02 * torch.randn(*SHAPES[name], generator=gen, device=DEV)).to(BF)
            for name in ("qkv", "o")}
    attention = PagedAttentionBlock(half, num_pages=16, requests=2, max_tokens=256)
    block = FeedForwardBlock(weights)
    for q_lens in ([70, 1], [1, 1]):
        _, stream = inputs(sum(q_lens), seed=sum(q_lens))
        before = stream.clone()
        out = attention.step(stream, q_lens)
        result = block.forward(out, stream)
        assert result is stream and torch.isfinite(stream.float()).all()
        # what the layer adds is not nothing, and not out of proportion
        added = (stream.float() - before.float()).abs().mean()
        assert 0.01 < added < 10
    assert_status_ok()


def test_refusals(weights):
    with pytest.raises(ValueError):
        FeedForwardBlock(weights, "w4a8")
    with pytest.raises(ValueError):
        FeedForwardBlock({"gate_up": weights["down"], "down": weights["down"]})
