"""The operators on 8 bits with block scales together, as a training step runs them: layer norm,
products with 8-bit outputs, the activation's backward, checkpoints turned in 8 bits, weight
gradients added to in place, the norm's backward; eagerly, for one token, and captured.

The limit.  An e4m3 code keeps 3 bits: a normal one is off by at most 2^-4 of its value, in the mean
square by 2^-4 / sqrt(3) or less (0.036; with the values spread over an octave 0.026).  y is behind
four such roundings of its factors (n, W1, a, W2), a gradient behind up to six (dy, W2, u, du, W1 and
the norm's h, or their transposes'), independent and of zero mean: 0.026 sqrt(6) = 0.064; the
values near a block's smallest codes add to that.  0.09 is under half of what one factor left out,
or one scale taken of a neighbouring block, changes (0.2 and more).
"""

import os
import sys

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,width,hidden", [(300, 512, 1000), (257, 1000, 520), (40, 128, 256)])
def test_training_step_and_one_token(tokens, width, hidden):
    import block_scaled_mlp
    errors = block_scaled_mlp.run(tokens, width, hidden)
    assert all(e < 0.09 for e in errors.values()), errors
    assert errors["y"] > 1e-3      # (it does compute in 8 bits)
    assert errors["one token"] < 1e-2


def test_captured_step_repeats_and_gradients_add_up():
    """The same step from a graph, twice: outputs bit for bit those of an eager step, and the
    weight gradients twice theirs, rounded after each addition."""
    import block_scaled_mlp
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(5)
    x, r, dy, dh = (torch.randn(200, 512, generator=g, device=dev).bfloat16() for _ in range(4))

    def step(block):
        y, h, saved = block.forward(x, r, keep=True)
        return (y, h, *block.backward(dy, dh, saved))

    eager = block_scaled_mlp.Block(512, 640, dev)
    want = step(eager)
    once = eager.dw1.clone(), eager.dw2.clone()
    step(eager)
    block = block_scaled_mlp.Block(512, 640, dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(block)                      # (first calls outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(block)
    block.dw1.zero_()
    block.dw2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(block.dw1, once[0]) and torch.equal(block.dw2, once[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(block.dw1, eager.dw1) and torch.equal(block.dw2, eager.dw2)
    assert gge.gge_read_device_status(dev)[0] == "GGE_OK"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k,tile", [(300, 264, 700, 256), (300, 264, 700, 128), (130, 72, 4000, 64), (16, 512, 2048, 0)])
def test_sum_in_place_is_the_sum(m, n, k, tile, dtype):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(m + n)
    qa, qb = (block_scaled_quantised(torch.randn(rows, k, generator=g, device=dev), block) for rows, block in ((m, 1), (n, 1)))
    c = torch.randn(m, n, generator=g, device=dev).to(dtype)
    cfg = gge.make_config(tile_n=tile) if tile else None
    want = torch.empty_like(c)
    gge.gge_gemm_b128(qa, qb, D=want, C=c, alpha=0.5, beta=2.0, config=cfg)
    gge.gge_gemm_b128(qa, qb, D=c, C=c, alpha=0.5, beta=2.0, config=cfg)
    assert torch.equal(c, want)


def block_scaled_quantised(x, block):
    q = gge.b128_empty(x.shape[0], x.shape[1], block, device=x.device)
    gge.gge_b128_quantize(x, q)
    return q


# Sizes past 2^31 places: the last rows of a tall matrix, which a 32-bit offset would miss.

def test_tall_matrices_pass_32_bits():
    dev = torch.device("cuda", torch.cuda.current_device())
    rows, cols, n = 1_050_003, 2080, 136            # 2.18e9 codes
    gen = torch.Generator(device=dev).manual_seed(3)
    tail = torch.randn(300, cols, generator=gen, device=dev).bfloat16()
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=dev)
    x[-300:] = tail
    q = block_scaled_quantised(x, 1)
    few = block_scaled_quantised(tail, 1)
    assert torch.equal(q.codes[-300:].view(torch.uint8), few.codes.view(torch.uint8))
    assert torch.equal(q.scales[-300:], few.scales)
    back = torch.empty_like(x)
    gge.gge_b128_dequantize(q, back)
    back_few = torch.empty_like(tail)
    gge.gge_b128_dequantize(few, back_few)
    assert torch.equal(back[-300:], back_few) and not back[:-300].any()
    w = block_scaled_quantised(torch.randn(n, cols, generator=gen, device=dev), 128)
    d, d_few = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=dev), torch.empty(300, n, dtype=torch.bfloat16, device=dev)
    # (the same tiles, K unsplit: the few rows alone would be split along K, and their sums, joined
    # in another order, may differ in the last bit)
    cfg = gge.make_config(tile_n=128, flags=32)
    gge.gge_gemm_b128(q, w, D=d, config=cfg)
    gge.gge_gemm_b128(few, w, D=d_few, config=cfg)
    assert torch.equal(d[-300:], d_few) and not d[:-300].any()
    # the norm, its 8-bit output and its backward over the same rows
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    y8 = gge.b128_empty(rows, cols, device=dev)
    gge.gge_layernorm(x, None, None, Y=back, Q=y8, mean=mean, rstd=rstd)
    m2, r2, y2, few8 = mean[:300].clone(), rstd[:300].clone(), torch.empty_like(tail), gge.b128_empty(300, cols, device=dev)
    gge.gge_layernorm(tail, None, None, Y=y2, Q=few8, mean=m2, rstd=r2)
    assert torch.equal(back[-300:], y2) and torch.equal(mean[-300:], m2) and torch.equal(rstd[-300:], r2)
    assert torch.equal(y8.codes[-300:].view(torch.uint8), few8.codes.view(torch.uint8))
    dx, dx2 = torch.empty_like(x), torch.empty_like(tail)
    gge.gge_layernorm_bwd(back, q, None, mean, rstd, dx)
    gge.gge_layernorm_bwd(y2, few, None, m2, r2, dx2)
    assert torch.equal(dx[-300:], dx2)
    # and turned: the last 300 columns of a row that spans the tall matrix
    t = gge.b128_empty(cols, rows, device=dev)
    gge.gge_b128_transpose(q, t)
    values = torch.empty(cols, rows, dtype=torch.bfloat16, device=dev)
    gge.gge_b128_dequantize(t, values)
    first = (rows - 300) // 128 * 128          # (whole blocks of the turned rows)
    numbers = torch.empty(300, cols, device=dev)   # (fp32: what the codes stand for, exactly)
    gge.gge_b128_dequantize(few, numbers)
    part = torch.zeros(rows - first, cols, device=dev)
    part[-300:] = numbers
    again = block_scaled_quantised(part.t(), 1)
    want = torch.empty(cols, rows - first, dtype=torch.bfloat16, device=dev)
    gge.gge_b128_dequantize(again, want)
    assert torch.equal(values[:, first:], want)
    assert gge.gge_read_device_status(dev)[0] == "GGE_OK"
