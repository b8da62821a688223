"""The oracle of 8-bit codes with a scale for each block of 128 and of layer norm, against
values fixed by hand, torch's conversions and torch's autograd."""

import numpy as np
import pytest
import torch

from oracle import b128, formats


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (130, 300), (128, 128)])
def test_quantise_is_torchs_arithmetic(fmt, dtype, block_rows, rows, cols):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    top = b128.TOP[fmt]
    nr, nc = -(-rows // block_rows), -(-cols // 128)
    pad = torch.zeros(nr * block_rows, nc * 128)
    pad[:rows, :cols] = x
    amax = pad.view(nr, block_rows, nc, 128).abs().amax((1, 3))
    scale = (amax * (1.0 / top)).clamp_min(2.0 ** -126)
    up = scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    code = (x * (1.0 / up)).clamp(-top, top).to(dtype)
    got, s = b128.quantise(x.numpy(), fmt, block_rows)
    assert np.array_equal(s, scale.double().numpy())
    assert np.array_equal(got, code.double().numpy() * up.double().numpy())
    bits = code.view(torch.uint8).numpy()
    assert np.array_equal(b128.decode(bits, s, fmt, block_rows), got)


def test_quantise_by_hand():
    x = np.zeros((2, 200))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, 17.0, 18.0     # scale 1: 17 ties to 16, 18 is a code
    x[0, 128] = -896.0                                # the second block's scale is 2
    x[1, 5], x[1, 150] = np.inf, 1e-45
    v, s = b128.quantise(x)
    assert s[0].tolist() == [1.0, 2.0] and np.isnan(s[1, 0]) and s[1, 1] == 2.0 ** -126
    assert v[0, :3].tolist() == [448.0, 16.0, 18.0] and v[0, 128] == -896.0
    assert np.isnan(v[1, :128]).all() and not v[1, 128:].any()
    v, s = b128.quantise(x[:1], block_rows=128)
    assert s.shape == (1, 2) and s[0, 1] == 2.0


def test_off_codes_notices_what_is_off():
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 300)).astype(np.float32).astype(np.float64)
    v, s = b128.quantise(x)
    assert max(b128.off_codes(v, s, x, 0.0)) <= 1.0
    assert b128.off_codes(v * 1.1, s, x, 0.0)[0] > 1.0
    assert b128.off_codes(v, s * 1.01, x, 0.0)[1] > 1.0


def test_layernorm_and_its_backward_are_autograds():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 50, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(50, generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(50, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(6, 50, generator=g, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (50,), w, b, 1e-5)
    y.backward(dy)
    xn, wn = x.detach().numpy(), w.detach().numpy()
    _, mean, rstd, got = b128.layernorm(xn, wn, b.detach().numpy(), 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = b128.layernorm_bwd(dy.numpy(), xn, wn, mean, rstd)
    for a, r in ((dx, x.grad), (dw, w.grad), (db, b.grad)):
        assert np.allclose(a, r.numpy(), rtol=1e-10, atol=1e-12)
    dh = np.ones_like(dx)
    assert np.allclose(b128.layernorm_bwd(dy.numpy(), xn, wn, mean, rstd, dh)[0], dx + 1.0)


def test_layernorm_backward_is_the_difference_quotient():
    g = np.random.default_rng(2)
    x, w, b, dy = (g.standard_normal(s) for s in ((3, 20), 20, 20, (3, 20)))
    _, mean, rstd, _ = b128.layernorm(x, w, b, 1e-5)
    dx = b128.layernorm_bwd(dy, x, w, mean, rstd)[0]
    step = 1e-5
    for r, c in ((0, 0), (1, 7), (2, 19)):
        up, down = x.copy(), x.copy()
        up[r, c] += step
        down[r, c] -= step
        slope = ((b128.layernorm(up, w, b, 1e-5)[3] - b128.layernorm(down, w, b, 1e-5)[3]) * dy).sum() / (2 * step)
        assert abs(slope - dx[r, c]) < 1e-8


def test_layernorm_residual_is_rounded():
    x, r = np.array([[1.0, 2.0]]), np.array([[2.0 ** -9, 0.0]])
    h = b128.layernorm(x, 1.0, 0.0, 1e-5, r, formats.BF16)[0]
    assert h[0].tolist() == [1.0, 2.0]
