"""The low-precision oracle against values fixed by hand, by torch's own casts, by
finite differences, and against planted mistakes."""

import numpy as np
import pytest
import torch

from oracle import formats, lowp


def test_e2m1_rounding_table():
    x = np.array([0.0, 0.25, 0.2500001, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 6.0, 99.0, -0.75, -2.6])
    want = [0, 0, 0.5, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 6, -1, -3]
    assert lowp.round_e2m1(x)[1].tolist() == want


@pytest.mark.parametrize("fmt,top", [("mxfp8", 448.0), ("mxfp4", 6.0)])
def test_power_of_two_scale_is_the_smallest(fmt, top):
    """amax exactly at top * 2^k keeps 2^k; one step above needs 2^(k+1); zero, tiny and
    huge blocks are clamped."""
    for k in (-5, 0, 3):
        for amax, e in ((top * 2.0 ** k, k), (top * 2.0 ** k * (1 + 2.0 ** -8), k + 1),
                        (top * 2.0 ** k * (1 - 2.0 ** -9), k)):
            x = np.zeros((1, 32))
            x[0, 5] = -amax
            assert lowp.quantise(x, fmt)[1][0, 0] == e + 127
    assert lowp.quantise(np.zeros((1, 32)), fmt)[1][0, 0] == 0
    assert lowp.quantise(np.full((1, 32), 2.0 ** -133), fmt)[1][0, 0] == 0
    assert lowp.quantise(np.full((1, 32), 3e38), fmt)[1][0, 0] == (247 if fmt == "mxfp8" else 253)  # 1.763 * 2^127


def test_quantise_against_torch_casts():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(40, 64, generator=g).bfloat16()
    v, s = lowp.quantise(x.double().numpy(), "mxfp8")
    unit = torch.ldexp(torch.ones(40, 2), torch.from_numpy(s.astype(np.int32)) - 127).repeat_interleave(32, 1)
    back = (x.float() / unit).to(torch.float8_e4m3fn).float() * unit
    assert np.array_equal(back.double().numpy(), v)
    v, s = lowp.quantise(x.double().numpy(), "nvfp4", t=float(x.abs().max()) / 2688)
    assert np.abs(v - x.double().numpy()).max() <= float(x.abs().max()) / 6 * 1.1
    assert s.max() == 0x7E                                     # the largest block uses 448


def test_not_finite_blocks_are_nan():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    for fmt in lowp.BLOCK:
        v, _ = lowp.quantise(x, fmt)
        size = lowp.BLOCK[fmt]
        assert np.isnan(v[0, :size]).all() and np.isfinite(v[0, 32:]).all()
        assert np.isnan(v[1, 40 // size * size:(40 // size + 1) * size]).all() and np.isfinite(v[1, :32]).all()


def test_scale_layout_is_a_permutation_and_decodes():
    rows, blocks = 200, 10
    r, b = np.meshgrid(np.arange(256), np.arange(12), indexing="ij")
    at = lowp.scale_offset(r, b, blocks)
    assert sorted(at.ravel().tolist()) == list(range(2 * 3 * 512))
    assert lowp.scale_offset(0, 0, blocks) == 0 and lowp.scale_offset(33, 5, blocks) == 512 + 16 + 4 + 1
    assert lowp.scale_offset(128, 0, blocks) == 3 * 512
    # e2m1 codes: low nibble first, bit 3 the sign
    flat = np.full(512, 127, dtype=np.uint8)
    codes = np.zeros((1, 16), dtype=np.uint8)
    codes[0, 0], codes[0, 1] = 0x7A, 0x01
    assert lowp.decode(codes, flat, 1, 32, "mxfp4")[0, :4].tolist() == [-1.0, 6.0, 0.5, 0.0]


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((3, 11)), rng.standard_normal(11)
    dy, dh = rng.standard_normal((3, 11)), rng.standard_normal((3, 11))
    eps = 1e-3
    h, inv, _ = lowp.rmsnorm(x, w, eps)
    dx, dw = lowp.rmsnorm_bwd(dy, h, w, inv, dh)

    def loss(x, w):
        h, _, y = lowp.rmsnorm(x, w, eps)
        return (y * dy).sum() + (h * dh).sum()

    d = 1e-5
    for idx in [(0, 0), (1, 7), (2, 10)]:
        e = np.zeros_like(x)
        e[idx] = d
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dx[idx]) < 1e-7
    for j in (0, 5):
        e = np.zeros_like(w)
        e[j] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[j]) < 1e-7
    # against autograd
    tx = torch.from_numpy(x).requires_grad_()
    tw = torch.from_numpy(w).requires_grad_()
    y = tx * torch.rsqrt((tx * tx).mean(1, keepdim=True) + eps) * tw
    ((y * torch.from_numpy(dy)).sum() + (tx * torch.from_numpy(dh)).sum()).backward()
    assert np.allclose(tx.grad.numpy(), dx, rtol=1e-12, atol=1e-12)
    assert np.allclose(tw.grad.numpy(), dw, rtol=1e-12, atol=1e-12)


def test_norm_residual_is_rounded_before_the_norm():
    x, r = np.array([[1.0, 2.0 ** -9]]), np.array([[2.0 ** -9, 1.0]])
    h, _, _ = lowp.rmsnorm(x, np.ones(2), 0.0, residual=r, h_fmt=formats.BF16)
    assert h.tolist() == [[1.0, 1.0]]


def test_planted_mistakes_are_seen():
    """A floor instead of a ceiling in the scale, swapped nibbles and a transposed scale
    tile each change a result that the pins above fix."""
    x = np.zeros((1, 32))
    x[0, 0] = 449.0
    v, s = lowp.quantise(x, "mxfp8")
    floor = int(np.floor(np.log2(449.0))) - 8 + 127
    assert s[0, 0] == floor + 1 and v[0, 0] == 448.0
    flat = np.arange(512, dtype=np.uint8)
    got = lowp.scale_bytes(flat, 128, 128, "mxfp8")[0]
    wrong = flat.reshape(128, 4)
    assert got[1].tolist() == flat[16:20].tolist() and got[1].tolist() != wrong[1].tolist()
