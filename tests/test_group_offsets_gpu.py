"""Offsets of grouped rows that break the rules: any 32-bit numbers.  Each is held to [0, total_M] and to
the largest before it, reported, and the call does what it does with offsets that are so; nothing
outside the matrices is read or written."""

import numpy as np
import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TOTAL, N, K = 700, 136, 192
TOP, LOW = 2 ** 31 - 1, -2 ** 31


def _offsets(kind, groups):
    g = np.random.default_rng(groups)
    n = groups + 1
    if kind == "what floats look like":       # differences leave 32 bits
        return g.standard_normal(n).astype(np.float32).view(np.int32).astype(np.int64)
    if kind == "ends of the range":
        return np.where(np.arange(n) % 2 == 0, TOP, LOW)
    if kind == "ends, the other way round":
        return np.where(np.arange(n) % 2 == 0, LOW, TOP)
    if kind == "every second group has all rows":
        return np.where(np.arange(n) % 2 == 0, TOTAL, 0)
    if kind == "behind the rows":
        return np.full(n, TOTAL + 1) + np.arange(n)
    if kind == "before the rows":
        return np.arange(n) - n
    if kind == "falling":
        return np.linspace(TOTAL, 0, n).astype(np.int64)
    if kind == "any":
        return g.integers(LOW, TOP, n)
    cu = np.sort(g.integers(0, TOTAL, n))
    cu[n // 2] = {"one too large": TOTAL + 5, "one negative": -1, "one falls": 0 if n // 2 and cu[n // 2 - 1] else -1}[kind]
    return cu


KINDS = ["what floats look like", "ends of the range", "ends, the other way round", "every second group has all rows",
         "behind the rows", "before the rows", "falling", "any", "one too large", "one negative", "one falls"]


def _check(kind, groups, call):
    """call(cu) -> outputs, each filled before with the same numbers."""
    cu = _offsets(kind, groups)
    held = np.maximum.accumulate(np.clip(cu, 0, TOTAL))
    assert not np.array_equal(cu, held)
    assert gge.gge_read_device_status(DEV)[0] == "GGE_OK"
    got = call(torch.tensor(cu, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    status, where, group = gge.gge_read_device_status(DEV)
    assert status == "GGE_ERR_INDEX_RANGE" and where == 5 and 0 <= group < groups
    want = call(torch.tensor(held, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert gge.gge_read_device_status(DEV)[0] == "GGE_OK"
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def _guarded(dtype, fill):
    return torch.full((TOTAL + 16, N), fill, dtype=dtype, device=DEV)


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device=DEV).manual_seed(1)
    a = torch.randn(TOTAL, K, generator=g, device=DEV).bfloat16()
    b = torch.randn(130, N, K, generator=g, device=DEV).bfloat16()
    pre = torch.randn(TOTAL, N, generator=g, device=DEV)
    return a, b, pre


def _held(x, block):
    q = gge.b128_empty(x.shape[-2], x.shape[-1], block, device=DEV, batch=x.shape[0] if x.dim() == 3 else None)
    gge.gge_b128_quantize(x, q)
    return q


@pytest.mark.parametrize("tile_n", [0, 256, 128, 64])
@pytest.mark.parametrize("groups", [1, 3, 40, 130])
@pytest.mark.parametrize("kind", KINDS)
def test_block_scaled(data, kind, groups, tile_n):
    a, b, pre = data
    A, B, X = _held(a, 1), _held(b[:groups], 128), _held(pre, 1)
    cfg = gge.make_config(tile_n=tile_n) if tile_n else None

    def forward(cu):
        buf = _guarded(torch.bfloat16, 3.0)
        gge.gge_gemm_b128_varlen_m(A, B, cu, D=buf[8:8 + TOTAL], config=cfg)
        return (buf.view(torch.int16),)

    def to_codes(cu):
        scales = torch.full((2, TOTAL + 16), 5.0, device=DEV)
        wide = torch.full((TOTAL + 16, 144), 0x5A, dtype=torch.uint8, device=DEV)
        q = gge.B128Tensor(wide[8:8 + TOTAL, :N].view(torch.float8_e4m3fn), scales[:, 8:8 + TOTAL].t())
        gge.gge_gemm_b128_varlen_m(A, B, cu, PostAct=q, act="silu", config=cfg)
        return wide, scales

    def backward(cu):
        buf = _guarded(torch.float16, 3.0)
        gge.gge_gemm_b128_dact(A, B, X, buf[8:8 + TOTAL], "silu", cu_seqlens_m=cu, config=cfg)
        return (buf.view(torch.int16),)

    for call in (forward, backward) if tile_n == 64 else (forward, to_codes, backward):
        _check(kind, groups, call)


@pytest.mark.parametrize("config", [dict(), dict(cta_group=1, tile_n=128), dict(cta_group=2, tile_n=256), dict(cta_group=2, tile_n=160)])
@pytest.mark.parametrize("groups", [1, 3, 40, 130])
@pytest.mark.parametrize("kind", KINDS)
def test_sixteen_bits(data, kind, groups, config):
    a, b, _ = data
    cfg = gge.make_config(**config) if config else None

    def call(cu):
        buf = _guarded(torch.bfloat16, 3.0)
        gge.gge_gemm_varlen_m(a, b[:groups], cu, D=buf[8:8 + TOTAL], config=cfg)
        return (buf.view(torch.int16),)

    _check(kind, groups, call)


@pytest.mark.parametrize("cta_group", [1, 2])
@pytest.mark.parametrize("groups", [3, 130])
@pytest.mark.parametrize("kind", KINDS)
def test_gathered_rows(data, kind, groups, cta_group):
    a, b, _ = data
    idx = torch.randperm(TOTAL, device=DEV).int()

    def call(cu):
        buf = _guarded(torch.bfloat16, 3.0)
        gge.gge_gemm_gather_a(a, b[:groups], idx, cu, PostAct=buf[8:8 + TOTAL], act="silu",
                              config=gge.make_config(cta_group=cta_group, tile_n=256))
        return (buf.view(torch.int16),)

    _check(kind, groups, call)
