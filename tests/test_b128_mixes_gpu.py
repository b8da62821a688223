"""Every mix of a C, a D and a PostAct in 8, 16 and 32 bits, at N that end in each of a block's four
chunks of 32 columns: an 8-bit output's scale goes by the columns that are there.  Tolerances as in
test_b128_gpu.py."""

import pytest
import torch

from grouped_gemm_epilogues_gb300 import binding as gge
from test_b128_gpu import _product

pytestmark = pytest.mark.gpu
C = {"none": None, "bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": "e4m3", "e5m2": "e5m2"}
OUT = [(None, "e4m3"), ("e4m3", "e4m3"), (torch.bfloat16, "e4m3"), ("e4m3", torch.float16), (torch.float32, "e5m2"),
       ("e5m2", torch.float32)]


@pytest.mark.parametrize("n", [8, 40, 72, 104, 128, 136, 264, 480])
@pytest.mark.parametrize("tile_n", [256, 128])
@pytest.mark.parametrize("c", list(C))
def test_mixes(n, tile_n, c):
    for i, (d, p) in enumerate(OUT):
        act = ("gelu_tanh", "silu", "relu", "relu_sq")[i % 4]
        _product(70, n, 200, act=act, c=C[c], d=d, p=p, alpha=0.5, beta=0.0 if c == "none" else 3.0,
                 config=gge.make_config(tile_n=tile_n), seed=n + i)
