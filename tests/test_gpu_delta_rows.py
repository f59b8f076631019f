"""The gated delta rule on the GPU where the number of state rows decides the
kernel: eight lanes a row on CUDA cores (many rows) against a warp a row (few),
two strips of rows a CTA on the tensor cores against one.  Oracle, tolerances
and their reasons as in test_gpu_delta.py.
"""
import pytest
import torch

from deterministic_mamba2_ssd_gb300.inputs import make_delta_inputs
from test_gpu_delta import _check

pytestmark = pytest.mark.gpu

GENERAL = [
    dict(b=2, T=70, H=16, P=40, G=4, N=72, with_init=True, with_dfinal=True),       # 1280 rows
    dict(b=1, T=69, H=12, P=102, G=2, N=36, with_init=True),                         # 1224
    dict(b=1, T=66, H=16, P=39, G=8, N=24, with_dfinal=True),                        # 624, short dstate
    dict(b=1, T=67, H=8, P=77, G=4, N=200, with_init=True, with_dfinal=True),        # 616, long dstate
    dict(b=1, T=150, H=16, P=40, G=4, N=66, seq_lens=(64, 1, 0, 85), with_init=True, with_dfinal=True),
]
# the same sizes with few rows, around the ends of a block of eight tokens
FEW = [dict(b=1, T=T, H=2, P=5, G=1, N=N, with_init=True, with_dfinal=True) for T in (1, 3, 4, 7, 8, 9, 17)
       for N in (36, 200)]
# 120 CTAs and more have two strips each: with headdim 48 the second is half empty, with 112 the fourth
STRIPS = [
    dict(b=4, T=130, H=32, P=64, G=8, N=64, with_init=True, with_dfinal=True),
    dict(b=8, T=65, H=16, P=48, G=16, N=128, with_dfinal=True),
    dict(b=1, T=400, H=20, P=112, G=5, N=64, seq_lens=(64, 0, 127, 1, 200, 8), with_init=True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", GENERAL, ids=[str(i) for i in range(len(GENERAL))])
def test_many_rows(case, dtype):
    _check(make_delta_inputs(dtype=dtype, seed=case["T"], **case))


@pytest.mark.parametrize("case", FEW, ids=["%d-%d" % (c["T"], c["N"]) for c in FEW])
def test_few_rows(case):
    _check(make_delta_inputs(dtype=torch.float32, seed=case["T"], **case))


@pytest.mark.parametrize("case", STRIPS, ids=[str(i) for i in range(len(STRIPS))])
def test_two_strips(case):
    _check(make_delta_inputs(dtype=torch.bfloat16, seed=case["T"], **case))
