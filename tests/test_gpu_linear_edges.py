"""GPU parity of the layer products where a kernel's own structure has an edge: the last column tile ends inside a warp
and the epilogue makes several trips, alone and with the K range shared by a cluster.

Reference, tolerances and inputs are those of test_gpu_linear.py.
"""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_linear import _grouped, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


@pytest.mark.parametrize("N", [1, 31, 33, 97, 130, 2079])
@pytest.mark.parametrize("M,K", [(9, 64), (9, 2048), (32, 192), (32, 4096), (63, 128), (63, 1024), (128, 64), (128, 1600)])
def test_last_columns_end_inside_a_warp(gq, M, N, K):
    """Lanes without a column leave the epilogue's branches early; the loads from tensor memory and the cluster's barriers
    that follow are executed by whole warps.  One K range a tile (few column blocks) and a split one."""
    _run(gq, M, N, K, 6, "silu", "f32", "bf16")


def test_last_columns_of_experts_end_inside_a_warp(gq):
    for counts, K in (([20, 0, 32, 11], 64), ([20, 0, 32, 11], 2048), ([100, 70, 0, 120], 128), ([100, 70, 0, 120], 1536)):
        _grouped(gq, counts, 161, K, 8, "relu2", "bf16", "f32", torch.bfloat16, first=1, behind=2)
