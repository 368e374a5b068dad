"""Grouped routing against the FP64 oracle with the comparison of ids kept from running empty: of every case at least
nine rows in ten are decided (no two of their order values or group scores within 2e-6 of each other)."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from test_gpu_route_topk import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


@pytest.mark.parametrize("E,n_group,topk_group,k", [(248, 8, 4, 8), (136, 8, 3, 9), (200, 2, 1, 8), (80, 16, 3, 4),
                                                    (93, 31, 7, 5), (510, 30, 4, 11), (29, 29, 9, 9), (1023, 11, 2, 6),
                                                    (256, 8, 4, 8), (1024, 32, 2, 20), (64, 8, 3, 6)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ids_of_decided_rows(E, n_group, topk_group, k, group_score, score, dtype):
    bias = 0.05 * np.random.default_rng(E).standard_normal(E).astype(np.float32)
    for b in (None, bias):
        check(make(70, E, dtype, seed=k), k, least=0.9, score=score, bias=b, n_group=n_group, topk_group=topk_group,
              group_score=group_score)
