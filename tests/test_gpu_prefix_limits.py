"""Attention of rows that share a prefix where its arithmetic ends: scales and queries next to nothing."""
import pytest
import torch

import persistent_monokernel_decode_gb300 as kie
from test_gpu_paged import BF16, E4M3, F16, F32
from test_gpu_prefix import check, grouped

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kie.build()
    yield


@pytest.mark.parametrize("cache,qt", [(F16, F32), (E4M3, F32), (E4M3, BF16), (E4M3, F16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-20, 1e-38])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, -1e-38, 1e-30, -1e-6])
def test_scores_of_next_to_nothing(cache, qt, size, scale):
    """Every position weighs the same; rows that end before their prefix does have masked ones among them."""
    q, *rest = grouped([(150, [160, 170, 130, 1]), (64, [64, 63])], [20, 0], 8, 4, 128, 16, cache, qt, seed=4)
    check((q.float() * size).to(qt), *rest, scale=scale)
