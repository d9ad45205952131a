"""The eviction on devices that hold no clusters of 16 thread blocks, or of fewer: the same results."""
import pytest
import torch

import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
from test_gpu_weights import evict_check, listed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _limit(cuda_device):
    build()
    yield
    _lib.gqa_paged_decode_test_cluster_limit(0)


@pytest.mark.parametrize("limit", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("lens,budget,first,last", [([131072, 90000], 16384, 64, 1000), ([40000, 3, 0], 100, 0, 0),
                                                    ([500_000, 3], 200_000, 10, 1000)])
def test_limits(lens, budget, first, last, limit):
    w, indptr, ids = listed(lens, max(lens), 7, "few")
    want = pkg.kv_evict(w, indptr, ids, budget, first, last)
    assert _lib.gqa_paged_decode_test_cluster_limit(limit) == 0
    got = pkg.kv_evict(w, indptr, ids, budget, first, last)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    evict_check((w, indptr, ids, budget, first, last), got)
