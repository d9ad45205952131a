"""Shared prefixes with offsets that pass what they point into: every range is cut to it, and the results are those of the
cut lists."""
import pytest
import torch

import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
from test_gpu_shared import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


CASES = [
    # prefixes, members, own lengths; then prefix_indptr, group_indptr, kv_indptr as the call gets them
    ([100], [2], [10, 0], [0, 1000], [0, 2], [0, 10, 500]),
    # the second group's prefix begins past the prefixes; the last sequences past the indices
    ([300, 0], [3, 2], [40, 3, 0, 50, 7], [0, 400, 2 ** 30], [0, 3, 5], [0, 40, 43, 43, 200, 2 ** 31 - 1]),
    # a group that reaches past the batch
    ([64, 500], [1, 2], [5, 6, 7], [0, 64, 564], [0, 1, 1000], [0, 5, 11, 18]),
    # nothing of a long prefix but its first 5 tokens is there, and the last sequence has none of its own
    ([5], [40], [1] * 40, [0, 100000], [0, 40], [*range(40), 2 ** 30]),
    # lists longer than their offsets say
    ([200, 50], [2, 2], [9, 9, 9, 9], [0, 150, 190], [0, 2, 4], [0, 9, 18, 20, 25]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_cut_offsets(case, fp8):
    prefixes, members, own, p_at, g_at, k_at = CASES[case]
    args = list(make(prefixes, members, 0, own, fp8, seed=case))
    args[3], args[5], args[6] = i32(p_at), i32(g_at), i32(k_at)
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)  # the oracle cuts the lists in the same places
    cut = list(args)
    for indptr, n in ((3, args[4].numel()), (5, args[0].shape[0]), (6, args[7].numel())):
        cut[indptr] = args[indptr].clamp(max=n)
    same, same_lse = pkg.shared_run(*cut)
    assert torch.equal(out, same) and torch.equal(lse, same_lse)
