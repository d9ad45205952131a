"""The forms for long and shared contexts at counts where an index of 32 bits would pass its end."""
import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(x, dtype=I32).cuda()


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free memory")


@pytest.mark.parametrize("ahead", [0, 40])
def test_bounds_of_a_block_of_more_than_2_25_tokens(ahead):
    """Token t of a block begins 64 t 16-byte words behind its first: 2^31 of them at t = 2^25. The keys are zeros but for
    one large and one small value on either side, and one behind the length."""
    room(40)
    page = 2 ** 25 + 77
    k = torch.zeros(1, page, 4, 128, dtype=BF, device="cuda")
    k[0, 5, 1, 3], k[0, 6, 1, 4] = 2.0, -3.0
    k[0, 2 ** 25 + 9, 2, 7], k[0, 2 ** 25 + 10, 2, 8] = 5.0, -7.0
    k[0, page - 1, 0, 0] = 1.0
    want = np.zeros((1, 2, 4, 128))
    want[0, 0, 1, 3], want[0, 1, 1, 4], want[0, 0, 2, 7], want[0, 1, 2, 8] = 2, -3, 5, -7
    want[0, 0, 0, 0] = 0 if ahead else 1
    bounds = torch.full((1, 2, 4, 128), 9.0, dtype=BF, device="cuda")
    pkg.block_bounds(k, bounds, i32([[0]]), i32([page - ahead]), i32([page - ahead - 1]))
    assert np.array_equal(cx.f64(bounds), want)
