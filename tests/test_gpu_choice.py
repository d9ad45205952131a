"""The choice of blocks where scores leave fp32's range on the way or at the end, and among many equal ones."""
import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
from test_gpu_blocks import chosen, make, select

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOP = 2.0 ** 128 - 2.0 ** 120  # bf16's largest


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def rows_of_values(values, blocks):
    """Bounds whose scores for a query of ones are the sums of `values[i]` in block i, and of nothing in the others."""
    b = torch.zeros(blocks, 2, 4, 128)
    for i, x in enumerate(values):
        b[i, :, :, :len(x)] = torch.tensor(x)
    return b.to(BF)


BIG = 3 * 2.0 ** 126
SUMS = [
    [BIG, BIG, -BIG, -BIG],                      # 0, by way of 3 * 2^127
    [-BIG, -BIG, -BIG, BIG, BIG, BIG, 2.0 ** 100],  # 2^100
    [2.0 ** 101], [2.0 ** 99], [-2.0 ** 90], [1.0],
    [BIG, -BIG] * 30 + [2.0 ** 102],
    [TOP, 2.0 ** 120 - 2.0 ** 112, 2.0 ** 112 - 2.0 ** 104],                # fp32's largest
    [TOP, 2.0 ** 120 - 2.0 ** 112, 2.0 ** 112 - 2.0 ** 104, 2.0 ** 102],    # rounds to it
    [-TOP, -TOP, TOP, -2.0 ** 110],
]
OVER = [[TOP, 2.0 ** 120 - 2.0 ** 112, 2.0 ** 112 - 2.0 ** 104, 2.0 ** 103],  # half a step past it: rounds to infinity
        [BIG, BIG], [-BIG, -BIG], [TOP] * 128, [float("inf")], [float("-inf")], [float("inf"), float("-inf")]]


def order(w, values):
    """The table's blocks in an order of their own, the values' in front of the pool."""
    blocks = w["k"].shape[0]
    w["bounds"].copy_(rows_of_values(values, blocks))
    g = torch.Generator().manual_seed(len(values))
    w["table"][0, :blocks] = torch.randperm(blocks, generator=g).to(torch.int32).cuda()[:w["table"].shape[1]]


@pytest.mark.parametrize("top", list(range(1, 19)))
@pytest.mark.parametrize("over", [False, True])
def test_sums_that_leave_the_range_on_the_way(top, over):
    values = SUMS + (OVER if over else [])
    w = make([8 * 40], 8, 1, spare=1)
    order(w, values)
    w["q"].fill_(1.0)
    got = select(w, top, 0, 0)
    assert np.array_equal(got.cpu().numpy(), chosen(w, top, 0, 0))


def test_the_rank_of_each_sum():
    """By hand: block 0's score of 0 stays behind 1 and 2^99; blocks past the range come before all."""
    w = make([8 * 4], 8, 1, spare=0)
    w["table"][0, :4] = torch.arange(4, dtype=torch.int32)
    w["q"].fill_(1.0)
    w["bounds"].copy_(rows_of_values([SUMS[0], [1.0], [2.0 ** 99], [BIG, BIG]], 4))
    assert select(w, 1, 0, 0)[0].tolist() == [[3]] * 4
    assert select(w, 2, 0, 0)[0].tolist() == [[2, 3]] * 4
    assert select(w, 3, 0, 0)[0].tolist() == [[1, 2, 3]] * 4


def test_heads_past_the_range():
    """The largest of the 8 heads decides: one far below the range does not lift a block whose best head is small."""
    w = make([8 * 5], 8, 1, spare=0)
    w["table"][0, :5] = torch.arange(5, dtype=torch.int32)
    w["q"].zero_()
    w["q"][0, 0::8, 0] = 1.0     # head 0 of each KV head: dim 0; the others: dim 1
    w["q"][0, 0::8, 2] = 1.0
    for h in range(1, 8):
        w["q"][0, h::8, 1] = 1.0
    b = torch.zeros(5, 2, 4, 128)
    b[0, ..., 0], b[0, ..., 2], b[0, ..., 1] = -BIG, -BIG, 5.0   # head 0: past the range, below; the others 5
    b[1, ..., 0], b[1, ..., 1] = 7.0, 1.0
    b[2, ..., 0], b[2, ..., 1] = 3.0, 2.0
    b[3, ..., 0], b[3, ..., 2], b[3, ..., 1] = BIG, BIG, -9.0    # head 0: past the range, above
    b[4, ..., 0], b[4, ..., 1] = 6.0, 6.0
    w["bounds"].copy_(b.to(BF))
    for top, want in ((1, [3]), (2, [1, 3]), (3, [1, 3, 4]), (4, [0, 1, 3, 4])):
        assert select(w, top, 0, 0)[0].tolist() == [want] * 4
        assert np.array_equal(select(w, top, 0, 0).cpu().numpy(), chosen(w, top, 0, 0))


@pytest.mark.parametrize("scale", [2.0 ** 60, 2.0 ** 63, 2.0 ** 66, 2.0 ** 100])
def test_random_scores_about_the_range(scale):
    """Queries and bounds whose products pass the range now and then; integers, so that 64 bits hold every sum."""
    w = make([8 * 300], 8, 2, spare=0)
    g = torch.Generator().manual_seed(5)
    w["q"].copy_((torch.randint(-3, 4, w["q"].shape, generator=g) * scale).to(BF))
    w["bounds"].copy_((torch.randint(-3, 4, w["bounds"].shape, generator=g) * 2.0 ** 60).to(BF))
    for top in (1, 10, 100, 299):
        assert np.array_equal(select(w, top, 0, 0).cpu().numpy(), chosen(w, top, 0, 0)), top


@pytest.mark.parametrize("blocks", [1500, 49153, 60000])
@pytest.mark.parametrize("kind", ["same", "two", "cancel"])
def test_many_undecided_blocks(blocks, kind):
    """More equal or nearly equal scores than are compared one with another, by the large block of threads, its words in
    shared memory and (over 49152 blocks) in global memory."""
    w = make([blocks], 1, 3)
    g = torch.Generator().manual_seed(blocks)
    held = w["bounds"].shape[0]
    w["q"].fill_(1.0)
    x = torch.zeros(held, 2, 4, 128)
    if kind == "same":
        x[..., 0] = score = torch.ones(held, 1, 4)
    elif kind == "two":
        x[..., 0] = score = torch.randint(1, 3, (held, 1, 4), generator=g).float()
    else:  # large terms that cancel, and a small one that decides
        x[..., 0], x[..., 1] = 2.0 ** 20, -2.0 ** 20
        x[..., 2] = score = torch.randint(0, 64, (held, 1, 4), generator=g) * 2.0 ** -9
    w["bounds"].copy_(x.to(BF))
    score = score[w["table"][0, :blocks].cpu().long(), 0].numpy()
    at = np.arange(blocks)
    for top, first, last in ((700, 0, 0), (129, 1, 2), (blocks - 1, 0, 0)):
        got = select(w, top, first, last).cpu().numpy()
        for head in range(4):
            fixed = (at < first) | (at >= blocks - last)
            want = np.sort(np.lexsort((at, -score[:, head], ~fixed))[:top])
            assert np.array_equal(got[0, head], want), (top, first, last, head)
