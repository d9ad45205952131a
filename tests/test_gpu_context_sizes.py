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


def test_chosen_blocks_of_nearly_2_31_tokens():
    """One row whose listed blocks make 2^31 - 128 places: the reads ahead of the last ones end where the list ends. All
    places but those of the last 4 listed blocks are -1, so the result is that of these blocks alone."""
    room(48)
    page, top = 128, 2 ** 24 - 1
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(4, page, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(1, 32, 128, generator=g).to(BF).cuda()
    table, req, lens = i32([[2, 0, 3, 1]]), i32([0]), i32([3 * page + 77])
    few = i32([[[0, 1, 2, 3]] * 4])
    blocks = torch.full((1, 4, top), -1, dtype=I32, device="cuda")
    blocks[..., -4:] = few
    out, lse = pkg.block_sparse_run(q, k, v, blocks, table, req, lens)
    (want,) = cx.block_sparse_oracle(q, k, v, few, table, req, lens, 128 ** -0.5)
    assert np.all(np.abs(cx.f64(out)[0] - want.out) <= want.out_bound(False))
    assert np.all(np.abs(cx.f64(lse)[0] - want.lse) <= want.lse_bound())
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("tuning", [(0, 0, 0, 0, 0, 0), (0, 0, 4, 16, 5, 1)])
def test_decode_of_nearly_2_31_tokens(tuning):
    """The plain decode by copies and by tensor copies, every token the same page: all probabilities are 2^-31, the sums of
    values that are powers of two are exact, and so is the result; the LSE is the score and 31."""
    room(16)
    n = 2 ** 31 - 1
    g = torch.Generator().manual_seed(2)
    k = torch.randn(3, 1, 4, 128, generator=g).to(BF).cuda()
    v = torch.exp2(torch.randint(-3, 4, (3, 1, 4, 128), generator=g).float()).to(BF).cuda()
    q = torch.randn(1, 32, 128, generator=g).to(BF).cuda()
    pages = torch.ones(n, dtype=I32, device="cuda")
    try:
        assert _lib.gqa_paged_decode_set_tuning(*tuning) == 0
        out, lse = pkg.run(q, k, v, i32([0, n]), pages, 128 ** -0.5)
    finally:
        _lib.gqa_paged_decode_set_tuning(0, 0, 0, 0, 0, 0)
    assert torch.equal(out[0].view(4, 8, 128), v[1, 0][:, None].expand(4, 8, 128))
    s = (cx.f64(q)[0].reshape(4, 8, 128) * cx.f64(k)[1, 0][:, None]).sum(-1).reshape(32) * 128 ** -0.5 / np.log(2)
    a = cx.Attended(q[0], cx.f64(k)[1], cx.f64(v)[1], 128 ** -0.5)
    # the pieces' own LSEs are rounded to 2^-24 of about 31, and 2^-19 of weight: 2^-18 in all
    assert np.all(np.abs(cx.f64(lse)[0] - s - 31) <= a.lse_bound() + 2.0 ** -18)
    assert _lib.gqa_paged_decode_device_error() == 0
