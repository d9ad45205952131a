"""A query head that meets a score of NaN or +inf gets NaN for its outputs and its LSE, as in a plain softmax, whether its
sequence is whole or cut into pieces, and wherever among them the token lies; the other heads keep their bits. The weights
accumulated beside it are NaN for the tokens of that sequence, but for those that are left out.
"""
import pytest
import torch

import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
from test_gpu_shared import caches, offsets

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
SICK = slice(16, 24)  # the query heads of KV head 2


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


@pytest.fixture(autouse=True)
def _defaults():
    yield
    _lib.gqa_paged_decode_set_tuning(0, 0, 0, 0, 0, 0)
    _lib.gqa_paged_decode_set_merge_mode(_lib.MERGE_KERNEL)


def make(lens, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    k, v = caches(total + 5, fp8, g)
    ids = torch.randperm(total + 5, generator=g)[:total].to(I32).cuda()
    return torch.randn(len(lens), 32, 128, generator=g).to(BF).cuda(), k, v, offsets(lens), ids


def spoil(k, pages, value=float("nan")):
    """KV head 2 of the pages' keys (FP8: their scales)."""
    k = k.clone()
    if k.dtype == torch.uint8:
        scales = k[:, 512:].clone().view(torch.float32)
        scales[pages.long(), 2] = value
        k[:, 512:] = scales.view(torch.uint8)
    else:
        k[pages.long(), 0, 2] = value
    return k


def check(got, clean, sick_rows):
    (out, lse), (out0, lse0) = got, clean
    for b in range(out.shape[0]):
        if b not in sick_rows:
            assert torch.equal(out[b], out0[b]) and torch.equal(lse[b], lse0[b]), b
            continue
        assert out[b, SICK].isnan().all() and lse[b, SICK].isnan().all(), b
        for heads in (slice(0, 16), slice(24, 32)):
            assert torch.equal(out[b, heads], out0[b, heads]) and torch.equal(lse[b, heads], lse0[b, heads]), b


# sequence 1 of these; which of its tokens
CASES = [([3, 1, 9], "all"), ([3, 40, 9], "last"), ([50, 5000, 9], "first"), ([50, 5000, 9], "last"), ([50, 5000, 9], "all"),
         ([50, 60000, 700], "middle"), ([50, 60000, 700], "all")]


def tokens(n, which):
    return {"all": slice(0, n), "first": slice(0, 1), "last": slice(n - 1, n), "middle": slice(n // 2, n // 2 + 1)}[which]


@pytest.mark.parametrize("mode", ["default", "pieces joined by the last", "one wave", "one head a CTA", "copies", "fp8"])
@pytest.mark.parametrize("lens,which", CASES)
def test_decode(lens, which, mode):
    args = make(lens, mode == "fp8", sum(lens))
    tuning = {"one head a CTA": (0, 0, 1, 16, 4, 0), "copies": (0, 0, 4, 16, 5, 1),
              "pieces joined by the last": (0, 0, 4, 16, 2, 0, 1000)}
    assert _lib.gqa_paged_decode_set_tuning(*tuning.get(mode, (0, 0, 0, 0, 0, 0))) == 0
    if mode == "one wave":
        assert _lib.gqa_paged_decode_set_merge_mode(_lib.MERGE_ONE_WAVE) == 0
    run = pkg.run_fp8 if mode == "fp8" else pkg.run
    clean = run(*args, 128 ** -0.5)
    bad = spoil(args[1], args[4][lens[0]:lens[0] + lens[1]][tokens(lens[1], which)])
    check(run(args[0], bad, *args[2:], 128 ** -0.5), clean, [1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,which", CASES)
def test_weights(lens, which, fp8):
    args = make(lens, fp8, sum(lens))
    old = torch.rand(3, max(lens) + 3, generator=torch.Generator().manual_seed(1)).cuda()
    if lens[1] > 5:
        args[4][lens[0] + 3] = -1  # left out
    clean = pkg.run_weighted(*args, old, decay=0.5)
    sick = args[4][lens[0]:lens[0] + lens[1]][tokens(lens[1], which)]
    got = pkg.run_weighted(args[0], spoil(args[1], sick[sick >= 0]), *args[2:], old, decay=0.5)
    check(got[:2], clean[:2], [1])
    assert torch.equal(got[2][[0, 2]], clean[2][[0, 2]]) and torch.equal(got[2][1, lens[1]:], old[1, lens[1]:])
    inside = torch.ones(lens[1], dtype=torch.bool)
    if lens[1] > 5:
        inside[3] = False
        assert got[2][1, 3] == 0.5 * old[1, 3]
    assert got[2][1, :lens[1]][inside].isnan().all()


@pytest.mark.parametrize("which", ["first", "last", "all"])
@pytest.mark.parametrize("blocks", [1, 20, 500])
def test_chosen_blocks(blocks, which):
    g = torch.Generator().manual_seed(blocks)
    k, v = (torch.randn(blocks + 3, 16, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(3, 32, 128, generator=g).to(BF).cuda()
    table = torch.arange(blocks + 3, dtype=I32).cuda()[None]
    listed = torch.arange(blocks, dtype=I32).cuda().expand(3, 4, blocks).contiguous()
    listed[0] = blocks + 1
    listed[2, :, 1:] = -1
    listed[2, :, 0] = blocks + 2
    args = (listed, table, torch.zeros(3, dtype=I32).cuda(), torch.full((3,), 16 * (blocks + 3), dtype=I32).cuda())
    clean = pkg.block_sparse_run(q, k, v, *args)
    k.view(-1, 4, 128)[:16 * blocks][tokens(16 * blocks, which), 2] = float("nan")
    check(pkg.block_sparse_run(q, k, v, *args), clean, [1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,own,where", [(0, 1, "own"), (0, 3000, "own"), (1, 0, "prefix"), (1000, 0, "prefix"),
                                              (1000, 200, "own"), (1000, 200, "prefix"), (40000, 3000, "own")])
def test_shared_prefixes(prefix, own, where, fp8):
    q, k, v, _, ids = make([prefix, 10, own, 25], fp8, prefix + own)
    q = torch.cat([q[:3], q[:1]])  # sequences 0 to 2 of the group, one of none
    args = (q, k, v, offsets([prefix]), ids[:prefix].contiguous(), offsets([3]), offsets([10, own, 25, 0]),
            ids[prefix:].contiguous())
    clean = pkg.shared_run(*args)
    sick = args[4] if where == "prefix" else ids[prefix + 10:prefix + 10 + own]
    got = pkg.shared_run(q, spoil(k, sick), *args[2:])
    check(got, clean, [0, 1, 2] if where == "prefix" else [1])


@pytest.mark.parametrize("n", [1, 300, 20000])
def test_scores_of_either_infinity(n):
    """Keys of +inf in one dim: heads whose query is positive there are NaN, the others' token has a weight of 0."""
    q, k, v, indptr, ids = make([n, 30], False, n)
    k = k.clone()
    k[ids[n // 2].long(), 0, 2, 5] = float("inf")
    up = q[0, SICK, 5] > 0
    for out, lse in (pkg.run(q, k, v, indptr, ids), pkg.run_weighted(q, k, v, indptr, ids, torch.zeros(2, n + 30).cuda())[:2]):
        assert torch.equal(out[0, SICK].isnan().all(1), up) and torch.equal(lse[0, SICK].isnan(), up)
        assert out[0, SICK][~up].isfinite().all() and out[1].isfinite().all() and lse[1].isfinite().all()
