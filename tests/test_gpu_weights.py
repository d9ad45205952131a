"""GPU parity of the decode that accumulates attention weights, and of the eviction by them."""
import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
from test_gpu_shared import caches, offsets

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def make(lens, width, fp8, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    k, v = caches(total + 5, fp8, g, std)
    ids = torch.randperm(total + 5, generator=g)[:total].to(torch.int32).cuda()
    q = torch.randn(len(lens), 32, 128, generator=g).to(BF).cuda()
    return q, k, v, offsets(lens), ids, (torch.rand(len(lens), width, generator=g) * 5).cuda()


def check(args, decay, got, scale=128 ** -0.5):
    rows, weights, bound = cx.weighted_oracle(*args, decay, scale)
    fp8 = args[1].dtype == torch.uint8
    o, l, w = (cx.f64(t) for t in got)
    for b, a in enumerate(rows):
        assert np.all(np.abs(o[b] - a.out) <= a.out_bound(fp8)), b
        empty = np.isneginf(a.lse)
        assert np.array_equal(np.isneginf(l[b]), empty) and np.all(np.abs(l[b][~empty] - a.lse[~empty]) <= a.lse_bound()[~empty])
    assert np.all(np.abs(w - weights) <= bound), np.abs(w - weights).max()
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,width,decay", [([1], 1, 1.0), ([0, 3, 700], 800, 1.0), ([17, 0, 300, 16, 33], 310, 0.9),
                                              ([5000, 2], 5001, 0.0), ([257] * 40, 257, 0.5), ([100, 50], 60, 1.0),
                                              ([9], 0, 1.0)])
def test_parity(lens, width, decay, fp8):
    args = make(lens, width, fp8, sum(lens))
    got = pkg.run_weighted(*args, decay=decay)
    check(args, decay, got)
    run = pkg.run_fp8 if fp8 else pkg.run
    out, lse = run(*args[:5])
    # the same kernel with its scores stored: the same results, but where its plan's CTAs lie
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_in_place_and_untouched_places(fp8):
    args = make([40, 0, 333], 400, fp8, 1)
    want = pkg.run_weighted(*args)[2]
    old = args[5].clone()
    got = pkg.run_weighted(*args, weights_out=args[5])[2]
    assert got is args[5] and torch.equal(got, want)
    for b, n in enumerate([40, 0, 333]):
        assert torch.equal(got[b, n:], old[b, n:])


def test_a_decay_of_zero_reads_no_weights():
    args = list(make([40, 3], 64, False, 2))
    args[5].fill_(float("nan"))
    got = pkg.run_weighted(*args, decay=0.0)[2]
    assert torch.isfinite(got[0, :40]).all() and torch.isnan(got[0, 40:]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_get_no_weight(fp8):
    args = list(make([40, 3, 2], 64, fp8, 3))
    args[4][[1, 7]] = torch.tensor([-1, args[1].shape[0]], dtype=torch.int32).cuda()
    args[4][43:] = 2 ** 31 - 1  # the last sequence has no page at all
    got = pkg.run_weighted(*args)
    check(args, 1.0, got)
    assert torch.equal(got[2][0, [1, 7]], args[5][0, [1, 7]]) and torch.equal(got[2][2], args[5][2])


def test_weights_of_a_step_sum_to_the_heads():
    args = make([1000, 1, 64], 1000, False, 4)
    got = pkg.run_weighted(*args, decay=0.0, weights_out=torch.zeros_like(args[5]))[2]
    assert torch.allclose(got[[0, 1, 2]].sum(1)[0], torch.tensor(32.0).cuda(), atol=1e-3)
    assert abs(float(got[1, 0]) - 32) < 1e-3 and abs(float(got[2, :64].sum()) - 32) < 1e-3


def evict_check(args, got):
    want = cx.evict_oracle(*args)
    for name, a, b in zip(("weights", "kv_indptr", "kv_indices", "freed_indptr", "freed"), got, want):
        assert np.array_equal(a.cpu().numpy(), b, equal_nan=name == "weights"), name


def listed(lens, width, seed, kind="random"):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(len(lens), width, generator=g)
    if kind == "few":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif kind == "same":
        w = torch.zeros_like(w)
    elif kind == "wide":
        w = torch.exp(w * 20) * torch.randint(0, 2, w.shape, generator=g)
    elif kind == "special":
        w[:, ::7], w[:, 1::7], w[:, 2::7] = float("nan"), float("inf"), float("-inf")
        w[:, 3::7], w[:, 4::7] = -0.0, 0.0
    ids = torch.randperm(sum(lens) + 9, generator=g)[:sum(lens)].to(torch.int32)
    return w.cuda(), offsets(lens), ids.cuda()


@pytest.mark.parametrize("kind", ["random", "few", "same", "wide", "special"])
@pytest.mark.parametrize("lens,width,budget,first,last", [
    ([1], 1, 1, 0, 0), ([5, 0, 9], 12, 4, 1, 1), ([2000, 1023, 1024, 1025, 3], 2048, 1000, 4, 128), ([3000], 3001, 1, 0, 0),
    ([100, 100], 100, 50, 50, 0), ([100, 200], 200, 60, 0, 60), ([100, 7], 100, 0, 0, 0), ([40] * 300, 41, 33, 2, 5),
    ([500, 400], 300, 350, 3, 40), ([70000, 20], 70000, 5000, 10, 100)])
def test_evict(lens, width, budget, first, last, kind):
    w, indptr, ids = listed(lens, width, sum(lens) + budget, kind)
    evict_check((w, indptr, ids, budget, first, last), pkg.kv_evict(w, indptr, ids, budget, first, last))


def test_evict_nothing_and_everything():
    w, indptr, ids = listed([30, 0, 12], 40, 1)
    evict_check((w, indptr, ids, 2 ** 31 - 1, 0, 0), pkg.kv_evict(w, indptr, ids, 2 ** 31 - 1))
    got = pkg.kv_evict(w, indptr, ids, 0)
    assert torch.equal(got[4], ids) and torch.equal(got[3], indptr)
    empty = pkg.kv_evict(w[:0], indptr[:1], ids[:0], 5)
    assert [t.numel() for t in empty] == [0, 1, 0, 1, 0] and int(empty[1][0]) == int(empty[3][0]) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_steps_with_eviction(fp8):
    """Decode and accumulate, evict, decode on the shorter table: as a serving loop runs them, captured and not."""
    lens = [300, 90, 500]
    args = make(lens, 512, fp8, 7)
    _, _, w = pkg.run_weighted(*args)
    w2, indptr, ids, freed_at, freed = pkg.kv_evict(w, args[3], args[4], 128, keep_first=4, keep_last=32)
    evict_check((w, args[3], args[4], 128, 4, 32), (w2, indptr, ids, freed_at, freed))
    assert [int(x) for x in indptr] == [0, 128, 218, 346]
    got = pkg.run_weighted(*args[:3], indptr, ids, w2, decay=0.5)
    check((*args[:3], indptr, ids[:346], w2), 0.5, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, cw = pkg.run_weighted(*args)
        kept = pkg.kv_evict(cw, args[3], args[4], 128, keep_first=4, keep_last=32)
        res = pkg.run_weighted(*args[:3], kept[1], kept[2], kept[0], decay=0.5)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, got))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    side = pkg.run_weighted(*args, stream=stream)
    side = pkg.kv_evict(side[2], args[3], args[4], 128, keep_first=4, keep_last=32, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(side, (w2, indptr, ids, freed_at, freed)))


def test_offsets_past_the_indices_are_cut():
    args = list(make([30, 20], 64, False, 8))
    whole = pkg.run_weighted(*args)
    args[3] = torch.tensor([0, 30, 5000], dtype=torch.int32).cuda()
    got = pkg.run_weighted(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, whole))
    args[3] = torch.tensor([0, 50, 5000], dtype=torch.int32).cuda()  # the second begins where the indices end
    out, lse, w = pkg.run_weighted(*args)
    assert torch.equal(out[1], torch.zeros_like(out[1])) and torch.isneginf(lse[1]).all() and torch.equal(w[1], args[5][1])


@pytest.mark.parametrize("n", [500_000])
def test_evict_more_than_the_blocks_hold(n):
    w, indptr, ids = listed([n, 3], n, 3, "few")
    evict_check((w, indptr, ids, n // 3, 10, 1000), pkg.kv_evict(w, indptr, ids, n // 3, 10, 1000))


@pytest.mark.parametrize("lens,budget", [([70000, 1, 0, 4096, 65536], 5000), ([33000], 33000 - 1), ([20000, 16384], 1), ([300] * 200 + [9000], 256)])
def test_evict_by_clusters_of_each_size(lens, budget):
    first, last = min(2, budget), min(40, budget - min(2, budget))
    w, indptr, ids = listed(lens, max(lens), 5, "few")
    evict_check((w, indptr, ids, budget, first, last), pkg.kv_evict(w, indptr, ids, budget, first, last))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[1] * 300, [0, 1, 2, 3] * 100, [15, 17, 0] * 40, [400] * 30, [300, 3] * 60])
def test_parity_over_the_plans(lens, fp8):
    """Sequences of a token or two (small shares), and as many tokens as one tier takes."""
    args = make(lens, max(lens), fp8, sum(lens) + 1)
    check(args, 0.5, pkg.run_weighted(*args, decay=0.5))
