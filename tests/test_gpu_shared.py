"""GPU parity of the decode over shared prefixes against the float64 definition on the joined lists.

Tolerances (oracle/context.py): probabilities rounded to bf16 (fp16 with an FP8 cache), scores off by what the MMA's
sums cut off, results rounded once.
"""
import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def caches(pool, fp8, g, std=1.0):
    got = []
    for big in (4.0, 1.0):
        x = torch.randn(pool, 4, 128, generator=g) * std
        x[..., ::32] *= big
        if fp8:
            scale = (x.abs().amax(-1) / 448).clamp(min=1e-30) * torch.exp2(torch.randint(-3, 1, (pool, 4), generator=g).float())
            rows = torch.empty(pool, 528, dtype=torch.uint8)
            rows[:, :512] = (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1).view(torch.uint8)
            rows[:, 512:] = scale.view(torch.uint8)
            got.append(rows.cuda())
        else:
            got.append(x.to(BF).view(pool, 1, 4, 128).cuda())
    return got


def make(prefixes, members, alone, own, fp8=False, seed=0, before=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    batch = before + sum(members) + alone
    own = [own[i % len(own)] for i in range(batch)]
    total = sum(prefixes) + sum(own)
    pool = total + 7
    ids = torch.randperm(pool, generator=g)[:total].to(torch.int32).cuda()
    k, v = caches(pool, fp8, g, std)
    q = torch.randn(batch, 32, 128, generator=g).to(BF).cuda()
    return (q, k, v, offsets(prefixes), ids[:sum(prefixes)].contiguous(), offsets(members) + before, offsets(own),
            ids[sum(prefixes):].contiguous())


def check(args, out, lse, sm_scale=128 ** -0.5):
    want = cx.shared_oracle(*args, sm_scale)
    fp8 = args[1].dtype == torch.uint8
    o, l = cx.f64(out), cx.f64(lse)
    for b, a in enumerate(want):
        assert np.all(np.abs(o[b] - a.out) <= a.out_bound(fp8)), (b, np.abs(o[b] - a.out).max())
        empty = np.isneginf(a.lse)
        assert np.array_equal(np.isneginf(l[b]), empty)
        assert np.all(np.abs(l[b][~empty] - a.lse[~empty]) <= a.lse_bound()[~empty]), b
    assert _lib.gqa_paged_decode_device_error() == 0


CASES = [
    ([1], [1], 0, [0], 0),
    ([1], [1], 0, [1], 0),
    ([130], [3], 0, [5, 0, 17], 0),
    ([127, 128, 129], [1, 2, 3], 0, [3], 0),
    ([300], [16], 0, [1, 40], 0),
    ([257], [33], 1, [0, 9], 2),
    ([0, 64, 0], [2, 2, 0], 1, [0, 3], 0),
    ([50, 400, 7, 1000], [1, 40, 0, 17], 2, [0, 1, 33, 129], 3),
    ([5000], [2], 0, [11, 700], 0),
    ([2100], [70], 0, [12], 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefixes,members,alone,own,before", CASES)
def test_parity(prefixes, members, alone, own, before, fp8):
    args = make(prefixes, members, alone, own, fp8, seed=len(own) + sum(prefixes), before=before)
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_prefix_is_the_plain_decode(fp8):
    args = make([], [], 5, [0, 1, 200, 33], fp8, seed=5)
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_to_read_gives_zero(fp8):
    args = make([0], [3], 1, [0], fp8)
    out, lse = pkg.shared_run(*args, out=torch.full((4, 32, 128), 7.0, dtype=BF, device="cuda"))
    assert torch.equal(out, torch.zeros_like(out)) and torch.isneginf(lse).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    args = make([200, 31], [5, 2], 0, [4], seed=9)
    out, lse = pkg.shared_run(*args, sm_scale=scale)
    check(args, out, lse, scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_are_left_out(fp8):
    args = list(make([300, 2], [4, 2], 1, [3, 0, 40], fp8, seed=3))
    bad = torch.tensor([-1, 2 ** 31 - 1, args[1].shape[0], -2 ** 31], dtype=torch.int64).to(torch.int32).cuda()
    args[4] = args[4].clone()
    args[4][3:7] = bad
    args[4][300:302] = -1  # a prefix with no page of the pool
    args[7] = args[7].clone()
    args[7][:3] = -5       # a sequence with none of its own
    args[7][4:8] = bad
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)


def test_large_and_small_values():
    for std in (1e-3, 30.0):
        args = make([260], [3], 0, [2], seed=1, std=std)
        out, lse = pkg.shared_run(*args)
        check(args, out, lse)


def test_one_page_many_times():
    args = list(make([150], [4], 0, [6], seed=2))
    args[4], args[7] = torch.full_like(args[4], 11), torch.full_like(args[7], 11)
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)


def test_not_finite_tokens_stay_with_their_sequences():
    args = list(make([200, 200], [3, 3], 0, [9], seed=4))
    k = args[1].clone()
    k[args[7][args[6][1]].long()] = float("nan")      # a token of sequence 1's own
    k[args[4][250].long()] = float("nan")             # a token of prefix 1
    out, lse = pkg.shared_run(args[0], k, *args[2:])
    clean = pkg.shared_run(*args)
    for b in (0, 2):
        assert torch.equal(out[b], clean[0][b]) and torch.equal(lse[b], clean[1][b])
    assert torch.isnan(out[1]).all() and torch.isnan(out[3:]).all()


def test_repeats_streams_graphs_and_workspaces():
    args = make([3000, 40], [20, 3], 2, [60, 0, 300], seed=6)
    want = pkg.shared_run(*args)
    for _ in range(3):
        got = pkg.shared_run(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = pkg.shared_run(*args, stream=stream)
    stream.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    size = _lib.load().gqa_shared_paged_decode_ws_size(args[0].shape[0], 2, 0)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    got = pkg.shared_run(*args, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = pkg.shared_run(*args)
        graphs.append((graph, res))
    for graph, res in graphs * 2:
        res[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
    # new lengths in the same tensors: the captured call follows them
    args[3][1:] = torch.tensor([1500, 1540], dtype=torch.int32)
    want = pkg.shared_run(*args)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], want[0])
    check(args, *want)


def test_offsets_past_the_tables_are_cut():
    args = list(make([100], [2], 0, [10], seed=8))
    args[3] = torch.tensor([0, 1000], dtype=torch.int32).cuda()
    args[6] = torch.tensor([0, 10, 500], dtype=torch.int32).cuda()
    out, lse = pkg.shared_run(*args)
    assert torch.isfinite(out.float()[0]).all()


def test_many_groups():
    """More groups than a block of threads counts at once, most of them of one sequence, empty ones among them."""
    g = torch.Generator().manual_seed(11)
    members = torch.randint(0, 3, (1300,), generator=g).tolist()
    prefixes = torch.randint(0, 40, (1300,), generator=g).tolist()
    members[700], prefixes[700] = 70, 300
    args = make(prefixes, members, 2, [0, 1, 2], seed=12)
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)


def test_fp8_scales_of_zero_and_far_apart():
    args = list(make([400], [20], 0, [5, 0], True, seed=13))
    k, v = args[1], args[2]
    scales = v[:, 512:].view(torch.float32)
    scales[::3] = 0.0
    scales[1::7] *= 2.0 ** 20
    scales[2::7] *= 2.0 ** -30
    k[:, 512:].view(torch.float32)[::5] = 0.0
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)
    scales.zero_()
    out, lse = pkg.shared_run(*args)
    check(args, out, lse)
    assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_wait_that_gives_up_and_the_next_call(fp8):
    """With a limit of a few nanoseconds the waits of the prefix pass run out: the call completes, the device error word
    carries a timeout bit and no other, and the next call gives what the one before gave."""
    args = make([3000], [40], 0, [20], fp8, seed=14)
    want = pkg.shared_run(*args)
    assert _lib.gqa_paged_decode_device_error() == 0
    try:
        assert _lib.gqa_paged_decode_test_wait_limit_ns(5) == 0
        for _ in range(3):
            pkg.shared_run(*args)
        torch.cuda.synchronize()
        flags = _lib.gqa_paged_decode_device_error()
        assert flags & 3 and not flags & ~3, flags
    finally:
        _lib.gqa_paged_decode_test_wait_limit_ns(0)
    for _ in range(3):
        got = pkg.shared_run(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _lib.gqa_paged_decode_device_error() == 0


def test_two_streams_at_once():
    a, b = make([2000], [33], 0, [100], seed=15), make([50, 900], [2, 20], 1, [7, 300], True, seed=16)
    want = pkg.shared_run(*a), pkg.shared_run(*b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append([pkg.shared_run(*x, stream=s) for x, s in zip((a, b), streams)])
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefixes,members,own", [([1000], [100], [1]), ([300, 40], [70, 50], [0, 1, 2]), ([40], [60], [300, 500]), ([3000], [40], [2, 900])])
def test_parity_over_the_plans(prefixes, members, own, fp8):
    """Own tokens few, short and many beside the prefix: every share of the SMs."""
    args = make(prefixes, members, 1, own, fp8, seed=sum(prefixes) + sum(own))
    check(args, *pkg.shared_run(*args))
