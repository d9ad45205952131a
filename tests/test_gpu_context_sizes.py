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
    """The plain decode by copies and by tensor copies, every token's page alike: all probabilities are 2^-31, the sums of
    values that are powers of two are exact, and so is the result; the LSE is the score and 31."""
    room(16)
    n = 2 ** 31 - 1
    g = torch.Generator().manual_seed(2)
    k = torch.randn(1, 1, 4, 128, generator=g).to(BF).cuda().expand(8192, 1, 4, 128).contiguous()
    v = torch.exp2(torch.randint(-3, 4, (1, 1, 4, 128), generator=g).float()).to(BF).cuda().expand_as(k).contiguous()
    q = torch.randn(1, 32, 128, generator=g).to(BF).cuda()
    pages = torch.arange(n, dtype=I32, device="cuda").bitwise_and_(8191)
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


def listed(lens, width, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 4, (len(lens), width), generator=g).float().cuda()
    ids = torch.randperm(sum(lens) + 9, generator=g)[:sum(lens)].to(I32).cuda()
    return w, i32(np.concatenate([[0], np.cumsum(lens)])), ids


def evicted(w, indptr, ids, budget, first, last):
    got = pkg.kv_evict(w, indptr, ids, budget, first, last)
    for name, a, b in zip(("weights", "kv_indptr", "kv_indices", "freed_indptr", "freed"), got,
                          cx.evict_oracle(w, indptr, ids, budget, first, last)):
        assert np.array_equal(a.cpu().numpy(), b), name
    return got


@pytest.mark.parametrize("batch", [1023, 1024, 1025, 8192, 8193, 20001, 70000])
def test_eviction_of_many_sequences(batch):
    """More sequences than every block sums up by itself, and than there are clusters or blocks of threads."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 12, (batch,), generator=g).tolist()
    evicted(*listed(lens, 12, batch), 6, 1, 2)


def test_eviction_of_many_sequences_of_which_one_is_long():
    lens = [3] * 3000 + [40000] + [7] * 3000
    w, indptr, ids = listed(lens, 40000, 1)
    want = evicted(w, indptr, ids, 5, 1, 1)
    cut = indptr.clone()
    cut[3001 + 2000:] = 2 ** 30  # the last sequences reach past the indices: all of them end where those end
    short = ids[:int(indptr[3001 + 2000])].contiguous()
    got = pkg.kv_evict(w, cut, short, 5, 1, 1)
    ends = cut.clamp(max=short.numel())
    for a, b in zip(got, cx.evict_oracle(w, ends, short, 5, 1, 1)):
        assert np.array_equal(a.cpu().numpy(), b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = pkg.kv_evict(w, indptr, ids, 5, 1, 1)
    for _ in range(2):
        for t in res:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))


MANY = 70_000  # rows: more than a grid's second dimension, and than the join's blocks


def scores64(q, k, scale=128 ** -0.5):
    """(scores [N, 32] in base 2, the sum of their terms' sizes) of q [N, 32, 128] and k [N, 4, 128]."""
    q, k = q.double().unflatten(1, (4, 8)), k.double()[:, :, None]
    return ((q * k).sum(-1).flatten(1) * scale / np.log(2), (q * k).abs().sum(-1).flatten(1) * scale)


def test_rows_past_a_grids_second_dimension():
    """One token a row: its value is the output, its score the LSE, and 32 heads of weight 1 its weight."""
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    k, v, q = rand(500, 1, 4, 128), rand(500, 1, 4, 128), rand(MANY, 32, 128)
    pages = torch.randint(0, 500, (MANY,), generator=g, device="cuda").to(I32)
    at = torch.arange(MANY + 1, dtype=I32, device="cuda")
    old = torch.rand(MANY, 3, generator=g, device="cuda")
    out, lse, weights = pkg.run_weighted(q, k, v, at, pages, old, decay=0.5)
    want, (score, size) = v[pages.long(), 0].repeat_interleave(8, 1), scores64(q, k[pages.long(), 0])
    bound = cx.SCORE_ERROR * size / np.log(2) + 2.0 ** -20 * (1 + score.abs())
    assert torch.equal(out, want) and ((lse - score).abs() <= bound).all()
    assert ((weights[:, 0] - (0.5 * old[:, 0] + 32)).abs() <= 2.0 ** -12).all() and torch.equal(weights[:, 1:], old[:, 1:])
    # the same rows as blocks of one token
    table, req, one = pages.view(-1, 1), at[:-1].contiguous(), torch.ones(MANY, dtype=I32, device="cuda")
    bounds = torch.zeros(500, 2, 4, 128, dtype=BF, device="cuda")
    pkg.block_bounds(k, bounds, table, one)
    assert torch.equal(bounds[pages.long()], k[pages.long()].expand(-1, 2, 4, 128))
    blocks = pkg.block_select(q, bounds, table, req, one, 2, 1)
    assert (blocks[..., 0] == 0).all() and (blocks[..., 1] == -1).all()
    out, lse = pkg.block_sparse_run(q, k, v, blocks, table, req, one)
    assert torch.equal(out, want) and ((lse - score).abs() <= bound).all()
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("members", [2, 1])
def test_shared_prefixes_of_many_groups_and_sequences(members):
    """A prefix of one token a group, and one own token a sequence: a softmax of two scores."""
    g = torch.Generator(device="cuda").manual_seed(members)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    groups = MANY // members
    k, v, q = rand(500, 1, 4, 128), rand(500, 1, 4, 128), rand(MANY, 32, 128)
    prefix, own = (torch.randint(0, 500, (n,), generator=g, device="cuda").to(I32) for n in (groups, MANY))
    at = torch.arange(MANY + 1, dtype=I32, device="cuda")
    out, lse = pkg.shared_run(q, k, v, at[:groups + 1].contiguous(), prefix, at[:groups + 1] * members, at, own)
    first = prefix.long().repeat_interleave(members)
    (s0, z0), (s1, z1) = scores64(q, k[first, 0]), scores64(q, k[own.long(), 0])
    want = torch.logaddexp2(s0, s1)
    off = cx.SCORE_ERROR * torch.maximum(z0, z1)
    assert ((lse - want).abs() <= off / np.log(2) + 2.0 ** -20 * (1 + want.abs())).all()
    v0, v1 = (v[x, 0].double().repeat_interleave(8, 1) for x in (first, own.long()))
    p0 = torch.exp2(s0 - want)[..., None]
    o, room = p0 * v0 + (1 - p0) * v1, p0 * v0.abs() + (1 - p0) * v1.abs()
    inner = room * (torch.expm1(2 * off)[..., None] + 2.0 ** -8 + 2.0 ** -16)
    assert ((out - o).abs() <= inner + (o.abs() + inner) * 2.0 ** -8 + 1e-30).all()
    assert _lib.gqa_paged_decode_device_error() == 0
