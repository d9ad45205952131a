"""GPU parity of the attention over selected blocks: bounds (exact), choice (exact), the decode over the chosen blocks."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def make(lens, page, seed, rows=1, spare=3):
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    blocks, width = sum(used) + spare, max(1, max(used)) + 1
    ids = torch.randperm(blocks, generator=g)[:sum(used)].tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for r, u in enumerate(used):
        table[r, :u] = torch.tensor(ids[:u], dtype=torch.int32)
        ids = ids[u:]
    k, v = (torch.randn(blocks, page, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(len(lens) * rows, 32, 128, generator=g).to(BF).cuda()
    req = i32([r for r in range(len(lens)) for _ in range(rows)])
    row_lens = i32([max(0, n - rows + 1 + i) for n in lens for i in range(rows)])
    bounds = torch.full((blocks, 2, 4, 128), 3.0, dtype=BF, device="cuda")
    return dict(q=q, k=k, v=v, table=table.cuda(), req=req, row_lens=row_lens, lens=i32(lens), bounds=bounds)


def same_values(got, want):
    a, nan = cx.f64(got), np.isnan(want)
    return np.array_equal(np.isnan(a), nan) and np.array_equal(a[~nan], want[~nan])


@pytest.mark.parametrize("lens,page,first", [
    ([1], 1, None), ([0, 5], 16, None), ([64, 65, 63], 64, [63, 64, 0]), ([1000, 17, 0, 333], 16, [999, 16, 0, 100]),
    ([50, 50], 7, [50, 49]), ([2000], 128, [0]), ([300, 300], 256, [-5, 299]), ([9, 9], 3, [1000, 2 ** 31 - 1]),
])
def test_bounds(lens, page, first):
    w = make(lens, page, sum(lens))
    first = None if first is None else i32(first)
    want = cx.bounds_oracle(w["k"], w["bounds"], w["table"], w["lens"], first)
    got = pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"], first)
    assert got is w["bounds"] and same_values(got, want)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"], first)
    assert same_values(got, want)


def test_bounds_follow_the_steps():
    """Token by token, as a decode renews them: the same as all at once."""
    w = make([0, 40], 16, 1)
    for n in range(1, 41):
        pkg.block_bounds(w["k"], w["bounds"], w["table"], i32([0, n]), i32([0, n - 1]))
    assert same_values(w["bounds"], cx.bounds_oracle(w["k"], torch.full_like(w["bounds"], 3.0), w["table"], w["lens"]))


def test_bounds_of_special_values_and_bad_tables():
    w = make([100, 30], 16, 2)
    k = w["k"]
    k[int(w["table"][0, 1]), 3, 2, 5] = float("nan")
    k[int(w["table"][0, 2]), 0, 0, 0], k[int(w["table"][0, 2]), 1, 0, 0] = float("inf"), float("-inf")
    k[int(w["table"][1, 1]), 14:] = float("nan")  # past the length
    w["table"][0, 0], w["table"][0, 3], w["table"][0, 4] = -1, k.shape[0], 2 ** 31 - 1
    want = cx.bounds_oracle(k, w["bounds"], w["table"], w["lens"])
    assert same_values(pkg.block_bounds(k, w["bounds"], w["table"], w["lens"]), want)
    lens = i32([2 ** 31 - 1, -7])  # cut to the table; none
    want = cx.bounds_oracle(k, w["bounds"], w["table"], lens)
    assert same_values(pkg.block_bounds(k, w["bounds"], w["table"], lens), want)


def select(w, top, first=1, last=1, lens=None, **more):
    return pkg.block_select(w["q"], w["bounds"], w["table"], w["req"], w["row_lens"] if lens is None else lens, top,
                            w["k"].shape[1], keep_first=first, keep_last=last, **more)


def chosen(w, top, first=1, last=1, lens=None):
    return cx.select_oracle(w["q"], w["bounds"], w["table"], w["req"], w["row_lens"] if lens is None else lens, top,
                            w["k"].shape[1], first, last)


SELECT = [([1], 16, 1, 1, 0, 0), ([0, 3, 900], 16, 1, 5, 1, 1), ([5000, 33, 1024], 16, 1, 17, 2, 3),
          ([4096, 100], 32, 5, 64, 0, 0), ([40000], 8, 1, 200, 1, 4), ([2000, 3, 17], 64, 3, 4, 2, 2),
          ([700] * 40, 16, 2, 10, 0, 1), ([20000], 1, 1, 300, 3, 9), ([1200], 16, 1, 100, 1, 1)]


@pytest.mark.parametrize("lens,page,rows,top,first,last", SELECT)
def test_choice(lens, page, rows, top, first, last):
    w = make(lens, page, sum(lens) + top, rows)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    got = select(w, top, first, last)
    assert np.array_equal(got.cpu().numpy(), chosen(w, top, first, last))
    again = select(w, top, first, last)
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["zero", "few", "near", "one"])
def test_choice_of_equal_and_near_scores(kind):
    """Scores that tie, or differ by less than the MMA's rounding: exact in 64 bits for these small integers."""
    w = make([3000, 500], 8, 3)
    g = torch.Generator().manual_seed(1)
    shape = w["bounds"].shape
    if kind == "zero":
        w["q"].zero_()
        w["bounds"].copy_(torch.randn(shape, generator=g).to(BF))
    elif kind == "one":
        w["bounds"].fill_(1.0)
    elif kind == "few":
        w["q"].copy_(torch.randint(-2, 3, w["q"].shape, generator=g).to(BF))
        w["bounds"].copy_(torch.randint(0, 2, shape, generator=g).to(BF))
    else:  # large terms that cancel, and a small one that decides
        w["q"].fill_(1.0)
        x = torch.zeros(shape)
        x[..., 0], x[..., 1] = 2.0 ** 20, -2.0 ** 20
        x[..., 2] = torch.randint(0, 64, shape[:-1], generator=g) * 2.0 ** -9
        w["bounds"].copy_(x.to(BF))
    for top, first, last in ((7, 0, 0), (40, 1, 1), (1, 0, 1)):
        assert np.array_equal(select(w, top, first, last).cpu().numpy(), chosen(w, top, first, last)), (top, first, last)


def test_choice_with_numbers_that_are_not_finite():
    w = make([600, 300], 8, 4, rows=2)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    b, t = w["bounds"], w["table"].long()
    b[t[0, 5], 0, 1, 7] = float("nan")
    b[t[0, 9], 0] = float("inf")
    b[t[0, 11], 1, :, 3] = float("-inf")
    b[t[1, 2]] = 3e38                       # finite bounds whose products are not
    w["q"][3, 9, 4] = float("nan")          # a query of request 1's second row
    for top, first, last in ((4, 0, 0), (9, 1, 1)):
        assert np.array_equal(select(w, top, first, last).cpu().numpy(), chosen(w, top, first, last))


def test_choice_of_bad_rows_tables_and_lengths():
    w = make([600, 300, 100], 8, 5, rows=2)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    w["table"][0, 3:6] = i32([-1, w["k"].shape[0], 2 ** 31 - 1])
    w["table"][2] = -1
    w["req"].copy_(i32([0, 3, 1, -1, 2, 2]))
    for lens in (w["row_lens"], i32([2 ** 31 - 1, 5, -3, 7, 100, 100])):
        for top, first, last in ((6, 2, 1), (5, 5, 0), (100, 3, 3)):
            assert np.array_equal(select(w, top, first, last, lens).cpu().numpy(), chosen(w, top, first, last, lens))


def attend(w, blocks, scale=None, lens=None, **more):
    return pkg.block_sparse_run(w["q"], w["k"], w["v"], blocks, w["table"], w["req"], w["row_lens"] if lens is None else lens,
                                scale, **more)


def check(w, blocks, out, lse, scale=128 ** -0.5, lens=None):
    want = cx.block_sparse_oracle(w["q"], w["k"], w["v"], blocks, w["table"], w["req"], w["row_lens"] if lens is None else lens,
                                  scale)
    o, l = cx.f64(out), cx.f64(lse)
    for r, a in enumerate(want):
        assert np.all(np.abs(o[r] - a.out) <= a.out_bound(False)), (r, np.abs(o[r] - a.out).max())
        empty = np.isneginf(a.lse)
        assert np.array_equal(np.isneginf(l[r]), empty)
        assert np.all(np.abs(l[r][~empty] - a.lse[~empty]) <= a.lse_bound()[~empty]), r
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("lens,page,rows,top,first,last", SELECT)
def test_bound_choose_attend(lens, page, rows, top, first, last):
    """The three together, as a step runs them."""
    w = make(lens, page, sum(lens) + top, rows)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    blocks = select(w, top, first, last)
    out, lse = attend(w, blocks)
    check(w, blocks, out, lse)


def test_all_blocks_is_the_dense_decode():
    w = make([500, 40, 0], 16, 6)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    out, lse = attend(w, select(w, 40))
    pages = [int(w["table"][r, t // 16]) * 16 + t % 16 for r, n in enumerate([500, 40, 0]) for t in range(n)]
    flat = [x.view(-1, 1, 4, 128) for x in (w["k"], w["v"])]
    want, want_lse = pkg.run(w["q"], *flat, i32([0, 500, 540, 540]), i32(pages))
    # the same tokens in pieces cut elsewhere: probabilities rounded to bf16 twice, and the results
    assert (out.float() - want.float()).abs().max() <= 2 * 2.0 ** -7 * w["v"].float().abs().max()
    fine = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), fine) and (lse - want_lse)[fine].abs().max() <= 1e-4


def test_any_lists():
    w = make([300, 129], 16, 7, rows=2)
    g = torch.Generator().manual_seed(0)
    blocks = torch.randint(-3, 25, (4, 4, 6), generator=g).to(torch.int32).cuda()  # outside, repeated, in any order
    blocks[0, 1] = -1
    blocks[3] = 2 ** 31 - 1
    w["table"][0, 2] = -1
    out, lse = attend(w, blocks, -0.2)
    check(w, blocks, out, lse, -0.2)
    lens = i32([2 ** 31 - 1, -1, 16, 5])
    out, lse = attend(w, blocks, lens=lens)
    check(w, blocks, out, lse, lens=lens)
    none, no_lse = attend(w, blocks, lens=lens, with_lse=False)
    assert torch.equal(none, out) and no_lse is None


def test_not_finite_tokens_stay_where_they_are_chosen():
    w = make([200, 200], 16, 8)
    blocks = i32(np.tile([0, 4, 12], (2, 4, 1)))
    clean = attend(w, blocks)
    w["k"][int(w["table"][0, 5])] = float("nan")         # not chosen
    w["v"][int(w["table"][1, 12]), 8:] = float("inf")    # past the length
    got = attend(w, blocks)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    w["k"][int(w["table"][1, 4]), 3, 2] = float("nan")   # chosen, KV head 2
    got = attend(w, blocks)
    assert torch.equal(got[0][0], clean[0][0]) and torch.equal(got[0][1, :16], clean[0][1, :16])
    assert torch.isnan(got[0][1, 16:24]).all() and torch.equal(got[0][1, 24:], clean[0][1, 24:])


def test_streams_graphs_and_workspaces():
    w = make([3000, 700, 50], 16, 9, rows=2)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])

    def step(**more):
        blocks = select(w, 20, **more)
        return (blocks, *attend(w, blocks, **more))

    want = step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = step(stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
            res = step()
        graphs.append((graph, res))
    for graph, res in graphs * 2:
        for t in res:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))
    lib = _lib.load()
    rows, width = w["q"].shape[0], w["table"].shape[1]
    ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
          for n in (lib.gqa_block_select_ws_size(rows, width), lib.gqa_block_sparse_decode_ws_size(rows, 20, 16))]
    blocks = select(w, 20, workspace=ws[0])
    assert torch.equal(blocks, want[0]) and torch.equal(attend(w, blocks, workspace=ws[1])[0], want[1])


def test_choice_among_more_blocks_than_are_held():
    w = make([50_000], 1, 10)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    assert np.array_equal(select(w, 700, 1, 2).cpu().numpy(), chosen(w, 700, 1, 2))


def test_bounds_of_many_requests():
    """More requests than are numbered at once; few blocks to renew, and more than there are blocks of threads."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    w = make(lens, 8, 11)
    for first in (None, i32([max(0, n - 1) for n in lens])):
        want = cx.bounds_oracle(w["k"], w["bounds"], w["table"], w["lens"], first)
        assert same_values(pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"], first), want)


@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 30 + 1])
def test_choice_of_the_longest_pages(page):
    """One block as long as a table's product with its width may be: lengths and block counts stay within 31 bits."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(4, 32, 128, generator=g).to(BF).cuda()
    bounds = torch.randn(1, 2, 4, 128, generator=g).to(BF).cuda()
    table, req = i32([[0]]), i32([0, 0, 0, 0])
    lens = i32([2 ** 31 - 1, 2 ** 30 + 1, 1, 0])
    got = pkg.block_select(q, bounds, table, req, lens, 3, page)
    assert got[:3].cpu().tolist() == [[[0, -1, -1]] * 4] * 3 and (got[3] == -1).all()


@pytest.mark.parametrize("top,first,last", [(4, 0, 0), (9, 1, 1), (40, 2, 3)])
@pytest.mark.parametrize("bad", [1, 5, 60])
def test_choice_where_errors_have_no_bound(top, first, last, bad):
    """Bounds so large where the queries are 0 that the scores' error has no finite bound: the scores themselves are the
    lowest, and whole numbers of blocks before them are to be chosen."""
    w = make([600, 8000], 8, 6)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    w["q"].mul_(10000.0)
    w["q"][:, :, 5] = 0
    for r in range(2):
        blocks = w["table"][r, 7:7 + bad].long()
        w["bounds"][blocks] = -20.0
        w["bounds"][blocks, :, :, 5] = 3e38
    assert np.array_equal(select(w, top, first, last).cpu().numpy(), chosen(w, top, first, last))


@pytest.mark.parametrize("lens,page,rows,top", [([40] * 200, 1, 1, 1), ([500] * 50, 4, 2, 3), ([3000] * 8, 16, 2, 100)])
def test_attention_over_the_plans(lens, page, rows, top):
    """Rows of a token or a few (small shares), and as many tokens as one tier takes."""
    w = make(lens, page, sum(lens), rows)
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    blocks = select(w, top, 0, 1)
    check(w, blocks, *attend(w, blocks))
