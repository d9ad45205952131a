"""A sequence's tokens that are not finite reach that sequence's rows alone, and pages of no sequence reach none.

Bit for bit: the other rows are what they are when those values are zeros.
"""
import pytest
import torch

from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
LENS = [700, 0, 33, 2500, 1, 17, 16, 300, 5, 31, 4000, 64]
SICK = [2, 4, 7]  # sequences whose tokens are made NaN


@pytest.fixture(autouse=True)
def _defaults(cuda_device):
    _lib.gqa_paged_decode_set_tuning(0, 0, 0, 0, 0, 0)
    yield
    _lib.gqa_paged_decode_set_tuning(0, 0, 0, 0, 0, 0)
    _lib.gqa_paged_decode_set_merge_mode(_lib.MERGE_KERNEL)


def pages(w):
    """(pages of the sick sequences and of no sequence, rows of the others)."""
    listed = torch.zeros(w.k_cache.shape[0], dtype=torch.bool)
    listed[w.kv_indices.long()] = True
    away = ~listed
    for b in SICK:
        away[w.kv_indices[w.kv_indptr[b]:w.kv_indptr[b + 1]].long()] = True
    rows = torch.ones(w.batch, dtype=torch.bool)
    rows[SICK] = False
    return away, rows


@pytest.mark.parametrize("mode", ["default", "one wave", "one head a CTA", "copies", "copies 32"])
def test_decode(mode):
    w = wl.make_workload(LENS, seed=71, pool_factor=1.3)
    away, rows = pages(w)
    tuning = {"one head a CTA": (0, 0, 1, 16, 4, 0), "copies": (0, 0, 4, 16, 5, 1), "copies 32": (0, 0, 4, 32, 3, 1)}
    assert _lib.gqa_paged_decode_set_tuning(*tuning.get(mode, (0, 0, 0, 0, 0, 0))) == 0
    if mode == "one wave":
        assert _lib.gqa_paged_decode_set_merge_mode(_lib.MERGE_ONE_WAVE) == 0
    got = []
    for value in (0.0, float("nan"), float("inf")):
        w.k_cache[away] = value
        w.v_cache[away] = value
        g = w.to("cuda")
        got.append([x[rows] for x in _lib.run(g.q, g.k_cache, g.v_cache, g.kv_indptr, g.kv_indices, w.sm_scale)])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1]) and out.isfinite().all()
    assert _lib.gqa_paged_decode_device_error() == 0


def test_decode_fp8():
    w = wl.make_fp8_workload(LENS, seed=72, pool_factor=1.3)
    away, rows = pages(w)
    got = []
    for code in (0, 0x7F):  # NaN codes, and scales of NaN bits
        w.k_cache[away] = code
        w.v_cache[away] = code
        if code:
            for c in (w.k_cache, w.v_cache):
                c[away, 512:] = torch.tensor([0, 0, 0xC0, 0x7F] * 4, dtype=torch.uint8)
        g = w.to("cuda")
        got.append([x[rows] for x in _lib.run_fp8(g.q, g.k_cache, g.v_cache, g.kv_indptr, g.kv_indices, w.sm_scale)])
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[1][0].isfinite().all()


@pytest.mark.parametrize("topk", [7, 16, 33, 256])
def test_selected_tokens(topk):
    """Rows in turn of request 0 and of request 1, whose blocks are NaN; columns of padding among the used ones."""
    g = torch.Generator().manual_seed(topk)
    bf, ps, blocks, rows = torch.bfloat16, 16, 40, 30
    kc, vc = (torch.randn(blocks, ps, 4, 128, generator=g).to(bf) for _ in range(2))
    table = torch.stack([torch.arange(1, 19), torch.arange(20, 38)]).to(torch.int32)
    req = (torch.arange(rows) % 2).to(torch.int32)
    idx = torch.randint(-60, 18 * ps, (rows, topk), generator=g, dtype=torch.int32)
    q = torch.randn(rows, 32, 128, generator=g).to(bf).cuda()
    got = []
    for value in (0.0, float("nan")):
        for c in (kc, vc):
            c[20:] = value
            c[0] = value
        out, lse = _lib.sparse_run(q, kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), req.cuda())
        got.append((out[0::2], lse[0::2]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[1][0].isfinite().all()


@pytest.mark.parametrize("kernel,h_q,ps", [(0, 32, 64), (1, 64, 32), (3, 16, 16), (4, 16, 1)])
def test_latent_decode(kernel, h_q, ps):
    w = wl.make_mla_workload(LENS, h_q, 1, ps, 73)
    assert _lib.gqa_mla_set_tuning(kernel) == 0
    try:
        away = torch.ones(w.kv_cache.shape[0], dtype=torch.bool)
        rows = torch.ones(w.batch, dtype=torch.bool)
        rows[SICK] = False
        for b in range(w.batch):
            if rows[b]:
                away[w.block_table[b, :-(-LENS[b] // ps)].long()] = False
        got = []
        for value in (0.0, float("nan")):
            w.kv_cache[away] = value
            g = w.to("cuda")
            out, lse = _lib.mla_run(g.q, g.kv_cache, g.block_table, g.cache_seqlens, w.softmax_scale)
            got.append((out[rows], lse[rows]))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and got[1][0].isfinite().all()
    finally:
        _lib.gqa_mla_set_tuning(0)
