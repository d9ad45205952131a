"""Argument checks of the decode's forms for long and shared contexts (no GPU), and their oracle against brute force."""
import math

import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib, context
from paged_kv_gqa_split_gb300.build import build

A = 1 << 20  # a 256-byte aligned dummy address; no call below reaches the device
BAD, SPACE = _lib.GQA_ERR_INVALID_ARGUMENT, _lib.GQA_ERR_WORKSPACE
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def refused(fn, ok, cases, code=BAD):
    for changes in cases:
        assert set(changes) <= set(ok), changes
        assert fn(*dict(ok, **changes).values()) == code, changes


def test_shared_refusals(lib):
    ok = dict(q=A, k=A, v=A, pi=A, px=A, gi=A, ki=A, kx=A, scale=0.1, out=A, lse=A, batch=3, groups=2, pn=9, n=5, pages=20,
              fmt=0, ws=A, size=1 << 40, stream=None)
    assert lib.gqa_shared_paged_decode(*dict(ok, batch=0, q=None).values()) == 0
    refused(lib.gqa_shared_paged_decode, ok, [
        dict(batch=-1), dict(batch=(1 << 20) + 1), dict(groups=-1), dict(groups=(1 << 20) + 1), dict(pn=-1), dict(n=-1),
        dict(pages=-1), dict(fmt=2), dict(fmt=-1), dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38), dict(q=None),
        dict(out=None), dict(ki=None), dict(pi=None), dict(gi=None), dict(px=None), dict(kx=None), dict(k=None), dict(v=None),
        dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(out=A + 8), dict(lse=A + 4), dict(pi=A + 1), dict(px=A + 2),
        dict(gi=A + 2), dict(ki=A + 2), dict(kx=A + 1)])
    refused(lib.gqa_shared_paged_decode, ok, [dict(ws=None), dict(ws=A + 128)], SPACE)
    for bad in ((0, 1, 0), (-1, 1, 0), ((1 << 20) + 1, 1, 0), (3, -1, 0), (3, 1, 2)):
        assert lib.gqa_shared_paged_decode_ws_size(*bad) == 0


def test_bounds_refusals(lib):
    ok = dict(k=A, bounds=A, table=A, lens=A, first=A, requests=3, page=16, blocks=9, width=4, stream=None)
    assert lib.gqa_block_bounds(*dict(ok, requests=0, k=None).values()) == 0
    refused(lib.gqa_block_bounds, ok, [
        dict(requests=-1), dict(page=0), dict(blocks=0), dict(width=0), dict(blocks=1 << 28), dict(width=1 << 28), dict(k=None),
        dict(bounds=None), dict(table=None), dict(lens=None), dict(k=A + 8), dict(bounds=A + 2), dict(table=A + 2),
        dict(lens=A + 1), dict(first=A + 2)])


def test_select_refusals(lib):
    ok = dict(q=A, bounds=A, table=A, req=A, lens=A, out=A, rows=3, requests=2, page=16, blocks=9, width=4, top=5, first=1,
              last=2, ws=A, size=1 << 40, stream=None)
    assert lib.gqa_block_select(*dict(ok, rows=0, q=None).values()) == 0
    refused(lib.gqa_block_select, ok, [
        dict(rows=-1), dict(requests=0), dict(page=0), dict(blocks=0), dict(width=0), dict(blocks=1 << 28), dict(width=1 << 28),
        dict(top=0), dict(top=-1), dict(first=-1), dict(last=-1), dict(first=6), dict(first=3, last=3), dict(first=BIG, last=BIG),
        dict(last=BIG), dict(rows=1 << 20, top=1 << 20), dict(q=None), dict(bounds=None), dict(table=None), dict(req=None),
        dict(lens=None), dict(out=None), dict(q=A + 8), dict(bounds=A + 8), dict(table=A + 1), dict(req=A + 2), dict(lens=A + 2),
        dict(out=A + 2)])
    refused(lib.gqa_block_select, ok, [dict(ws=None), dict(ws=A + 64), dict(size=0)], SPACE)
    size = lib.gqa_block_select_ws_size(3, 4)
    assert size > 0
    refused(lib.gqa_block_select, ok, [dict(size=size - 1)], SPACE)
    for bad in ((0, 4), (3, 0), (-1, 4), (BIG, BIG)):
        assert lib.gqa_block_select_ws_size(*bad) == 0


def test_block_decode_refusals(lib):
    ok = dict(q=A, k=A, v=A, blocks=A, table=A, req=A, lens=A, scale=0.1, out=A, lse=None, rows=3, requests=2, top=5, page=16,
              held=9, width=4, ws=A, size=1 << 40, stream=None)
    assert lib.gqa_block_sparse_decode(*dict(ok, rows=0, q=None).values()) == 0
    refused(lib.gqa_block_sparse_decode, ok, [
        dict(rows=-1), dict(requests=0), dict(top=0), dict(page=0), dict(held=0), dict(width=0), dict(held=1 << 28),
        dict(width=1 << 28), dict(rows=1 << 16, top=1 << 16), dict(top=BIG, page=BIG), dict(scale=math.nan), dict(scale=3e38),
        dict(q=None), dict(k=None), dict(v=None), dict(blocks=None), dict(table=None), dict(req=None), dict(lens=None),
        dict(out=None), dict(q=A + 8), dict(k=A + 8), dict(v=A + 8), dict(out=A + 8), dict(lse=A + 4), dict(blocks=A + 2),
        dict(table=A + 2), dict(req=A + 2), dict(lens=A + 2)])
    refused(lib.gqa_block_sparse_decode, ok, [dict(ws=None), dict(ws=A + 128)], SPACE)
    for bad in ((0, 5, 16), (3, 0, 16), (3, 5, 0), (1 << 16, 1 << 16, 1)):
        assert lib.gqa_block_sparse_decode_ws_size(*bad) == 0


def test_weighted_refusals(lib):
    ok = dict(q=A, k=A, v=A, ki=A, kx=A, scale=0.1, w=A, decay=1.0, wo=A, out=A, lse=A, batch=3, width=7, n=5, pages=20, fmt=1,
              ws=A, size=1 << 40, stream=None)
    assert lib.gqa_paged_decode_weighted(*dict(ok, batch=0, q=None).values()) == 0
    refused(lib.gqa_paged_decode_weighted, ok, [
        dict(batch=-1), dict(width=-1), dict(n=-1), dict(pages=-1), dict(fmt=2), dict(scale=math.inf), dict(scale=3e38),
        dict(decay=math.nan), dict(decay=math.inf), dict(q=None), dict(k=None), dict(v=None), dict(ki=None), dict(kx=None),
        dict(w=None), dict(wo=None), dict(out=None), dict(lse=None), dict(q=A + 8), dict(k=A + 8), dict(v=A + 8),
        dict(out=A + 8), dict(lse=A + 4), dict(w=A + 2), dict(wo=A + 1), dict(ki=A + 2), dict(kx=A + 2)])
    refused(lib.gqa_paged_decode_weighted, ok, [dict(ws=None), dict(ws=A + 128)], SPACE)
    for bad in ((-1, 0), (5, 2), (5, -1)):
        assert lib.gqa_paged_decode_weighted_ws_size(*bad) == 0


def test_evict_refusals(lib):
    ok = dict(w=A, ki=A + 4096, kx=A + 8192, budget=9, first=2, last=3, wo=A + 4, ni=A + 8, nx=A + 12, fi=A + 16, fx=A + 20,
              batch=3, width=7, n=5, stream=None)
    assert lib.gqa_kv_evict(*dict(ok, batch=0, w=None).values()) == 0
    refused(lib.gqa_kv_evict, ok, [
        dict(batch=-1), dict(width=-1), dict(n=-1), dict(budget=-1), dict(first=-1), dict(last=-1), dict(first=10),
        dict(first=5, last=5), dict(first=BIG, last=BIG, budget=BIG), dict(w=None), dict(ki=None), dict(kx=None), dict(wo=None),
        dict(ni=None), dict(nx=None), dict(fi=None), dict(fx=None), dict(wo=A), dict(nx=A + 8192), dict(fx=A + 8192),
        dict(fx=A + 12), dict(ni=A + 4096), dict(fi=A + 4096), dict(fi=A + 8), dict(w=A + 2), dict(kx=A + 8193), dict(ni=A + 9)])


def test_counts_past_what_the_kernels_walk_are_refused(lib):
    most = 1 << 30
    ok = dict(q=A, k=A, v=A, pi=A, px=A, gi=A, ki=A, kx=A, scale=0.1, out=A, lse=A, batch=3, groups=2, pn=9, n=5, pages=20,
              fmt=0, ws=A, size=0, stream=None)
    refused(lib.gqa_shared_paged_decode, ok, [dict(pn=most + 1), dict(n=most + 1), dict(n=BIG)])
    ok = dict(k=A, bounds=A, table=A, lens=A, first=A, requests=3, page=1, blocks=9, width=4, stream=None)
    refused(lib.gqa_block_bounds, ok, [dict(requests=most + 1), dict(width=most + 1), dict(width=BIG)])
    ok = dict(q=A, k=A, v=A, ki=A, kx=A, scale=0.1, w=A, decay=1.0, wo=A, out=A, lse=A, batch=3, width=7, n=5, pages=20, fmt=1,
              ws=A, size=0, stream=None)
    refused(lib.gqa_paged_decode_weighted, ok, [dict(width=BIG), dict(width=most + 1), dict(n=most + 1), dict(batch=most + 1)])
    assert lib.gqa_paged_decode_weighted_ws_size(most + 1, 0) == 0 and lib.gqa_block_select_ws_size(1, most + 1) == 0
    ok = dict(w=A, ki=A + 4096, kx=A + 8192, budget=9, first=2, last=3, wo=A + 4, ni=A + 8, nx=A + 12, fi=A + 16, fx=A + 20,
              batch=3, width=7, n=5, stream=None)
    refused(lib.gqa_kv_evict, ok, [dict(width=BIG), dict(n=most + 1), dict(batch=most + 1)])
    context._fit(BIG, 0)
    with pytest.raises(ValueError, match="entries"):
        context._fit(3, BIG + 1)


def test_cpu_tensors_raise(lib):
    bf, i = torch.bfloat16, torch.zeros(3, dtype=torch.int32)
    q, c, f = torch.zeros(2, 32, 128, dtype=bf), torch.zeros(5, 1, 4, 128, dtype=bf), torch.zeros(5, 528, dtype=torch.uint8)
    b, t = torch.zeros(5, 2, 4, 128, dtype=bf), torch.zeros(2, 4, dtype=torch.int32)
    w = torch.zeros(2, 8)
    calls = [lambda: pkg.shared_run(q, c, c, i, i, i, i, i), lambda: pkg.shared_run(q, f, f, i, i, i, i, i),
             lambda: pkg.block_bounds(c, b, t, i[:2]), lambda: pkg.block_select(q, b, t, i[:2], i[:2], 3, 1),
             lambda: pkg.block_sparse_run(q, c, c, torch.zeros(2, 4, 3, dtype=torch.int32), t, i[:2], i[:2]),
             lambda: pkg.run_weighted(q, c, c, i, i, w), lambda: pkg.kv_evict(w, i, i, 2)]
    for call in calls:
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def test_the_look_at_tensors_in_one_step(lib):
    host = pytest.importorskip("paged_kv_gqa_split_gb300._context_host")
    assert host.gather(b"f1", torch.zeros(3)) is None and host.gather(b"x1", torch.zeros(3)) is None
    assert host.gather(b"f1", [0.0]) is None
    for bad in ((), (b"f1",), (b"f", torch.zeros(3)), (b"f1f1", torch.zeros(3)), ("f1", torch.zeros(3)), (b"f1" * 17, *[torch.zeros(1)] * 17)):
        with pytest.raises(TypeError):
            host.gather(*bad)
    assert host.torch_version == torch.__version__.split("+")[0]


def test_names_are_exported():
    for name in ("shared_run", "block_bounds", "block_select", "block_sparse_run", "run_weighted", "kv_evict"):
        assert name in pkg.__all__ and callable(getattr(pkg, name))


# ------------------------------------------------------------------ the oracle
def test_oracle_attention_against_sums_in_order():
    g = torch.Generator().manual_seed(0)
    q, k, v = torch.randn(32, 128, generator=g), torch.randn(5, 4, 128, generator=g), torch.randn(5, 4, 128, generator=g)
    a = cx.Attended(q, cx.f64(k), cx.f64(v), 0.3)
    for h in (0, 7, 8, 31):
        s = [0.3 * sum(float(q[h, d]) * float(k[t, h // 8, d]) for d in range(128)) for t in range(5)]
        z = sum(math.exp(x) for x in s)
        assert math.isclose(a.lse[h], math.log2(z), rel_tol=1e-12)
        for d in (0, 77):
            assert math.isclose(a.out[h, d], sum(math.exp(x) / z * float(v[t, h // 8, d]) for t, x in enumerate(s)), abs_tol=1e-12)


def test_oracle_selection_bounds_every_key():
    g = torch.Generator().manual_seed(1)
    k = torch.randn(6, 4, 4, 128, generator=g).to(torch.bfloat16)
    table, lens = torch.tensor([[3, 0, 5, 1]], dtype=torch.int32), [14]
    bounds = torch.tensor(cx.bounds_oracle(k, torch.zeros(6, 2, 4, 128), table, lens))
    q = torch.randn(1, 32, 128, generator=g)
    order = []
    for i, block in enumerate([3, 0, 5, 1]):
        hi, lo = bounds[block]
        best = max(float((torch.clamp(q[0, h].double(), min=0) * hi[1] + torch.clamp(q[0, h].double(), max=0) * lo[1]).sum())
                   for h in range(8, 16))
        for t in range(4 if i < 3 else 2):
            for h in range(8, 16):
                assert float((q[0, h].double() * k[block, t, 1].double()).sum()) <= best + 1e-9
        order.append((-best, i))
    got = cx.select_oracle(q, bounds, table, [0], lens, 2, 4, 0, 0)
    assert list(got[0, 1]) == sorted(i for _, i in sorted(order)[:2])


def test_oracle_eviction_by_hand():
    w = torch.tensor([[5.0, 1.0, 9.0, 1.0, 0.0, 7.0], [1.0, 2.0, 0.0, 0.0, 0.0, 0.0]])
    got = cx.evict_oracle(w, [0, 6, 8], [10, 11, 12, 13, 14, 15, 20, 21], 4, 1, 1)
    assert got[0].tolist() == [[5, 1, 9, 7, 0, 0], [1, 2, 0, 0, 0, 0]]
    assert got[1].tolist() == [0, 4, 6] and got[2].tolist() == [10, 11, 12, 15, 20, 21, -1, -1]
    assert got[3].tolist() == [0, 2, 2] and got[4].tolist() == [13, 14] + [-1] * 6


def test_chained_kernels_use_no_noncoherent_load():
    """Kernels that start before the ones ahead of them end read with ld.cg or plain loads (source check): the
    non-coherent load may be moved ahead of the wait."""
    import os
    import re
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_split_gb300", "csrc")
    for name in ("gqa_shared.cu", "gqa_blocks.cu", "gqa_weights.cu", "gqa_select.cuh"):
        with open(os.path.join(src, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "__ldg(" not in text and "__restrict__" not in text, name
        for body in re.split(r"__global__", text)[1:]:
            assert "pdl_wait();" in body.split("launch_chained")[0], name
