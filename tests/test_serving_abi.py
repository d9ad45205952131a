"""Argument checks of the serving operators (no GPU): C entry points and tensor-level calls."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.serving as sv
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

A = 1 << 20  # a 256-byte aligned dummy address; no call below reaches the device
BAD = _lib.GQA_ERR_INVALID_ARGUMENT


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("scaling", [None, "linear", "base", "by_parts"])
def test_inv_freq(lib, rot, scaling):
    if scaling == "base" and rot == 2:
        return
    f, s = pkg.rope_inv_freq(rot, 500000.0, scaling, 1.0 if scaling is None else 8.0, 8192.0, 1.0, 32.0, device="cpu")
    want = sv.inv_freq_oracle(rot, 500000.0, scaling, 8.0, 8192.0)
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    assert math.isclose(s, 0.1 * math.log(8.0) + 1 if scaling == "by_parts" else 1.0, rel_tol=1e-6)


def test_inv_freq_refusals(lib):
    buf, s = (ctypes.c_double * 64)(), ctypes.c_float()
    ok = [64, 1e4, 3, 4.0, 4096.0, 1.0, 32.0, ctypes.addressof(buf), ctypes.byref(s)]
    assert lib.gqa_rope_inv_freq(*ok) == 0
    for i, bad in ((0, 0), (0, 63), (0, 1026), (1, 0.0), (1, -1.0), (1, math.inf), (1, math.nan), (2, -1), (2, 4),
                   (3, 0.5), (3, math.nan), (3, math.inf), (4, 0.0), (5, -1.0), (6, 1.0), (6, math.inf), (7, None)):
        args = list(ok)
        args[i] = bad
        assert lib.gqa_rope_inv_freq(*args) == BAD, (i, bad)
    assert lib.gqa_rope_inv_freq(2, 1e4, 2, 4.0, 0.0, 0.0, 0.0, ctypes.addressof(buf), None) == BAD
    assert lib.gqa_rope_inv_freq(64, 1e4, 0, 0.0, 0.0, 0.0, 0.0, ctypes.addressof(buf), None) == 0
    with pytest.raises(ValueError):
        pkg.rope_inv_freq(64, scaling="other", device="cpu")
    with pytest.raises(pkg.GqaError):
        pkg.rope_inv_freq(7, device="cpu")


def _refused(fn, ok, cases):
    for changes in cases:
        args = dict(ok, **changes)
        assert fn(*args.values()) == BAD, changes


def test_rope_refusals(lib):
    ok = dict(x=A, positions=A, inv_freq=A, scale=1.0, out=A + 4096, n=4, heads=3, dim=128, offset=0, rot=128, layout=0,
              inverse=0, dtype=0, xt=384, xh=128, ot=384, oh=128, stream=None)
    assert lib.gqa_rope(*dict(ok, n=0, x=None).values()) == 0
    _refused(lib.gqa_rope, ok, [
        dict(n=-1), dict(x=None), dict(out=None), dict(positions=None), dict(inv_freq=None), dict(scale=math.nan),
        dict(scale=math.inf), dict(heads=0), dict(heads=1025), dict(dim=0), dict(dim=1025), dict(rot=0), dict(rot=7),
        dict(rot=130), dict(offset=-2), dict(offset=2), dict(offset=2 ** 31 - 1), dict(layout=2), dict(layout=-1),
        dict(dtype=3), dict(dtype=-1), dict(x=A + 1), dict(dtype=2, x=A + 2), dict(out=A + 1), dict(positions=A + 2),
        dict(inv_freq=A + 4), dict(xt=-1), dict(oh=127), dict(ot=383), dict(ot=0)])


def test_append_refusals(lib):
    ok = dict(q=A, k=A, v=A, positions=A, slots=A, freq=A, scale=1.0, offset=0, rot=128, layout=0, q_out=A, kc=A, vc=A,
              fmt=1, n=3, pages=9, qs=4096, ks=512, vs=512, stream=None)
    assert lib.gqa_rope_kv_append(*dict(ok, n=0, k=None).values()) == 0
    _refused(lib.gqa_rope_kv_append, ok, [
        dict(n=-1), dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(pages=0), dict(q=None),
        dict(q_out=None), dict(positions=None), dict(scale=math.nan), dict(rot=0), dict(rot=3), dict(offset=1), dict(offset=-1),
        dict(layout=5), dict(fmt=2), dict(fmt=-1), dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(q_out=A + 8),
        dict(kc=A + 8), dict(vc=A + 8), dict(slots=A + 2), dict(qs=4095), dict(qs=4100), dict(ks=511), dict(vs=516)])
    ok = dict(k=A, v=A, slots=A, kc=A, vc=A, n=3, pages=9, stream=None)
    assert lib.gqa_paged_kv_append_fp8(*dict(ok, n=0).values()) == 0
    _refused(lib.gqa_paged_kv_append_fp8, ok, [dict(n=-1), dict(k=None), dict(vc=None), dict(pages=0), dict(v=A + 8)])
    ok = dict(kc=A, vc=A, idx=A, ko=A, vo=A, n=3, pages=9, stream=None)
    assert lib.gqa_paged_kv_read_fp8(*dict(ok, n=0, kc=None).values()) == 0
    _refused(lib.gqa_paged_kv_read_fp8, ok, [dict(n=-1), dict(kc=None), dict(idx=None), dict(ko=None), dict(pages=0),
                                             dict(kc=A + 8), dict(vo=A + 8), dict(idx=A + 1)])


def test_latent_refusals(lib):
    ok = dict(lat=A, kr=A, positions=A, slots=A, freq=A, scale=1.0, layout=1, kv=A, n=3, nslots=64, ls=576, rs=576,
              stream=None)
    assert lib.gqa_mla_kv_append(*dict(ok, n=0, lat=None).values()) == 0
    _refused(lib.gqa_mla_kv_append, ok, [
        dict(n=-1), dict(lat=None), dict(kr=None), dict(slots=None), dict(kv=None), dict(nslots=0), dict(positions=None),
        dict(layout=2), dict(scale=math.inf), dict(lat=A + 8), dict(kr=A + 2), dict(kv=A + 8), dict(ls=511), dict(ls=514),
        dict(rs=63), dict(rs=65)])
    ok = dict(q=A, w=A, positions=A, freq=A, scale=1.0, layout=1, out=A, n=3, heads=5, qt=960, qh=192, stream=None)
    assert lib.gqa_mla_absorb_q(*dict(ok, n=0, q=None).values()) == 0
    _refused(lib.gqa_mla_absorb_q, ok, [
        dict(n=-1), dict(n=(1 << 20) + 1), dict(q=None), dict(w=None), dict(out=None), dict(heads=0), dict(heads=1025),
        dict(positions=None), dict(layout=9), dict(q=A + 2), dict(w=A + 8), dict(out=A + 8), dict(qt=191), dict(qh=196)])
    ok = dict(o=A, w=A, out=A, n=3, heads=5, stream=None)
    assert lib.gqa_mla_expand_out(*dict(ok, n=0, o=None).values()) == 0
    _refused(lib.gqa_mla_expand_out, ok, [dict(n=-1), dict(o=None), dict(w=None), dict(out=None), dict(heads=0),
                                          dict(heads=1025), dict(o=A + 8), dict(out=A + 2)])


def test_prefill_refusals(lib):
    ok = dict(q=A, w=A, kv=A, table=A, lens=A, cu=A, scale=0.1, causal=1, out=A, lse=A, batch=2, total=7, heads=3, page=16,
              blocks=9, width=4, max_kv=100, qt=576, qh=192, ws=A, ws_bytes=1 << 40, stream=None)
    assert lib.gqa_mla_prefill(*dict(ok, batch=0).values()) == 0
    assert lib.gqa_mla_prefill(*dict(ok, total=0, q=None).values()) == 0
    _refused(lib.gqa_mla_prefill, ok, [
        dict(batch=-1), dict(total=-1), dict(q=None), dict(w=None), dict(kv=None), dict(table=None), dict(lens=None),
        dict(cu=None), dict(out=None), dict(scale=math.nan), dict(scale=3e38), dict(heads=0), dict(heads=1025), dict(page=0), dict(blocks=0),
        dict(width=0), dict(max_kv=-1), dict(max_kv=1 << 31), dict(blocks=1 << 26, page=64), dict(width=1 << 26, page=64),
        dict(q=A + 8), dict(w=A + 8), dict(kv=A + 2), dict(out=A + 8), dict(lse=A + 2), dict(table=A + 1), dict(qt=191),
        dict(qt=580), dict(qh=100)])
    for bad in (dict(ws=None), dict(ws=A + 128), dict(ws_bytes=0)):
        assert lib.gqa_mla_prefill(*dict(ok, **bad).values()) == _lib.GQA_ERR_WORKSPACE
    size = lib.gqa_mla_prefill_ws_size(2, 3, 100)
    assert size > 0
    assert lib.gqa_mla_prefill(*dict(ok, ws_bytes=size - 1).values()) == _lib.GQA_ERR_WORKSPACE
    assert lib.gqa_mla_prefill_ws_size(2, 3, 0) > 0
    for bad in ((0, 3, 100), (2, 0, 100), (2, 3, -1), (2, 1025, 100), (2, 3, 1 << 31)):
        assert lib.gqa_mla_prefill_ws_size(*bad) == 0
    # the expanded keys and values of one pass are bounded, whatever the head count
    assert lib.gqa_mla_prefill_ws_size(1, 128, 1 << 20) < (8 << 30)


def test_prefill_fill_refusals(lib):
    ok = dict(q=A, w=A, kv=A, table=A, lens=A, cu=A, scale=0.1, causal=1, fill=3, out=A, lse=A, batch=2, total=7, heads=3,
              page=16, blocks=9, width=4, max_kv=100, qt=576, qh=192, ws=A, ws_bytes=1 << 40, stream=None)
    assert lib.gqa_mla_prefill_fill(*dict(ok, batch=0).values()) == 0
    _refused(lib.gqa_mla_prefill_fill, ok, [dict(fill=-1), dict(fill=4), dict(fill=2, lse=None), dict(q=None), dict(width=0)])
    assert lib.gqa_mla_prefill_fill(*dict(ok, ws=None).values()) == _lib.GQA_ERR_WORKSPACE


def test_cpu_tensors_raise(lib):
    bf = torch.bfloat16
    i = torch.zeros(2, dtype=torch.int32)
    f, _ = pkg.rope_inv_freq(64, device="cpu")
    f128, _ = pkg.rope_inv_freq(128, device="cpu")
    k, c = torch.zeros(2, 4, 128, dtype=bf), torch.zeros(8, 528, dtype=torch.uint8)
    w, lat = torch.zeros(16, 256, 512, dtype=bf), torch.zeros(4, 16, 1, 576, dtype=bf)
    calls = [lambda: pkg.rope(torch.zeros(2, 3, 64, dtype=bf), i, f),
             lambda: pkg.rope_kv_append(torch.zeros(2, 32, 128, dtype=bf), k, k, i, c, c, i, f128),
             lambda: pkg.kv_append_fp8(k, k, i, c, c),
             lambda: pkg.kv_read_fp8(c, c, i),
             lambda: pkg.mla_kv_append(torch.zeros(2, 512, dtype=bf), torch.zeros(2, 64, dtype=bf), i, lat),
             lambda: pkg.mla_absorb_q(torch.zeros(2, 16, 192, dtype=bf), w),
             lambda: pkg.mla_expand_out(torch.zeros(2, 16, 512, dtype=bf), w),
             lambda: pkg.mla_prefill(torch.zeros(2, 16, 192, dtype=bf), w, lat, torch.zeros(1, 4, dtype=torch.int32),
                                     i[:1], i)]
    for call in calls:
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def test_rope_in_place_needs_the_same_strides(lib):
    ok = dict(x=A, positions=A, inv_freq=A, scale=1.0, out=A, n=4, heads=3, dim=128, offset=0, rot=128, layout=0,
              inverse=0, dtype=0, xt=384, xh=128, ot=384, oh=128, stream=None)
    _refused(lib.gqa_rope, ok, [dict(ot=512, oh=128), dict(ot=128, oh=512), dict(xt=512), dict(n=1, xh=256),
                                dict(heads=1, xt=512)])
