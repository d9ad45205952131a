"""The decode's forms for long and shared contexts together on one cache, as a serving step runs them, and what their
tensor-level calls refuse."""
import numpy as np
import pytest
import torch

import oracle.context as cx
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def i32(x):
    return torch.tensor(x, dtype=I32).cuda()


def within(out, lse, want, fp8=False):
    o, l = cx.f64(out), cx.f64(lse)
    for b, a in enumerate(want):
        assert np.all(np.abs(o[b] - a.out) <= a.out_bound(fp8)), b
        assert np.all(np.abs(l[b] - a.lse) <= a.lse_bound()), b


def test_steps_on_one_cache():
    """Three requests behind one prefix: each step stores its tokens, renews the bounds and decodes in all four forms. The
    blocks of the block table are 16 pages each of the page tables."""
    g = torch.Generator().manual_seed(0)
    blocks, prefix, own = 40, 160, [33, 5, 70]
    k, v = (torch.randn(blocks * PAGE, 1, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    kb, vb = (x.view(blocks, PAGE, 4, 128) for x in (k, v))
    table = torch.randperm(blocks, generator=g)[:10 + 3 * 8].tolist()
    tables = i32([table[:10] + table[10 + 8 * r:18 + 8 * r] for r in range(3)])
    page_of = lambda r, t: int(tables[r, t // PAGE]) * PAGE + t % PAGE  # noqa: E731
    bounds = torch.zeros(blocks, 2, 4, 128, dtype=BF, device="cuda")
    pkg.block_bounds(kb, bounds, tables, i32([prefix + n for n in own]))
    freq, _ = pkg.rope_inv_freq(128)
    weights = torch.zeros(3, 400, device="cuda")
    for step in range(3):
        q, kn, vn = (torch.randn(3, h, 128, generator=g).to(BF).cuda() for h in (32, 4, 4))
        lens = [prefix + n for n in own]
        slots = i32([page_of(r, n) for r, n in enumerate(lens)])
        q = pkg.rope_kv_append(q, kn, vn, slots, k, v, i32(lens), freq)
        first, lens = i32(lens), [n + 1 for n in lens]
        own = [n + 1 for n in own]
        pkg.block_bounds(kb, bounds, tables, i32(lens), first)
        assert np.array_equal(cx.f64(bounds), cx.bounds_oracle(kb, bounds, tables, i32(lens)))
        pages = [[page_of(r, t) for t in range(n)] for r, n in enumerate(lens)]
        indptr = i32(np.concatenate([[0], np.cumsum(lens)]))
        whole = [cx.Attended(q[r], cx.rows64(k, pages[r]), cx.rows64(v, pages[r]), 128 ** -0.5) for r in range(3)]
        # one prefix for all, and each one's own
        within(*pkg.shared_run(q, k, v, i32([0, prefix]), i32(pages[0][:prefix]), i32([0, 3]),
                               i32(np.concatenate([[0], np.cumsum(own)])), i32(sum((p[prefix:] for p in pages), []))), whole)
        # all blocks, then some
        rows = i32([0, 1, 2])
        within(*pkg.block_sparse_run(q, kb, vb, pkg.block_select(q, bounds, tables, rows, i32(lens), 20, PAGE), tables, rows,
                                     i32(lens)), whole)
        some = pkg.block_select(q, bounds, tables, rows, i32(lens), 6, PAGE)
        assert np.array_equal(some.cpu().numpy(), cx.select_oracle(q, bounds, tables, rows, i32(lens), 6, PAGE, 1, 1))
        within(*pkg.block_sparse_run(q, kb, vb, some, tables, rows, i32(lens)),
               cx.block_sparse_oracle(q, kb, vb, some, tables, rows, i32(lens), 128 ** -0.5))
        # weights, and what an eviction by them would leave
        args = (q, k, v, indptr, i32(sum(pages, [])), weights)
        _, new, bound = cx.weighted_oracle(*args, 0.9, 128 ** -0.5)
        out, lse, weights = pkg.run_weighted(*args, decay=0.9)
        within(out, lse, whole)
        assert np.all(np.abs(cx.f64(weights) - new) <= bound)
        left = pkg.kv_evict(weights, indptr, args[4], 120, keep_first=4, keep_last=16)
        for a, b in zip(left, cx.evict_oracle(weights, indptr, args[4], 120, 4, 16)):
            assert np.array_equal(a.cpu().numpy(), b)
    assert _lib.gqa_paged_decode_device_error() == 0


def tensors():
    z = lambda *s, d=BF: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    return dict(q=z(2, 32, 128), k=z(9, 1, 4, 128), v=z(9, 1, 4, 128), pi=z(2, d=I32), px=z(4, d=I32), gi=z(2, d=I32),
                ki=z(3, d=I32), kx=z(5, d=I32), kb=z(3, 4, 4, 128), vb=z(3, 4, 4, 128), b=z(3, 2, 4, 128), t=z(2, 3, d=I32),
                l=z(2, d=I32), r=z(2, d=I32), s=z(2, 4, 3, d=I32), w=z(2, 8, d=torch.float32), f=z(9, 528, d=torch.uint8))


CALLS = {
    "shared": lambda a, **m: pkg.shared_run(a["q"], a["k"], a["v"], a["pi"], a["px"], a["gi"], a["ki"], a["kx"], **m),
    "bounds": lambda a, **m: pkg.block_bounds(a["kb"], a["b"], a["t"], a["l"], **m),
    "select": lambda a, **m: pkg.block_select(a["q"], a["b"], a["t"], a["r"], a["l"], **dict(dict(top=3, page_size=4), **m)),
    "sparse": lambda a, **m: pkg.block_sparse_run(a["q"], a["kb"], a["vb"], a["s"], a["t"], a["r"], a["l"], **m),
    "weighted": lambda a, **m: pkg.run_weighted(a["q"], a["k"], a["v"], a["ki"], a["kx"], a["w"], **m),
    "evict": lambda a, **m: pkg.kv_evict(a["w"], a["ki"], a["kx"], **dict(dict(budget=2), **m)),
}
USES = {"shared": "q k v pi px gi ki kx", "bounds": "kb b t l", "select": "q b t r l", "sparse": "q kb vb s t r l",
        "weighted": "q k v ki kx w", "evict": "w ki kx"}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_refusals_of_tensors(name):
    """Every tensor: on the CPU, of another type, not contiguous, of another shape, and no tensor at all."""
    call, good = CALLS[name], tensors()
    call(good)
    for key in USES[name].split():
        t = good[key]
        if t.dtype == I32 and t.dim() == 1:
            shapes = [t.view(1, -1)] + ([] if key in ("px", "kx") else [t[:-1], torch.cat([t, t])])
        else:
            shapes = [t[None], t[..., :-1].contiguous()]
        if name == "evict" and key == "w":
            shapes.pop()  # any width will do
        if name == "weighted" and key == "w":
            shapes.pop()
        if name == "sparse" and key == "s":
            shapes.pop()  # any number of blocks
        if key == "t":
            shapes[1] = t[0]
        strided = torch.stack([t, t], -1)[..., 0]
        for bad in [t.cpu(), t.to(torch.float64 if t.dtype != torch.float64 else BF), strided, *shapes]:
            with pytest.raises(ValueError):
                call(dict(good, **{key: bad}))
        with pytest.raises(TypeError):
            call(dict(good, **{key: [1, 2]}))


def test_refusals_of_numbers_and_outputs():
    a = tensors()
    f32 = torch.float32
    bad_out, bad_lse = torch.zeros(3, 32, 128, dtype=BF, device="cuda"), torch.zeros(2, 31, dtype=f32, device="cuda")
    for name in ("shared", "sparse", "weighted"):
        for more in (dict(out=bad_out), dict(lse=bad_lse), dict(out=torch.zeros(2, 32, 128, dtype=f32, device="cuda"))):
            with pytest.raises(ValueError):
                CALLS[name](a, **more)
        for scale in (float("nan"), float("inf"), 3e38):
            with pytest.raises(pkg.GqaError):
                CALLS[name](a, sm_scale=scale)
        with pytest.raises(pkg.GqaError):
            CALLS[name](a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    for more in (dict(top=0), dict(top=2 ** 31), dict(page_size=0), dict(keep_first=-1), dict(keep_first=3), dict(keep_last=4),
                 dict(blocks=torch.zeros(2, 4, 2, dtype=I32, device="cuda"))):
        with pytest.raises(ValueError):
            CALLS["select"](a, **more)
    with pytest.raises(pkg.GqaError):
        CALLS["select"](a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    for more in (dict(budget=-1), dict(budget=2 ** 31), dict(keep_first=3), dict(keep_first=1, keep_last=2), dict(keep_last=-1)):
        with pytest.raises(ValueError):
            CALLS["evict"](a, **more)
    for more in (dict(decay=float("nan")), dict(decay=float("inf")), dict(weights_out=torch.zeros(2, 9, device="cuda"))):
        with pytest.raises(ValueError):
            CALLS["weighted"](a, **more)
    with pytest.raises(ValueError):
        CALLS["bounds"](a, first=torch.zeros(3, dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        pkg.shared_run(a["q"], a["k"], a["f"], a["pi"], a["px"], a["gi"], a["ki"], a["kx"])


def test_empty_batches():
    a = tensors()
    none = dict(a, q=a["q"][:0], ki=a["ki"][:1], l=a["l"][:0], r=a["r"][:0], t=a["t"][:0], s=a["s"][:0], w=a["w"][:0])
    out, lse = CALLS["shared"](none)
    assert out.shape == (0, 32, 128) and lse.shape == (0, 32)
    CALLS["bounds"](none)
    none["t"] = a["t"]
    assert CALLS["select"](none).shape == (0, 4, 3)
    assert CALLS["sparse"](none)[0].shape == (0, 32, 128)
    assert CALLS["weighted"](none)[2].shape == (0, 8)
    got = CALLS["evict"](none)
    assert torch.equal(got[2], torch.full((5,), -1, dtype=I32, device="cuda")) and torch.equal(got[4], got[2])


@pytest.mark.parametrize("name", sorted(CALLS))
def test_without_the_look_in_one_step(name, monkeypatch):
    """The same results and refusals where the C++ step is not there."""
    from paged_kv_gqa_split_gb300 import context

    g, a = torch.Generator().manual_seed(9), tensors()
    for key in ("q", "k", "v", "kb", "vb", "b", "w"):
        a[key].copy_(torch.randn(a[key].shape, generator=g).to(a[key].dtype))
    for key, values in dict(pi=[0, 4], px=[1, 2, 3, 4], gi=[0, 2], ki=[0, 2, 5], kx=[5, 6, 7, 8, 0], l=[4, 12]).items():
        a[key].copy_(torch.tensor(values, dtype=I32))
    a["t"].copy_(torch.tensor([[0, 1, 2], [2, 1, 0]], dtype=I32))
    fast = CALLS[name](a)
    fast = [x.clone() for x in (fast if isinstance(fast, tuple) else (fast,))]
    monkeypatch.setattr(context, "_gather", context._no_gather)
    slow = CALLS[name](a)
    for x, y in zip(fast, slow if isinstance(slow, tuple) else (slow,)):
        assert torch.equal(x, y)
    for key in USES[name].split():
        for bad in (a[key].cpu(), a[key][None]):
            with pytest.raises(ValueError):
                CALLS[name](dict(a, **{key: bad}))


def test_fp8_rows_of_more_dimensions():
    """FP8 caches [P, 1, 528] as the plain decode takes them."""
    a, f = tensors(), torch.zeros(9, 1, 528, dtype=torch.uint8, device="cuda")
    flat = dict(a, k=f.view(9, 528), v=f.view(9, 528))
    for name in ("shared", "weighted"):
        for x, y in zip(CALLS[name](dict(a, k=f, v=f)), CALLS[name](flat)):
            assert torch.equal(x, y)
