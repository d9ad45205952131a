"""GPU parity of the rotary positions against the float64 definition.

Bound: the angle's fraction of a turn is cut to 2^-33 and its float to 2^-25 of a half turn (pi 2^-25 radians), sincospif
is within 2 ulp, and scale, product and sum round once each: below 2^-21 of scale * (|x1| + |x2|) together. The store adds
half a step of the type.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.serving as sv
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def close(got, x, positions, freq, scale, offset, layout, inverse=False):
    want = sv.rope_oracle(x, positions, freq, scale, offset, layout, inverse)
    d = 2.0 ** -21 * abs(scale) * sv.rope_pair_size(x, 2 * freq.numel(), offset, layout)
    tol = torch.finfo(x.dtype).eps / 2 * (np.abs(want) + d) + d
    err = np.abs(sv.f64(got) - want)
    assert np.all(err <= tol), f"{np.max(err - tol)} over, at {np.unravel_index(np.argmax(err - tol), err.shape)}"
    r = 2 * freq.numel()
    for part in (slice(0, offset), slice(offset + r, None)):
        assert torch.equal(got[..., part].cpu(), x[..., part].cpu())


def make(n, heads, dim, rot, dtype, seed, span=1 << 20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=g).to(dtype).cuda()
    pos = torch.randint(-span, span, (n,), generator=g, dtype=torch.int32)
    pos[:3] = torch.tensor([0, 2 ** 31 - 1, -2 ** 31 + 1], dtype=torch.int32)[:n]
    return x, pos.cuda(), pkg.rope_inv_freq(rot)[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,dim,offset,rot", [
    (1, 1, 128, 0, 128), (64, 36, 128, 0, 128), (33, 4, 192, 128, 64), (5, 7, 80, 0, 80), (9, 3, 96, 86, 10),
    (3, 2, 64, 3, 18), (2, 5, 2, 0, 2), (130, 1, 256, 64, 128), (7, 2, 65, 1, 64), (1, 3, 1024, 0, 1024), (700, 5, 16, 8, 8)])
def test_rope(dtype, layout, n, heads, dim, offset, rot):
    x, pos, freq = make(n, heads, dim, rot, dtype, n + dim + rot)
    # the definition's own angle is exact to p * 2^-52: far positions with f = 1 stay below the bound
    close(pkg.rope(x, pos, freq, 1.25, offset, layout), x, pos, freq, 1.25, offset, layout)
    close(pkg.rope(x, pos, freq, 1.0, offset, layout, inverse=True), x, pos, freq, 1.0, offset, layout, True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("view", ["fused", "odd offset", "head major", "repeated"])
def test_rope_strides(layout, view):
    n, heads, dim = 17, 5, 64
    g = torch.Generator().manual_seed(3)
    if view == "fused":
        x = torch.randn(n, heads + 3, dim, generator=g).bfloat16().cuda()[:, 2:2 + heads]
    elif view == "odd offset":  # rows that start off 16-byte boundaries
        x = torch.randn(n, heads, dim + 3, generator=g).bfloat16().cuda()[..., 1:dim + 1]
    elif view == "head major":
        x = torch.randn(heads, n, dim, generator=g).bfloat16().cuda().transpose(0, 1)
    else:
        x = torch.randn(n, 1, dim, generator=g).bfloat16().cuda().expand(n, heads, dim)
    pos, freq = torch.arange(n, dtype=torch.int32).cuda() * 977, pkg.rope_inv_freq(32)[0]
    y = pkg.rope(x, pos, freq, 1.0, 16, layout)
    assert y.is_contiguous()
    close(y, x, pos, freq, 1.0, 16, layout)
    if view != "repeated":
        buf = torch.full((n, heads + 2, dim + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, 1:1 + heads, 3:3 + dim]
        pkg.rope(x, pos, freq, 1.0, 16, layout, out=out)
        assert torch.equal(out, y)
        buf[:, 1:1 + heads, 3:3 + dim] = 7.0
        assert torch.all(buf == 7.0)  # nothing written around the rows
        keep = x.clone()
        close(pkg.rope(x, pos, freq, 1.0, 16, layout, out=x), keep, pos, freq, 1.0, 16, layout)


def test_rope_scaled_frequencies_and_far_positions():
    x = torch.randn(64, 2, 128, generator=torch.Generator().manual_seed(9)).cuda()
    pos = (torch.arange(64, dtype=torch.int64) * 16777259 % (1 << 31)).int().cuda()
    for scaling in (None, "linear", "base", "by_parts"):
        freq, s = pkg.rope_inv_freq(128, 10000.0, scaling, 32.0 if scaling else 1.0)
        close(pkg.rope(x, pos, freq, s), x, pos, freq, s, 0, "half")


def test_rope_values_that_are_not_finite_stay_in_their_pair():
    x, pos, freq = make(6, 2, 64, 32, torch.bfloat16, 4)
    clean = pkg.rope(x, pos, freq)
    x[2, 1, 5], x[3, 0, 40] = float("nan"), float("inf")
    y = pkg.rope(x, pos, freq)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[2, 1, 5] = touched[2, 1, 21] = touched[3, 0, 40] = True
    assert torch.equal(y[~touched], clean[~touched]) and torch.isnan(y[2, 1, 5]) and torch.isinf(y[3, 0, 40])


def test_rope_gradient():
    """The inverse with the same scale is the transposed map: <rope(x), g> = <x, inverse(g)>, and against differences."""
    g = torch.Generator().manual_seed(8)
    x, d = torch.randn(5, 3, 32, generator=g).cuda(), torch.randn(5, 3, 32, generator=g).cuda()
    pos, freq = torch.arange(5, dtype=torch.int32).cuda() * 31, pkg.rope_inv_freq(16)[0]
    for layout in ("half", "interleaved"):
        y, back = pkg.rope(x, pos, freq, 1.5, 8, layout), pkg.rope(d, pos, freq, 1.5, 8, layout, inverse=True)
        a, b = (y.double() * d.double()).sum(), (x.double() * back.double()).sum()
        size = (x.double().abs().sum() * 4).item()
        assert abs((a - b).item()) <= 2.0 ** -20 * size
        step = torch.zeros_like(x)
        step[2, 1, 13] = 0.5  # linear: a difference is exact up to the rounding of both sides
        diff = ((pkg.rope(x + step, pos, freq, 1.5, 8, layout).double() - y.double()) * d.double()).sum() / 0.5
        assert abs((diff - back[2, 1, 13].double()).item()) <= 2.0 ** -18 * 16


def test_rope_empty_stream_and_graph():
    x, pos, freq = make(40, 3, 64, 64, torch.bfloat16, 11)
    assert pkg.rope(x[:0], pos[:0], freq).shape == (0, 3, 64)
    want = pkg.rope(x, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = pkg.rope(x, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.rope(x, pos, freq, out=out)
    x.copy_(torch.flip(x, (0,)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pkg.rope(x, pos, freq))


def test_rope_refusals():
    x, pos, freq = make(4, 2, 64, 64, torch.bfloat16, 1)
    for bad in (lambda: pkg.rope(x.double(), pos, freq), lambda: pkg.rope(x[0], pos, freq),
                lambda: pkg.rope(x, pos.long(), freq), lambda: pkg.rope(x, pos[:3], freq),
                lambda: pkg.rope(x, pos, freq.float()), lambda: pkg.rope(x, pos, None),
                lambda: pkg.rope(x, pos, freq, layout="other"), lambda: pkg.rope(x[..., ::2], pos, freq[:8]),
                lambda: pkg.rope(x, pos, freq, out=x.float()), lambda: pkg.rope(x, pos, freq, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pkg.rope(x, pos, freq, rot_offset=2), lambda: pkg.rope(x, pos, freq, scale=float("nan")),
                lambda: pkg.rope(x, pos, freq, out=x[:, :1].expand(4, 2, 64))):
        with pytest.raises(pkg.GqaError):
            bad()


def turns(p, f):
    """The fraction of a turn of the angle p * f (f a double), in [-1/2, 1/2], from rational arithmetic."""
    def atan_inverse(x, one):
        total, term, n = 0, one // x, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term, n = term // (x * x), n + 2
        return total
    one = 1 << 400
    pi = Fraction(4 * (4 * atan_inverse(5, one) - atan_inverse(239, one)), one)
    t = Fraction(p) * Fraction(f) / (2 * pi)
    return float(t - round(t))


def test_angles_of_far_positions():
    """(1, 0) turned gives (cos, sin) of the angle itself: off by 2^-25 of a half turn (the float), 2^-32 of a turn (the
    fixed-point fraction) and sincospif's 2 ulp of 2^-24, together below 2^-22. The angle is rational arithmetic's: a
    double's product loses as much as this bound."""
    freq = [1.0, 0.9, 3.7, 6.1, 500000.0 ** (-4 / 256), 1 / 3, 1e-4, 100.25, -0.7, 2.0 ** 70 / 3, 1e-12, 2.0 ** 116]
    r = len(freq)
    pos = [2 ** 31 - 1, -2 ** 31 + 1, 10 ** 9 + 7, -123456789, 1, 0]
    x = torch.zeros(len(pos), 1, 2 * r, device="cuda")
    x[..., :r] = 1.0
    got = sv.f64(pkg.rope(x, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(freq, dtype=torch.float64).cuda()))
    angle = 2 * np.pi * np.array([[turns(p, f) for f in freq] for p in pos])
    assert np.abs(got[:, 0, :r] - np.cos(angle)).max() <= 2.0 ** -22
    assert np.abs(got[:, 0, r:] - np.sin(angle)).max() <= 2.0 ** -22


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,dim,offset,rot", [(3, 5, 1023, 1, 1022), (2, 3, 1024, 301, 600), (5, 1, 1024, 0, 1024),
                                                    (1, 7, 900, 0, 30), (4, 2, 515, 0, 514)])
def test_heads_of_more_items_than_threads(n, heads, dim, offset, rot, layout, dtype):
    """One element an item (rows that start off a 16-byte boundary): a thread takes several items of a head, in place
    and out of place."""
    x, pos, freq = make(n, heads, dim + 3, rot, dtype, 7 * dim + n)
    x = x[..., 1:1 + dim]
    got = pkg.rope(x, pos, freq, 1.25, offset, layout)
    close(got, x, pos, freq, 1.25, offset, layout)
    back = pkg.rope(got, pos, freq, 1.0, offset, layout, inverse=True)
    close(back, got, pos, freq, 1.0, offset, layout, inverse=True)
    same = x.clone()
    wide = torch.full((n, heads, dim + 3), 9.0, dtype=dtype, device="cuda")
    wide[..., 1:1 + dim] = same
    pkg.rope(wide[..., 1:1 + dim], pos, freq, 1.25, offset, layout, out=wide[..., 1:1 + dim])
    assert torch.equal(wide[..., 1:1 + dim], got)
    assert (wide[..., 0] == 9).all() and (wide[..., 1 + dim:] == 9).all()
