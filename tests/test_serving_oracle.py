"""The serving operators' oracles against independent statements of the same definitions (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle.serving as sv
from oracle.fp8 import dequantize_rows, e4m3_decode


def test_e4m3_encode_inverts_decode_and_rounds_ties_to_even():
    codes = np.arange(256)
    vals = e4m3_decode(codes)
    fin = np.isfinite(vals)
    assert np.array_equal(sv.e4m3_encode(vals[fin]), codes[fin])
    pos = np.sort(vals[fin & (codes < 128)])
    mid = (pos[1:] + pos[:-1]) / 2
    assert np.all(sv.e4m3_encode(mid) % 2 == 0)
    assert sv.e4m3_encode(np.array([1e9, -1e9, np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7F]


def test_e4m3_encode_agrees_with_torch():
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 50
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(sv.e4m3_encode(x.double().numpy()), want)


def test_fp8_scale_is_the_smallest_that_fits():
    x = torch.randn(64, 4, 128, generator=torch.Generator().manual_seed(2)) * torch.logspace(-6, 6, 64)[:, None, None]
    s, top = sv.fp8_scale_oracle(x), np.abs(x.double().numpy()).max(-1)
    assert np.all(top / s <= 448) and np.all(top / (s / 2) > 448)
    assert sv.fp8_scale_oracle(np.zeros((1, 4, 128))).tolist() == [[1.0] * 4]
    assert sv.fp8_scale_oracle(np.full((1, 4, 128), 448.0))[0, 0] == 1.0


def test_fp8_rows_dequantise_within_half_a_step():
    x = torch.randn(9, 4, 128, generator=torch.Generator().manual_seed(3))
    back, s = dequantize_rows(sv.fp8_rows_oracle(x)), sv.fp8_scale_oracle(x)[..., None]
    x = x.double().numpy()
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_rotation_that_inverse_undoes(layout):
    g = torch.Generator().manual_seed(4)
    x, pos = torch.randn(7, 3, 20, generator=g), torch.randint(-50, 100000, (7,), generator=g)
    f = sv.inv_freq_oracle(12)
    y = sv.rope_oracle(x, pos, f, 1.0, 5, layout)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x.double().numpy(), axis=-1), rtol=1e-12)
    assert np.allclose(sv.rope_oracle(y, pos, f, 1.0, 5, layout, inverse=True), x.double().numpy(), atol=1e-12)
    assert np.array_equal(y[..., :5], x.double().numpy()[..., :5])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_scores_depend_on_distance_only(layout):
    g = torch.Generator().manual_seed(5)
    q, k = torch.randn(1, 1, 64, generator=g), torch.randn(1, 1, 64, generator=g)
    f = sv.inv_freq_oracle(64)
    dots = [(sv.rope_oracle(q, torch.tensor([a]), f, layout=layout) *
             sv.rope_oracle(k, torch.tensor([b]), f, layout=layout)).sum() for a, b in ((9, 2), (1007, 1000))]
    assert math.isclose(dots[0], dots[1], rel_tol=1e-9, abs_tol=1e-9)


def test_prefill_oracle_against_expanded_attention():
    """One sequence, identity page table: the same values from torch's softmax over explicit keys and values."""
    g = torch.Generator().manual_seed(6)
    n, nq, h = 11, 5, 2
    cache = torch.randn(3, 4, 1, 576, generator=g).double()
    w, q = torch.randn(h, 256, 512, generator=g).double() / 22, torch.randn(nq, h, 192, generator=g).double()
    out, lse, _, _ = sv.mla_prefill_oracle(q, w, cache, torch.tensor([[0, 1, 2]]), [n], [0, nq], 0.07)
    rows = cache.view(-1, 576)[:n]
    for a in range(h):
        k = torch.cat([rows[:, :512] @ w[a, :128].t(), rows[:, 512:]], 1)
        s = 0.07 * q[:, a] @ k.t()
        s = s.masked_fill(torch.arange(n) > (n - nq + torch.arange(nq))[:, None], -math.inf)
        assert np.allclose(out[:, a], (s.softmax(1) @ (rows[:, :512] @ w[a, 128:].t())).numpy(), atol=1e-12)
        assert np.allclose(lse[a], s.logsumexp(1).numpy(), atol=1e-12)


def test_prefill_oracle_matches_the_absorbed_form():
    """Expanded and absorbed latent attention are the same function (float64)."""
    from oracle.mla import mla_decode_oracle
    g = torch.Generator().manual_seed(7)
    n, h = 9, 16
    cache = torch.randn(3, 4, 1, 576, generator=g).double()
    w, q = torch.randn(h, 256, 512, generator=g).double() / 22, torch.randn(1, h, 192, generator=g).double()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    out, lse, _, _ = sv.mla_prefill_oracle(q, w, cache, table, [n], [0, 1], 0.07)
    lat = np.concatenate([sv.mla_absorb_q_oracle(q, w), q[..., 128:].numpy()], -1)
    o, l2 = mla_decode_oracle(torch.from_numpy(lat).view(1, 1, h, 576), cache, table, torch.tensor([n]), 0.07)
    assert np.allclose(sv.mla_expand_out_oracle(o[0], w)[0], out[0], atol=1e-10)
    assert np.allclose(l2[0, :, 0], lse[:, 0], atol=1e-10)
