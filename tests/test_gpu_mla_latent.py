"""GPU parity of latent attention's projections (absorbed form) and prompt pass (expanded form)."""
import math

import numpy as np
import pytest
import torch

import oracle.serving as sv
import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -23  # a step of the fp32 accumulation (rounded or cut)


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def weights(h, seed, std=512 ** -0.5):
    return (torch.randn(h, 256, 512, generator=torch.Generator().manual_seed(seed)) * std).to(BF)


# ------------------------------------------------------------------- projections
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 63, 64, 65, 130, 300])
@pytest.mark.parametrize("h", [1, 3, 16])
def test_projections(n, h):
    g = torch.Generator().manual_seed(n * 100 + h)
    w = weights(h, n)
    q, o = torch.randn(n, h, 192, generator=g).to(BF), torch.randn(n, h, 512, generator=g).to(BF)
    got = pkg.mla_absorb_q(q.cuda(), w.cuda())
    want = sv.mla_absorb_q_oracle(q, w)
    size = np.einsum("nhd,hdl->nhl", np.abs(sv.f64(q))[..., :128], np.abs(sv.f64(w))[:, :128])
    d = 128 * U * size
    assert np.all(np.abs(sv.f64(got)[..., :512] - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)
    assert torch.equal(got[..., 512:].cpu(), q[..., 128:])
    got = pkg.mla_expand_out(o.cuda(), w.cuda())
    want = sv.mla_expand_out_oracle(o, w)
    d = 512 * U * np.einsum("nhl,hdl->nhd", np.abs(sv.f64(o)), np.abs(sv.f64(w))[:, 128:])
    assert np.all(np.abs(sv.f64(got) - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n", [1, 20, 70])
def test_absorb_rotates_and_takes_strides(layout, n):
    g = torch.Generator().manual_seed(n)
    h = 5
    w, pos = weights(h, 3).cuda(), torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    freq = pkg.rope_inv_freq(64)[0]
    q = torch.randn(n, h + 2, 200, generator=g).to(BF).cuda()[:, 1:1 + h, :192]
    got = pkg.mla_absorb_q(q, w, pos, freq, 1.1, layout)
    assert torch.equal(got[..., :512], pkg.mla_absorb_q(q.contiguous(), w)[..., :512])
    want = sv.rope_oracle(q[..., 128:], pos, freq, 1.1, 0, layout)
    d = 2.0 ** -21 * 1.1 * sv.rope_pair_size(q[..., 128:], 64, 0, layout)
    assert np.all(np.abs(sv.f64(got[..., 512:]) - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)
    head_major = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(pkg.mla_absorb_q(head_major, w, pos, freq, 1.1, layout), got)
    buf = torch.zeros_like(got)
    assert pkg.mla_absorb_q(q, w, pos, freq, 1.1, layout, out=buf) is buf and torch.equal(buf, got)


def test_projections_not_finite_and_empty():
    n, h = 18, 2
    w = weights(h, 4).cuda()
    q = torch.randn(n, h, 192, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    clean = pkg.mla_absorb_q(q, w)
    q[4, 1, 3] = float("nan")
    got = pkg.mla_absorb_q(q, w)
    touched = torch.zeros(n, h, dtype=torch.bool)
    touched[4, 1] = True
    assert torch.equal(got[~touched], clean[~touched]) and torch.isnan(got[4, 1, :512]).all()
    assert pkg.mla_absorb_q(q[:0], w).shape == (0, h, 576)
    assert pkg.mla_expand_out(torch.zeros(0, h, 512, dtype=BF, device="cuda"), w).shape == (0, h, 128)


# -------------------------------------------------------------------- prompt pass
def case(lens, h, page, seed, std=1.0, extra=3, bad_blocks=0, width=None, w_std=512 ** -0.5):
    """Paged latent rows, every slot that no sequence owns being NaN."""
    g = torch.Generator().manual_seed(seed)
    width = width or max(1, max(-(-n // page) for _, n in lens))
    used = sum(-(-min(n, width * page) // page) for _, n in lens)
    blocks = used + extra
    cache = torch.full((blocks, page, 1, 576), float("nan"))
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    ids, at = torch.randperm(blocks, generator=g), 0
    for b, (_, n) in enumerate(lens):
        k = -(-min(n, width * page) // page)
        table[b, :k] = ids[at:at + k].to(torch.int32)
        for j in range(k):
            fill = min(page, n - j * page)
            cache[table[b, j], :fill, 0] = torch.randn(fill, 576, generator=g) * std
        at += k
    for i in range(bad_blocks):  # entries outside the pool: their tokens are left out
        b = i % len(lens)
        if lens[b][1]:
            table[b, (3 * i) % max(1, -(-min(lens[b][1], width * page) // page))] = [blocks, -1, 2 ** 31 - 1][i % 3]
    cu = [0]
    for nq, _ in lens:
        cu.append(cu[-1] + nq)
    q = torch.randn(cu[-1], h, 192, generator=g) * std
    return dict(q=q.to(BF), w_kv=weights(h, seed, w_std), kv_cache=cache.to(BF), block_table=table,
                cache_seqlens=torch.tensor([n for _, n in lens], dtype=torch.int32),
                cu_seqlens_q=torch.tensor(cu, dtype=torch.int32))


def on_gpu(c):
    return {k: v.cuda() for k, v in c.items()}


def check(out, lse, c, scale, causal):
    o, l, ob, lb = sv.mla_prefill_oracle(c["q"], c["w_kv"], c["kv_cache"], c["block_table"], c["cache_seqlens"],
                                         c["cu_seqlens_q"], scale, causal)
    done = ~np.isnan(l[0])
    got, gl = sv.f64(out), sv.f64(lse)
    err = np.abs(got - o)[done] - ob[done]
    assert np.all(err <= 0), f"out {err.max()} over its bound"
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl)[:, done], empty[:, done])
    assert np.all(got.transpose(1, 0, 2)[empty] == 0)
    fin = np.isfinite(l)
    err = np.abs(gl[fin] - l[fin]) - lb[fin]
    assert np.all(err <= 0), f"lse {err.max()} over its bound"


RAGGED = [(130, 130), (1, 1), (0, 0), (47, 300), (0, 50), (129, 128 + 129), (2, 700)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("h,page", [(1, 1), (3, 64), (2, 7), (16, 16)])
def test_prefill_ragged(h, page, causal):
    lens = RAGGED if h < 16 else RAGGED[:4]
    c = case(lens, h, page, 10 * h + page)
    g = on_gpu(c)
    out, lse = pkg.mla_prefill(**g, causal=causal)
    check(out, lse, c, 192 ** -0.5, causal)
    tight = sum(n for _, n in lens)
    out2, lse2 = pkg.mla_prefill(**g, causal=causal, max_kv_tokens=tight)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert pkg.mla_prefill(**g, causal=causal, with_lse=False)[1] is None
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("n", [1, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 640])
def test_prefill_lengths(n):
    for lens in ([(n, n)], [(1, n)], [(n, n + 129)]):
        c = case(lens, 2, 16, n)
        out, lse = pkg.mla_prefill(**on_gpu(c))
        check(out, lse, c, 192 ** -0.5, True)


@pytest.mark.parametrize("lens,h", [([(70, 10000)], 3), ([(40, 5000), (600, 2600), (1, 4000)], 5), ([(3, 700)] * 40, 1)])
def test_prefill_long_and_many(lens, h):
    """More units of the expansion than pairs of CTAs: runs that cross row tiles, and tiles shared by two pairs."""
    c = case(lens, h, 64, h)
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_several_units_a_pair(causal):
    """More units of the attention than pairs of CTAs, some without keys (in one query tile or both), long behind short."""
    lens = [(1, 1), (600, 100), (520, 0), (513, 700), (0, 40), (3, 900), (257, 257), (512, 129), (700, 30), (1, 128),
            (1030, 0), (1030, 1030), (40, 5), (256, 256), (2, 2)]
    c = case(lens, 16, 32, 24)
    g = on_gpu(c)
    out, lse = pkg.mla_prefill(**g, causal=causal)
    check(out, lse, c, 192 ** -0.5, causal)
    for _ in range(20):  # which pair takes a unit changes nothing
        out2, lse2 = pkg.mla_prefill(**g, causal=causal)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,h", [([(200, 6000)], 1), ([(1, 20000), (2, 129), (700, 1200)], 2), ([(520, 4000)] * 2, 20),
                                    ([(1, 9000), (600, 8100), (0, 0), (520, 0), (300, 40), (513, 9000)], 2)])
def test_prefill_units_split_over_the_keys(lens, h, causal):
    """Few units with many keys: pieces of a unit in several pairs of CTAs, joined by whichever is last."""
    c = case(lens, h, 64, 25 + h)
    g = on_gpu(c)
    out, lse = pkg.mla_prefill(**g, causal=causal)
    check(out, lse, c, 192 ** -0.5, causal)
    for _ in range(20):
        out2, lse2 = pkg.mla_prefill(**g, causal=causal)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [pkg.mla_prefill(**g, causal=causal, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(out, o) and torch.equal(lse, l) for o, l in got)
    out3 = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.mla_prefill(**g, causal=causal, out=out3, with_lse=False)
    for _ in range(2):
        out3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out3)
    assert _lib.gqa_paged_decode_device_error() == 0


def test_prefill_split_in_several_passes():
    """The pieces of one pass over the heads are joined before the next pass writes its own."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    c = case([(60, 9000)], 5, 64, 34)
    out, lse = pkg.mla_prefill(**on_gpu(c), max_kv_tokens=2_000_000)  # two heads a pass
    check(out, lse, c, 192 ** -0.5, True)


def test_prefill_split_rows_not_finite():
    """A token that is not finite, late in a long sequence: rows that see it are NaN, the others as without it."""
    c = case([(200, 6000)], 2, 64, 33)
    blk = int(c["block_table"][0, 5900 // 64])
    c["kv_cache"][blk, 5900 % 64, 0, :512] = 0
    want, _ = pkg.mla_prefill(**on_gpu(c))
    c["kv_cache"][blk, 5900 % 64, 0, :512] = float("inf")
    out, lse = pkg.mla_prefill(**on_gpu(c))
    assert torch.equal(out[:100], want[:100])  # row i sees the tokens up to 5800 + i
    assert out[100:].isnan().all() and lse[:, 100:].isnan().all() and lse[:, :100].isfinite().all()


def test_prefill_rows_that_see_nothing():
    """More queries than cached tokens (their first rows see none), lengths of 0, blocks outside the pool."""
    c = case([(70, 3), (5, 0), (40, 40), (300, 200)], 3, 8, 5, bad_blocks=5)
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)
    c["block_table"][2] = -1
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)
    assert torch.all(torch.isneginf(lse[:, 75:115]))


def test_prefill_lengths_past_the_table_and_negative():
    c = case([(20, 100), (9, 30)], 2, 16, 8, width=4)  # 64 tokens of room
    c["cache_seqlens"][1] = -5
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)


def test_prefill_rows_behind_the_last_sequence_stay():
    c = case([(30, 30), (10, 90)], 2, 16, 9)
    g = on_gpu(c)
    g["q"] = torch.cat([g["q"], torch.full((25, 2, 192), float("nan"), dtype=BF, device="cuda")])
    out = torch.full((65, 2, 128), 5.0, dtype=BF, device="cuda")
    lse = torch.full((2, 65), 5.0, device="cuda")
    pkg.mla_prefill(**g, out=out, lse=lse)
    assert torch.all(out[40:] == 5.0) and torch.all(lse[:, 40:] == 5.0)
    check(out[:40], lse[:, :40], c, 192 ** -0.5, True)


@pytest.mark.parametrize("std,w_std,scale", [(64.0, 1.0, 1e-5), (2.0 ** -30, 2.0 ** -20, 2.0 ** 70), (2.0 ** 40, 2.0 ** 30, 2.0 ** -120)])
def test_prefill_sizes_of_values(std, w_std, scale):
    """Values past fp16's range either way: the bounds scale with the values (powers of two change nothing)."""
    c = case([(40, 90)], 2, 16, 12, std=std, w_std=w_std)
    out, lse = pkg.mla_prefill(**on_gpu(c), softmax_scale=scale)
    if std == 64.0:
        check(out, lse, c, scale, True)
        return
    # bring the same numbers back to ordinary size by powers of two: the outputs have to agree to their roundings
    d = dict(c, q=c["q"] / std, kv_cache=c["kv_cache"] / std, w_kv=(c["w_kv"].float() / w_std * 2.0 ** -5).to(BF))
    rows = torch.arange(576) >= 512
    k = std * w_std * 32  # expanded keys are this much larger than d's, rotary ones std: keep only the former
    c["kv_cache"][..., rows] = 0
    d["kv_cache"][..., rows] = 0
    out, lse = pkg.mla_prefill(**on_gpu(c), softmax_scale=scale)
    o2, l2 = pkg.mla_prefill(**on_gpu(d), softmax_scale=scale * std * k)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert torch.equal((out.double() / k).to(BF), o2.double().to(BF))
    assert torch.allclose(lse, l2, rtol=0, atol=1e-5)


def test_prefill_a_sequence_of_huge_values_leaves_the_others():
    """Finite values near the type's largest in one sequence: the others' outputs are bit for bit what they were."""
    c = case([(50, 200), (30, 30), (129, 300)], 2, 16, 21)
    g = on_gpu(c)
    out, lse = pkg.mla_prefill(**g)
    g["kv_cache"][g["block_table"][1, 0].long(), 5] *= 2.0 ** 100
    got, gl = pkg.mla_prefill(**g)
    keep = torch.ones(209, dtype=torch.bool)
    keep[50:80] = False
    assert torch.equal(got[keep], out[keep]) and torch.equal(gl[:, keep], lse[:, keep])


def test_prefill_large_scores_and_not_finite_values():
    c = case([(50, 50), (40, 260)], 2, 16, 13, std=6.0)  # scores of many hundreds: one weight takes it all
    g = on_gpu(c)
    out, lse = pkg.mla_prefill(**g, softmax_scale=1.0)
    check(out, lse, c, 1.0, True)
    clean = out.clone()
    # a token of sequence 1 that is not finite reaches that sequence's rows that see it, and no others
    g["kv_cache"][g["block_table"][1, 15].long(), 3] = float("inf")
    out, _ = pkg.mla_prefill(**g, softmax_scale=1.0)
    sees = torch.arange(90) >= 50 + (15 * 16 + 3 - 220)
    assert torch.equal(out[~sees], clean[~sees]) and torch.isnan(out[sees]).all()
    q = g["q"].clone()
    q[7, 1, 100] = float("nan")
    g = on_gpu(c)
    g["q"] = q
    out, lse = pkg.mla_prefill(**g, softmax_scale=1.0)
    hit = torch.zeros(90, 2, dtype=torch.bool)
    hit[7, 1] = True
    assert torch.equal(out[~hit], clean[~hit]) and torch.isnan(out[7, 1]).all() and torch.isnan(lse[1, 7])


def test_prefill_strides():
    c = case([(90, 150), (33, 33)], 3, 16, 14)
    g = on_gpu(c)
    want = pkg.mla_prefill(**g)[0]
    wide = torch.zeros(123, 5, 208, dtype=BF, device="cuda")
    wide[:, 1:4, 8:200] = g["q"]
    g["q"] = wide[:, 1:4, 8:200]
    assert torch.equal(pkg.mla_prefill(**g)[0], want)
    g["q"] = c["q"].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert torch.equal(pkg.mla_prefill(**g)[0], want)


def test_prefill_bound_too_small_is_reported():
    c = case([(20, 100), (30, 500), (10, 40)], 2, 16, 15)
    g = on_gpu(c)
    _lib.gqa_paged_decode_device_error()
    out, lse = pkg.mla_prefill(**g, max_kv_tokens=120)
    assert _lib.gqa_paged_decode_device_error() == 64
    assert torch.all(torch.isneginf(lse[:, 20:50])) and torch.all(out[20:50] == 0)
    whole = pkg.mla_prefill(**g)[0]
    assert torch.equal(out[:20], whole[:20])


def test_prefill_malformed_offsets_are_reported_and_stay_in_range():
    c = case([(20, 20), (30, 30)], 1, 16, 16)
    g = on_gpu(c)
    for cu in ([0, 40, 20], [-3, 20, 50], [0, 20, 90]):
        g["cu_seqlens_q"] = torch.tensor(cu, dtype=torch.int32).cuda()
        guard = torch.full((150, 1, 128), 5.0, dtype=BF, device="cuda")
        pkg.mla_prefill(**g, out=guard[50:100])
        assert _lib.gqa_paged_decode_device_error() == 8
        assert torch.all(guard[:50] == 5.0) and torch.all(guard[100:] == 5.0)


@pytest.mark.parametrize("n,h", [(300, 3), (9000, 2)])
def test_prefill_malformed_offsets_that_share_rows(n, h):
    """More query tiles than the rows make: reported, nothing outside the rows written, and the next call is right."""
    c = case([(2048, n), (0, 0), (0, n), (0, 0)], h, 64, 23)
    g = on_gpu(c)
    g["cu_seqlens_q"] = torch.tensor([0, 2048, 0, 2048, 0], dtype=torch.int32, device="cuda")
    buf = torch.full((2048 + 64, h, 128), 5.0, dtype=BF, device="cuda")
    pkg.mla_prefill(**g, out=buf[32:-32])
    assert _lib.gqa_paged_decode_device_error() == 8
    assert (buf[:32] == 5).all() and (buf[-32:] == 5).all()
    c = case([(70, n)], h, 64, 24)
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)
    assert _lib.gqa_paged_decode_device_error() == 0


def test_prefill_many_sequences():
    """More sequences than one chunk of the plan's prefix sums (1024)."""
    g = torch.Generator().manual_seed(17)
    lens = [(int(a), int(a) + int(b)) for a, b in zip(torch.randint(0, 4, (1500,), generator=g),
                                                     torch.randint(0, 5, (1500,), generator=g))]
    c = case(lens, 1, 4, 17)
    out, lse = pkg.mla_prefill(**on_gpu(c))
    check(out, lse, c, 192 ** -0.5, True)


def test_prefill_passes_over_the_heads_agree():
    """A bound on the tokens that makes the heads take several passes gives the same values."""
    c = case([(60, 200)], 5, 16, 18)
    g = on_gpu(c)
    want, wl = pkg.mla_prefill(**g)
    big = 2_000_000  # 512 bytes a token and head: two heads a pass
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    out, lse = pkg.mla_prefill(**g, max_kv_tokens=big)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_prefill_repeats_and_streams_and_graph():
    c = case([(150, 400), (64, 64)], 4, 32, 19)
    g = on_gpu(c)
    want, wl = pkg.mla_prefill(**g)
    for _ in range(3):
        out, lse = pkg.mla_prefill(**g)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):  # two calls at once, each with its own workspace
        for s in streams:
            got.append(pkg.mla_prefill(**g, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(l, wl) for o, l in got)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.mla_prefill(**g, out=out, with_lse=False)
    g["q"].copy_(g["q"].flip(0))
    expect = pkg.mla_prefill(**g)[0]
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect)


def test_prefill_refusals():
    g = on_gpu(case([(5, 9)], 2, 16, 20))
    for change in (dict(q=g["q"].float()), dict(q=g["q"][:, :1]), dict(w_kv=g["w_kv"][:, :200]), dict(kv_cache=g["kv_cache"][:, :, 0]),
                   dict(block_table=g["block_table"].long()), dict(cache_seqlens=g["cache_seqlens"].repeat(2)),
                   dict(cu_seqlens_q=g["cu_seqlens_q"][:1]), dict(out=torch.empty(5, 2, 64, dtype=BF, device="cuda")),
                   dict(lse=torch.empty(5, 2, device="cuda")), dict(max_kv_tokens=-1), dict(max_kv_tokens=1 << 40)):
        with pytest.raises(ValueError):
            pkg.mla_prefill(**dict(g, **change))
    with pytest.raises(pkg.GqaError):
        pkg.mla_prefill(**g, softmax_scale=float("nan"))
    with pytest.raises(pkg.GqaError):
        pkg.mla_prefill(**g, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------- used together
def test_prompt_then_steps():
    """A serving run: a prompt's latents written and attended (expanded), then steps of one token (absorbed). Each
    output against the float64 definition on what the cache holds."""
    g = torch.Generator().manual_seed(30)
    h, page, n, steps = 16, 32, 90, 3
    w, freq = weights(h, 31), pkg.rope_inv_freq(64)[0]
    cache = torch.full((8, page, 1, 576), float("nan"), dtype=BF, device="cuda")
    table = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32)
    slot = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n + steps)], dtype=torch.int32).cuda()
    rows = torch.randn(n + steps, 576, generator=g).to(BF).cuda()
    q = torch.randn(n + steps, h, 192, generator=g).to(BF).cuda()
    pos = torch.arange(n + steps, dtype=torch.int32).cuda()
    pkg.mla_kv_append(rows[:n, :512], rows[:n, 512:], slot[:n], cache, pos[:n], freq)
    turned = pkg.rope(q, pos, freq, rot_offset=128, layout="interleaved")
    one = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out, lse = pkg.mla_prefill(turned[:n], w.cuda(), cache, table.cuda(), one([n]), one([0, n]))
    c = dict(q=turned[:n].cpu(), w_kv=w, kv_cache=cache.cpu(), block_table=table, cache_seqlens=one([n]).cpu(),
             cu_seqlens_q=one([0, n]).cpu())
    check(out, lse, c, 192 ** -0.5, True)
    for i in range(n, n + steps):
        pkg.mla_kv_append(rows[i:i + 1, :512], rows[i:i + 1, 512:], slot[i:i + 1], cache, pos[i:i + 1], freq)
        o, l = pkg.mla_absorbed_run(q[None, i:i + 1], w.cuda(), cache, table.cuda(), one([i + 1]), pos[i:i + 1], freq)
        ref, lref, _, _ = sv.mla_prefill_oracle(turned[i:i + 1].cpu(), w, cache.cpu(), table, [i + 1], [0, 1], 192 ** -0.5)
        assert np.all(np.abs(sv.f64(o)[0, 0] - ref[0]) <= 2e-2 + 2e-2 * np.abs(ref[0]))
        assert np.abs(sv.f64(l)[0, :, 0] - lref[:, 0]).max() <= 2e-2
        e, _ = pkg.mla_prefill(turned[i:i + 1], w.cuda(), cache, table.cuda(), one([i + 1]), one([0, 1]))
        assert np.abs(sv.f64(e)[0] - sv.f64(o)[0, 0]).max() <= 2e-2  # the two forms agree
    assert _lib.gqa_paged_decode_device_error() == 0


# -------------------------------------------------- tokens of very different size
def one_huge(n, nq, h, at, factor, seed):
    """A sequence with one token `factor` times as large, one of zeros, and the same without the huge one (its page,
    of a single token, is outside the pool there)."""
    c = case([(nq, n)], h, 1, seed)
    block = int(c["block_table"][0, at])
    c["kv_cache"][block] = (c["kv_cache"][block].double() * factor).to(BF)
    c["kv_cache"][int(c["block_table"][0, n // 3])] = 0
    without = dict(c, block_table=c["block_table"].clone())
    without["block_table"][0, at] = -1
    return c, without


def check_huge(out, lse, c, without, at, causal):
    """Rows that do not see the token or give it no weight are the definition's without it; rows that give it all of
    theirs are its value: half a step of bf16 (2^-8), one of fp16 each for value and weight (2^-10 together), and the
    accumulation of the value (512 steps of 2^-23 of its products, 2^-14)."""
    nq, n = c["q"].shape[0], int(c["cache_seqlens"][0])
    o, l, ob, lb = sv.mla_prefill_oracle(without["q"], without["w_kv"], without["kv_cache"], without["block_table"],
                                         without["cache_seqlens"], without["cu_seqlens_q"], 192 ** -0.5, causal)
    row = sv.f64(c["kv_cache"][int(c["block_table"][0, at]), 0, 0])
    full, mag = sv.f64(c["w_kv"]) @ row[:512], np.abs(sv.f64(c["w_kv"])) @ np.abs(row[:512])
    key = np.concatenate([full[:, :128], np.broadcast_to(row[512:], (full.shape[0], 64))], 1)
    score = 192 ** -0.5 * np.einsum("nhd,hd->nh", sv.f64(c["q"]), key)
    sees = np.ones(nq, bool) if not causal else np.arange(nq) >= at - (n - nq)
    takes = sees[:, None] & (score > 0)
    assert np.all(np.abs(score) > 1e4)  # nothing between all and no weight (the others' scores are a few units)
    got, gl = sv.f64(out), sv.f64(lse).T
    err = np.abs(got - o) - ob
    assert np.all(err[~takes] <= 0), f"out {err[~takes].max()} over its bound"
    err = np.abs(gl - l.T) - lb.T
    assert np.all(err[~takes] <= 0), f"lse {err[~takes].max()} over its bound"
    v = np.broadcast_to(full[:, 128:], got.shape)
    tol = (2.0 ** -8 + 2.0 ** -10) * np.abs(v) + 2.0 ** -13 * mag[:, 128:]
    assert np.all((np.abs(got - v) <= tol)[takes]) and takes.any() == sees.any()
    assert np.all(np.abs(gl - score)[takes] <= 2.0 ** -10 * 192 ** -0.5 * np.einsum(
        "nhd,hd->nh", np.abs(sv.f64(c["q"])), np.concatenate([mag[:, :128], np.abs(key[:, 128:])], 1))[takes])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,nq,h,at,factor", [
    (200, 200, 2, 150, 2.0 ** 60), (300, 300, 3, 299, 2.0 ** 100), (700, 530, 1, 640, 2.0 ** 40), (130, 1, 2, 5, 2.0 ** 60),
    (600, 600, 2, 0, 2.0 ** 60), (6000, 200, 2, 5900, 2.0 ** 60), (6000, 200, 2, 100, 2.0 ** 80)])
def test_prefill_one_huge_token(n, nq, h, at, factor, causal):
    """A finite token far larger than the others, late, early, and where units are split over their keys."""
    c, without = one_huge(n, nq, h, at, factor, n + h)
    out, lse = pkg.mla_prefill(**on_gpu(c), causal=causal)
    check_huge(out, lse, c, without, at, causal)
    assert _lib.gqa_paged_decode_device_error() == 0


def test_prefill_small_tokens_before_ordinary_ones():
    """Rows that see only tokens 2^-60 times the later ones' size keep full precision: their scores are 0, so a row is
    the mean of the values it sees. Bounds as in check_huge, and n steps of 2^-23 for the sum."""
    c = case([(200, 200)], 2, 1, 41)
    small = c["block_table"][0, :40].long()
    c["kv_cache"][small] = (c["kv_cache"][small].double() * 2.0 ** -60).to(BF)
    out, lse = pkg.mla_prefill(**on_gpu(c))
    rows, w = sv.f64(c["kv_cache"][small])[:, 0, 0, :512], sv.f64(c["w_kv"])[:, 128:]
    v, mag = np.einsum("tl,hdl->thd", rows, w), np.einsum("tl,hdl->thd", np.abs(rows), np.abs(w))
    count = np.arange(1, 41)[:, None, None]
    want, size, mags = (np.cumsum(x, 0) / count for x in (v, np.abs(v), mag))
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size + 2.0 ** -13 * mags
    assert np.all(np.abs(sv.f64(out)[:40] - want) <= tol)
    check(out[40:], lse[:, 40:], dict(c, q=c["q"][40:], cu_seqlens_q=torch.tensor([0, 160], dtype=torch.int32)),
          192 ** -0.5, True)


def test_prefill_one_huge_token_in_several_passes_and_beside_others():
    """Passes over the heads read the same row exponents; sequences without such a token keep their bits."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    c = case([(50, 90), (300, 300), (33, 700)], 5, 1, 42)
    plain, _ = pkg.mla_prefill(**on_gpu(c))
    block = int(c["block_table"][1, 250])
    c["kv_cache"][block] = (c["kv_cache"][block].double() * 2.0 ** 70).to(BF)
    want, wl = pkg.mla_prefill(**on_gpu(c))
    out, lse = pkg.mla_prefill(**on_gpu(c), max_kv_tokens=2_000_000)  # two heads a pass
    assert torch.equal(out, want) and torch.equal(lse, wl)
    assert torch.equal(out[:50], plain[:50]) and torch.equal(out[350:], plain[350:])


@pytest.mark.parametrize("others", [1.0, 2.0 ** 118])
def test_prefill_expansion_past_32_bits(others):
    """A finite latent whose keys and values pass fp32's range leaves the rows that do not see it alone, whether the
    tokens have their own exponents (the others 2^125 times smaller) or one (2^7 times)."""
    c = case([(200, 200)], 2, 1, 44, w_std=1.0)
    block, scale = int(c["block_table"][0, 150]), 192 ** -0.5 / others
    row = c["kv_cache"][block].double()
    c["kv_cache"] = (c["kv_cache"].double() * others).to(BF)
    c["kv_cache"][block] = (row * 2.0 ** 125).to(BF)
    assert c["kv_cache"][block].isfinite().all()
    assert np.abs(sv.f64(c["w_kv"]) @ sv.f64(c["kv_cache"][block, 0, 0, :512])).max() > 2.0 ** 128
    out, lse = pkg.mla_prefill(**on_gpu(c), softmax_scale=scale)
    o, l, ob, lb = sv.mla_prefill_oracle(c["q"][:150], c["w_kv"], c["kv_cache"], c["block_table"], [150], [0, 150], scale)
    assert np.all(np.abs(sv.f64(out)[:150] - o) <= ob) and np.all(np.abs(sv.f64(lse)[:, :150] - l) <= lb)


def test_prefill_not_finite_and_huge_tokens_together():
    """Rows before either are as without both; rows that see the one that is not finite are NaN."""
    c = case([(200, 200)], 2, 1, 43)
    want, _ = pkg.mla_prefill(**on_gpu(c))
    for t, x in ((120, 2.0 ** 60), (160, float("inf"))):
        c["kv_cache"][int(c["block_table"][0, t])] *= x
    out, lse = pkg.mla_prefill(**on_gpu(c))
    oracle = sv.mla_prefill_oracle(c["q"][:120], c["w_kv"], c["kv_cache"], c["block_table"], [120], [0, 120], 192 ** -0.5)
    assert np.all(np.abs(sv.f64(out)[:120] - oracle[0]) <= oracle[2])
    assert out[:160].isfinite().all() and out[160:].isnan().all() and lse[:, 160:].isnan().all()


# ------------------------------------------------------------ rows of no sequence
def poisoned(*shapes):
    """Leaves NaN in the memory that tensors of these shapes are likely to get next."""
    held = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("before,behind", [(0, 25), (7, 0), (5, 130)])
def test_prefill_own_outputs_have_no_rows_left_over(before, behind):
    c = case([(30, 30), (0, 0), (10, 90)], 2, 16, 9)
    g = on_gpu(c)
    pad = lambda n: torch.full((n, 2, 192), float("nan"), dtype=BF, device="cuda")  # noqa: E731
    g["q"] = torch.cat([pad(before), g["q"], pad(behind)])
    g["cu_seqlens_q"] += before
    n, rows = before + 40 + behind, slice(before, before + 40)
    poisoned(((n, 2, 128), BF), ((2, n), torch.float32))
    out, lse = pkg.mla_prefill(**g)
    check(out[rows], lse[:, rows], c, 192 ** -0.5, True)
    rest = torch.ones(n, dtype=torch.bool)
    rest[rows] = False
    assert (out[rest] == 0).all() and torch.isneginf(lse[:, rest]).all()
    kept = torch.full_like(out, 5.0)  # a given output keeps its rows, the call's own lse does not
    _, lse = pkg.mla_prefill(**g, out=kept)
    assert (kept[rest] == 5).all() and torch.equal(kept[rows], out[rows]) and torch.isneginf(lse[:, rest]).all()
    kept = torch.full_like(lse, 5.0)
    out2, _ = pkg.mla_prefill(**g, lse=kept)
    assert (kept[:, rest] == 5).all() and torch.equal(out2, out)
    assert _lib.gqa_paged_decode_device_error() == 0


def test_prefill_own_outputs_of_no_sequences():
    g = on_gpu(case([(5, 9)], 2, 16, 20))
    g |= dict(block_table=g["block_table"][:0], cache_seqlens=g["cache_seqlens"][:0], cu_seqlens_q=g["cu_seqlens_q"][:1])
    for stream in (None, torch.cuda.Stream()):
        poisoned(((5, 2, 128), BF), ((2, 5), torch.float32))
        out, lse = pkg.mla_prefill(**g, stream=stream)
        torch.cuda.synchronize()
        assert (out == 0).all() and torch.isneginf(lse).all()
    out = torch.full((5, 2, 128), 5.0, dtype=BF, device="cuda")
    assert (pkg.mla_prefill(**g, out=out, with_lse=False)[0] == 5).all()


# ------------------------------------------------------- the absorbed form's batch
@pytest.mark.parametrize("s_q,h,page", [(1, 32, 64), (3, 16, 32), (2, 64, 16), (4, 4, 1)])
def test_absorbed_run_of_a_batch(s_q, h, page):
    """Several sequences and new tokens: out and lse rows in their places, against the definition (tolerances as for
    one token above: queries, weights and latent outputs are rounded to bf16 on the way) and the three calls it makes."""
    lens = [(s_q, 40), (s_q, 700), (s_q, 1), (s_q, 129)]
    c = case(lens, h, page, 50 + h)
    g, n = on_gpu(c), len(lens) * s_q
    freq, pos = pkg.rope_inv_freq(64)[0], torch.randint(0, 5000, (n,), dtype=torch.int32, generator=torch.Generator().manual_seed(s_q)).cuda()
    args = (g["w_kv"], g["kv_cache"], g["block_table"], g["cache_seqlens"], pos, freq, 1.1)
    out, lse = pkg.mla_absorbed_run(g["q"].view(len(lens), s_q, h, 192), *args)
    assert out.shape == (len(lens), s_q, h, 128) and lse.shape == (len(lens), h, s_q)
    turned = pkg.rope(g["q"], pos, freq, 1.1, 128, "interleaved").cpu()
    o, l, _, _ = sv.mla_prefill_oracle(turned, c["w_kv"], c["kv_cache"], c["block_table"], c["cache_seqlens"],
                                       c["cu_seqlens_q"], 192 ** -0.5, causal=False)
    got = sv.f64(out).reshape(n, h, 128)
    assert np.all(np.abs(got - o) <= 2e-2 + 2e-2 * np.abs(o))
    assert np.abs(sv.f64(lse).transpose(1, 0, 2).reshape(h, n) - l).max() <= 2e-2
    lat = pkg.mla_absorb_q(g["q"], g["w_kv"], pos, freq, 1.1)
    o_lat, lse2 = pkg.mla_run(lat.view(len(lens), s_q, h, 576), g["kv_cache"], g["block_table"], g["cache_seqlens"], 192 ** -0.5)
    assert torch.equal(lse, lse2)
    assert torch.equal(out.view(n, h, 128), pkg.mla_expand_out(o_lat.view(n, h, 512), g["w_kv"]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = pkg.mla_absorbed_run(g["q"].view(len(lens), s_q, h, 192), *args, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert pkg.mla_absorbed_run(g["q"].view(len(lens), s_q, h, 192), *args, with_lse=False)[1] is None
    assert _lib.gqa_paged_decode_device_error() == 0


@pytest.mark.parametrize("n", [3, 200])
def test_projections_in_streams_and_a_graph(n):
    """Both forms of the projections (up to 16 tokens and above) in two streams at once and captured; out= given."""
    g, h = torch.Generator().manual_seed(n), 5
    w = weights(h, n).cuda()
    q, o = torch.randn(n, h, 192, generator=g).to(BF).cuda(), torch.randn(n, h, 512, generator=g).to(BF).cuda()
    pos, freq = torch.arange(n, dtype=torch.int32).cuda(), pkg.rope_inv_freq(64)[0]
    calls = [lambda **k: pkg.mla_absorb_q(q, w, pos, freq, **k), lambda **k: pkg.mla_expand_out(o, w, **k)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [f(stream=s) for _ in range(4) for s in streams for f in calls]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(got))
    outs = [torch.zeros_like(x) for x in want]
    assert all(f(out=x) is x and torch.equal(x, y) for f, x, y in zip(calls, outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f, x in zip(calls, outs):
            f(out=x)
    q.copy_(q.flip(0))
    o.copy_(o.flip(0))
    want = [f() for f in calls]
    for _ in range(2):
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    for bad in (torch.empty(n, h, 64, dtype=BF, device="cuda"), torch.empty(n, h, 128, device="cuda"),
                torch.empty(n, 128, h, dtype=BF, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            pkg.mla_expand_out(o, w, out=bad)


def test_absorbed_runs_share_no_workspace():
    """Calls in two streams at once, two captured graphs replayed at once, and a graph replayed after a call that needs
    far more room: each gives what it gives alone."""
    page, freq = 64, pkg.rope_inv_freq(64)[0]
    lens = [[3000, 40, 700, 1], [5, 2000, 2000, 64, 900]]
    sets = []
    for i, (ln, h) in enumerate(zip(lens, (32, 16))):
        c = case([(1, n) for n in ln], h, page, 60 + i)
        g, b = on_gpu(c), len(ln)
        pos = torch.tensor(ln, dtype=torch.int32).cuda() - 1
        sets.append((g["q"].view(b, 1, h, 192), g["w_kv"], g["kv_cache"], g["block_table"], g["cache_seqlens"], pos, freq))
    want = [pkg.mla_absorbed_run(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [(i, pkg.mla_absorbed_run(*sets[i], stream=streams[i])) for _ in range(10) for i in (0, 1)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for i, (o, l) in got)
    graphs, outs = [], []
    for a in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(pkg.mla_absorbed_run(*a))
        graphs.append(graph)
    large = case([(1, 9000)] * 40, 64, page, 62)
    g = on_gpu(large)
    pkg.mla_absorbed_run(g["q"].view(40, 1, 64, 192), g["w_kv"], g["kv_cache"], g["block_table"], g["cache_seqlens"],
                         g["cache_seqlens"] - 1, freq)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for (o, l), w in zip(outs, want))
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
    assert _lib.gqa_paged_decode_device_error() == 0


def test_absorbed_run_refusals():
    c = case([(1, 20), (1, 3)], 16, 16, 63)
    g = on_gpu(c)
    ok = dict(q=g["q"].view(2, 1, 16, 192), w_kv=g["w_kv"], kv_cache=g["kv_cache"], block_table=g["block_table"],
              cache_seqlens=g["cache_seqlens"])
    pkg.mla_absorbed_run(**ok)
    for name in ok:
        with pytest.raises((TypeError, ValueError)):
            pkg.mla_absorbed_run(**dict(ok, **{name: None}))
    for change in (dict(q=ok["q"][:, 0]), dict(kv_cache=ok["kv_cache"][:, :, 0]), dict(block_table=ok["block_table"][0]),
                   dict(block_table=ok["block_table"].long()), dict(block_table=ok["block_table"][:, :0]),
                   dict(cache_seqlens=ok["cache_seqlens"][:1]), dict(q=ok["q"][:, :, :8], w_kv=ok["w_kv"][:8])):
        with pytest.raises(ValueError):
            pkg.mla_absorbed_run(**dict(ok, **change))
    out, lse = pkg.mla_absorbed_run(**dict(ok, q=ok["q"][:0], block_table=ok["block_table"][:0], cache_seqlens=ok["cache_seqlens"][:0]))
    assert out.shape == (0, 1, 16, 128) and lse.shape == (0, 16, 1)


@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0 ** -130])
@pytest.mark.parametrize("huge", [False, True])
def test_prefill_scales_of_any_sign(scale, huge):
    """A negative scale turns the order round; 0 and one below what 32 bits hold give the mean of the values seen."""
    c = case([(150, 170), (40, 40)], 2, 1, 64)
    rows = torch.ones(190, dtype=torch.bool)
    if huge:
        block = int(c["block_table"][0, 120])
        c["kv_cache"][block] = (c["kv_cache"][block].double() * 2.0 ** 50).to(BF)
        rows[100:150] = False  # they see it
    out, lse = pkg.mla_prefill(**on_gpu(c), softmax_scale=scale)
    o, l, ob, lb = sv.mla_prefill_oracle(c["q"], c["w_kv"], c["kv_cache"], c["block_table"], c["cache_seqlens"],
                                         c["cu_seqlens_q"], scale)
    assert np.all((np.abs(sv.f64(out) - o) <= ob)[rows]) and np.all((np.abs(sv.f64(lse) - l) <= lb)[:, rows])


def test_prefill_small_scale_of_small_queries_and_large_keys():
    """The factors of a score pass the range of 32 bits only among themselves: bit for bit the outputs at ordinary size
    (all powers of two; rotary keys 0, which another power would scale)."""
    c = case([(40, 90)], 2, 16, 12)
    c["kv_cache"][..., 512:] = 0
    big = dict(c, q=(c["q"].double() * 2.0 ** -50).to(BF), kv_cache=(c["kv_cache"].double() * 2.0 ** 60).to(BF),
               w_kv=(c["w_kv"].double() * 2.0 ** 58).to(BF))
    want, wl = pkg.mla_prefill(**on_gpu(c), softmax_scale=2.0 ** -4)
    out, lse = pkg.mla_prefill(**on_gpu(big), softmax_scale=2.0 ** (-4 + 50 - 60 - 58))
    assert torch.equal((out.double() * 2.0 ** -118).to(BF), want) and torch.equal(lse, wl)
