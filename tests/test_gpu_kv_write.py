"""GPU parity of the cache's write and read: rotary append (bf16 and FP8 caches), FP8 append, FP8 read, latent append.

Codes and scales of values that are not turned are compared bit for bit. Turned keys differ from the definition by up
to 2^-21 of their pair (see the rotary tests) before they are quantised, so they are compared as values: half an e4m3
step (2^-4 of the value, 2^-10 of the scale at least) plus that.
"""
import numpy as np
import pytest
import torch

import oracle.serving as sv
import paged_kv_gqa_split_gb300 as pkg
from oracle.fp8 import dequantize_rows, gqa_paged_decode_fp8_oracle
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


def make(n, pool, seed, invalid=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, 40, 128, generator=g)
    qkv *= torch.exp2(torch.randint(-20, 20, (n, 40, 1), generator=g).float())  # scales of many sizes
    slots = torch.randperm(pool, generator=g)[:n].to(torch.int32)
    bad = torch.tensor([-1, pool, pool + 9, -2 ** 31, 2 ** 31 - 1], dtype=torch.int64).to(torch.int32)
    slots[:invalid] = bad[torch.arange(invalid) % 5]
    qkv = qkv.to(BF).cuda()
    return qkv[:, :32], qkv[:, 32:36], qkv[:, 36:], slots.cuda()


def fp8_cache(pool, fill=0xAB):
    return torch.full((pool, 528), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n,pool,invalid", [(1, 1, 0), (3, 10, 1), (64, 64, 0), (333, 1000, 40), (5000, 20000, 7)])
def test_append_fp8_bit_exact(n, pool, invalid):
    _, k, v, slots = make(n, pool, n, invalid)
    kc, vc = fp8_cache(pool), fp8_cache(pool)
    pkg.rope_kv_append(None, k, v, slots, kc, vc)
    ok = ((slots >= 0) & (slots < pool)).cpu()
    for cache, x in ((kc, k), (vc, v)):
        want = np.full((pool, 528), 0xAB, dtype=np.uint8)
        want[slots.cpu()[ok].numpy()] = sv.fp8_rows_oracle(x.cpu()[ok])
        assert np.array_equal(cache.cpu().numpy(), want)
    k2, v2 = fp8_cache(pool), fp8_cache(pool)
    pkg.kv_append_fp8(k.contiguous(), v.contiguous(), slots, k2, v2)
    assert torch.equal(k2, kc) and torch.equal(v2, vc)


def test_append_fp8_special_values():
    k = torch.zeros(6, 4, 128, dtype=BF)
    k[0] = torch.arange(512).view(4, 128).float() / 3
    k[1, 0, 0], k[1, 0, 1], k[1, 0, 2] = float("inf"), float("-inf"), 2.0   # saturate; the 2.0 keeps its own scale
    k[1, 1, 7], k[1, 1, 8] = float("nan"), -5.0
    k[1, 2] = float("inf")                                                   # nothing finite but zeros elsewhere
    k[2] = 448.0
    k[3, 0, :2] = torch.tensor([448.0, 450.0])
    k[4] = 1e-40                                                             # below the smallest scale's codes
    k[5] = torch.finfo(BF).max
    kc, vc = fp8_cache(6), fp8_cache(6)
    pkg.kv_append_fp8(k.cuda(), (-k).cuda(), torch.arange(6, dtype=torch.int32).cuda(), kc, vc)
    for cache, x in ((kc, k), (vc, -k)):
        want, got = sv.fp8_rows_oracle(x), cache.cpu().numpy()
        nan = (want[:, :512] & 0x7F) == 0x7F
        assert np.array_equal((got[:, :512] & 0x7F) == 0x7F, nan)  # NaN keeps no particular sign
        assert np.array_equal(np.where(nan, 0, got[:, :512]), np.where(nan, 0, want[:, :512]))
        assert np.array_equal(got[:, 512:], want[:, 512:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,offset,rot", [(1, 0, 128), (70, 0, 128), (33, 64, 64), (9, 0, 72), (5, 3, 18), (5, 1, 126),
                                          (4, 120, 2), (300, 4, 16)])
@pytest.mark.parametrize("cache", ["fp8", "bf16"])
def test_rope_append(layout, n, offset, rot, cache):
    pool = 2 * n + 3
    q, k, v, slots = make(n, pool, n + rot, invalid=n // 7)
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()
    freq, scale = pkg.rope_inv_freq(rot), 1.125
    freq = freq[0]
    if cache == "fp8":
        kc, vc = fp8_cache(pool), fp8_cache(pool)
    else:
        kc, vc = (torch.full((pool, 1, 4, 128), 3.0, dtype=BF, device="cuda") for _ in range(2))
    qo = pkg.rope_kv_append(q, k, v, slots, kc, vc, pos, freq, scale, offset, layout)
    ok = ((slots >= 0) & (slots < pool)).cpu().numpy()
    at = slots.cpu()[ok].long()

    def bound(x):
        return 2.0 ** -21 * scale * sv.rope_pair_size(x, rot, offset, layout)

    want, d = sv.rope_oracle(q, pos, freq, scale, offset, layout), bound(q)
    assert np.all(np.abs(sv.f64(qo) - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)
    want, d = sv.rope_oracle(k, pos, freq, scale, offset, layout)[ok], bound(k)[ok]
    others = torch.ones(pool, dtype=torch.bool)
    others[at] = False
    if cache == "bf16":
        got = sv.f64(kc)[at.numpy(), 0]
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)
        assert torch.equal(vc.cpu()[at, 0], v.cpu()[ok])
        assert torch.all(kc.cpu()[others] == 3.0) and torch.all(vc.cpu()[others] == 3.0)
        return
    rows = kc.cpu().numpy()[at.numpy()]
    got, s = dequantize_rows(rows), rows[:, 512:].copy().view("<f4").astype(np.float64)[:, :, None]
    assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * (np.abs(want) + d), 2.0 ** -10 * s) + d)
    ideal = sv.fp8_scale_oracle(want)[:, :, None]
    near = np.abs(want).max(-1, keepdims=True) / ideal > 447.9  # a key at the border may take the next scale
    assert np.all((s == ideal) | (near & (s == 2 * ideal)) | (s == ideal / 2) & (np.abs(want).max(-1, keepdims=True) / ideal < 224.1))
    assert np.array_equal(vc.cpu().numpy()[at.numpy()], sv.fp8_rows_oracle(v.cpu()[ok]))
    assert torch.all(kc.cpu()[others] == 0xAB) and torch.all(vc.cpu()[others] == 0xAB)


def test_append_rotation_of_q_in_place_and_without_q():
    q, k, v, slots = make(12, 30, 5)
    q = q.contiguous()
    pos, freq = torch.arange(12, dtype=torch.int32).cuda(), pkg.rope_inv_freq(128)[0]
    kc, vc, k2, v2 = (fp8_cache(30) for _ in range(4))
    want = pkg.rope_kv_append(q, k, v, slots, kc, vc, pos, freq)
    assert pkg.rope_kv_append(None, k, v, slots, k2, v2, pos, freq) is None
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
    pkg.rope_kv_append(q, k, v, slots, k2, v2, pos, freq, q_out=q)
    assert torch.equal(q, want)
    assert torch.equal(want, pkg.rope(q.clone().copy_(make(12, 30, 5)[0]), pos, freq))


def test_append_far_pages():
    """A page whose byte offset passes 32 bits: 528 * 8.2 M rows."""
    pool = 8_200_000
    if torch.cuda.mem_get_info()[0] < 3 * pool * 528:
        pytest.skip("needs 13 GB")
    _, k, v, _ = make(2, 2, 77)
    kc, vc = (torch.zeros(pool, 528, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.tensor([pool - 1, 0], dtype=torch.int32).cuda()
    pkg.kv_append_fp8(k.contiguous(), v.contiguous(), slots, kc, vc)
    want = torch.from_numpy(sv.fp8_rows_oracle(k.cpu()))
    assert torch.equal(kc[slots.long()].cpu(), want)
    ko, vo = pkg.kv_read_fp8(kc, vc, slots)
    assert np.array_equal(sv.f64(ko), np.asarray(torch.from_numpy(dequantize_rows(want.numpy())).bfloat16().double()))


@pytest.mark.parametrize("n", [1, 2, 31, 777, 20000])
def test_read_fp8_bit_exact(n):
    g = torch.Generator().manual_seed(n)
    pool = 501
    caches = []
    for _ in range(2):
        c = torch.randint(0, 256, (pool, 528), generator=g, dtype=torch.uint8)
        c[:, :512][(c[:, :512] & 0x7F) == 0x7F] = 1
        c[:, 512:] = torch.from_numpy((torch.randn(pool, 4, generator=g).numpy() * 3).astype("<f4").view(np.uint8))
        caches.append(c)
    idx = torch.randint(0, pool, (n,), generator=g, dtype=torch.int32)
    idx[::5] = torch.tensor([-1, pool, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64).to(torch.int32)[torch.arange(len(idx[::5])) % 4]
    ko, vo = pkg.kv_read_fp8(caches[0].cuda(), caches[1].cuda(), idx.cuda())
    ok = ((idx >= 0) & (idx < pool)).numpy()
    for c, got in zip(caches, (ko, vo)):
        rows = c.numpy()[np.where(ok, idx.numpy(), 0)]
        vals = torch.from_numpy(dequantize_rows(rows)).float().bfloat16()  # the product is rounded to fp32, then bf16
        vals[~torch.from_numpy(ok)] = 0
        assert torch.equal(got.cpu(), vals)


def test_read_nan_codes_and_repeated_pages():
    c = fp8_cache(3, 0x7F)
    c[:, 512:] = torch.ones(3, 4).view(torch.uint8).cuda()
    idx = torch.tensor([1, 1, 2, 1], dtype=torch.int32).cuda()
    ko, vo = pkg.kv_read_fp8(c, c, idx)
    assert torch.isnan(ko).all() and torch.isnan(vo).all()
    e = pkg.kv_read_fp8(c, c, idx[:0])
    assert e[0].shape == (0, 4, 128)


def test_step_on_an_fp8_cache():
    """Append a prompt and a step (rotated, quantised), decode, and read the batch back: each against the oracle
    fed with what the cache holds."""
    g = torch.Generator().manual_seed(21)
    lens, pool = [7, 0, 130, 1], 400
    total = sum(lens) + len(lens)
    qkv = torch.randn(total, 40, 128, generator=g).to(BF).cuda()
    pages = torch.randperm(pool, generator=g)[:total].to(torch.int32)
    kc, vc = fp8_cache(pool, 0x7F), fp8_cache(pool, 0x7F)  # NaN codes wherever nothing is stored
    freq, scale = pkg.rope_inv_freq(128, scaling="by_parts", factor=4.0)
    indices, ptr, last, at = [], [0], [], 0
    for n in lens:
        pos = torch.arange(n + 1, dtype=torch.int32).cuda()
        rows, mine = qkv[at:at + n + 1], pages[at:at + n + 1].cuda()
        if n:
            pkg.rope_kv_append(None, rows[:n, 32:36], rows[:n, 36:], mine[:n], kc, vc, pos[:n], freq, scale)
        last.append(pkg.rope_kv_append(rows[n:, :32], rows[n:, 32:36], rows[n:, 36:], mine[n:], kc, vc, pos[n:], freq, scale))
        indices.append(mine)
        ptr.append(ptr[-1] + n + 1)
        at += n + 1
    q, indices = torch.cat(last), torch.cat(indices)
    indptr = torch.tensor(ptr, dtype=torch.int32).cuda()
    out, lse = pkg.run_fp8(q, kc, vc, indptr, indices)
    o_ref, l_ref = gqa_paged_decode_fp8_oracle(q.cpu(), kc.cpu(), vc.cpu(), indptr.cpu(), indices.cpu(), 128 ** -0.5)
    assert np.all(np.abs(sv.f64(out) - o_ref) <= 2e-2 + 2e-2 * np.abs(o_ref))
    assert np.abs(sv.f64(lse) - l_ref).max() <= 1e-3
    ko, vo = pkg.kv_read_fp8(kc, vc, indices)
    assert torch.isfinite(ko).all() and torch.isfinite(vo).all()
    # the pages read back serve the bf16 decode: identity page table
    ids = torch.arange(total, dtype=torch.int32).cuda()
    out2, lse2 = pkg.run(q, ko.view(total, 1, 4, 128), vo.view(total, 1, 4, 128), indptr, ids)
    assert np.all(np.abs(sv.f64(out2) - o_ref) <= 2e-2 + 2e-2 * np.abs(o_ref))
    assert np.abs(sv.f64(lse2) - l_ref).max() <= 1e-3
    assert _lib.gqa_paged_decode_device_error() == 0


def test_append_graph_and_streams():
    q, k, v, slots = make(50, 200, 6)
    pos, freq = torch.arange(50, dtype=torch.int32).cuda(), pkg.rope_inv_freq(128)[0]
    kc, vc, k2, v2 = (fp8_cache(200) for _ in range(4))
    want = pkg.rope_kv_append(q, k, v, slots, kc, vc, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.rope_kv_append(q, k, v, slots, k2, v2, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, k2) and torch.equal(vc, v2)
    k2.fill_(0xAB)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        pkg.rope_kv_append(q, k, v, slots, k2, v2, pos, freq, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(k2, kc)


def test_write_refusals():
    q, k, v, slots = make(4, 9, 1)
    kc, vc = fp8_cache(9), fp8_cache(9)
    pos, freq = torch.arange(4, dtype=torch.int32).cuda(), pkg.rope_inv_freq(128)[0]
    bf = torch.zeros(9, 1, 4, 128, dtype=BF, device="cuda")
    for bad in (lambda: pkg.rope_kv_append(q, k, v, slots, kc, bf, pos, freq),
                lambda: pkg.rope_kv_append(q, k, v, slots, kc[:, :500], vc[:, :500], pos, freq),
                lambda: pkg.rope_kv_append(q, k[:3], v, slots, kc, vc, pos, freq),
                lambda: pkg.rope_kv_append(q[:, :16], k, v, slots, kc, vc, pos, freq),
                lambda: pkg.rope_kv_append(q, k.float(), v, slots, kc, vc, pos, freq),
                lambda: pkg.rope_kv_append(q, k, v, slots.long(), kc, vc, pos, freq),
                lambda: pkg.rope_kv_append(q, k, v, slots, kc, vc, None, freq),
                lambda: pkg.rope_kv_append(q, k, v, slots, kc, vc, pos[:2], freq),
                lambda: pkg.rope_kv_append(None, k, v, slots, kc, vc, pos, freq, q_out=q),
                lambda: pkg.kv_append_fp8(k, v, slots, bf, bf), lambda: pkg.kv_read_fp8(bf, bf, slots),
                lambda: pkg.kv_read_fp8(kc, vc, slots.long()), lambda: pkg.kv_read_fp8(kc, vc, slots, k_out=k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkg.GqaError):
        pkg.rope_kv_append(q, k, v, slots, kc, vc, pos, freq, rot_offset=2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,rotate", [(1, True), (37, True), (37, False), (4000, True)])
def test_latent_append(layout, n, rotate):
    g = torch.Generator().manual_seed(n)
    row = torch.randn(n, 600, generator=g).to(BF).cuda()
    lat, kr = row[:, :512], row[:, 520:584]  # views of one fused row
    blocks, page = n // 16 + 3, 16
    cache = torch.full((blocks, page, 1, 576), 2.0, dtype=BF, device="cuda")
    slots = torch.randperm(blocks * page, generator=g)[:n].to(torch.int32)
    slots[: n // 9] = -1
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    freq = pkg.rope_inv_freq(64)[0] if rotate else None
    pkg.mla_kv_append(lat, kr, slots.cuda(), cache, pos, freq, 1.25, layout)
    flat, ok = cache.view(-1, 576).cpu(), (slots >= 0).numpy()
    at = slots[ok].long()
    assert torch.equal(flat[at, :512], lat.cpu()[ok])
    if rotate:
        want = sv.rope_oracle(kr[:, None], pos, freq, 1.25, 0, layout)[ok, 0]
        d = 2.0 ** -21 * 1.25 * sv.rope_pair_size(kr[:, None], 64, 0, layout)[ok, 0]
        assert np.all(np.abs(sv.f64(flat[at, 512:]) - want) <= 2.0 ** -8 * (np.abs(want) + d) + d)
    else:
        assert torch.equal(flat[at, 512:], kr.cpu()[ok])
    others = torch.ones(blocks * page, dtype=torch.bool)
    others[at] = False
    assert torch.all(flat[others] == 2.0)


def test_missing_tensors_and_offsets_past_an_int_are_refused():
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    k, q = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 32, 128, dtype=torch.bfloat16, device="cuda")
    c, bc = torch.zeros(8, 528, dtype=torch.uint8, device="cuda"), torch.zeros(8, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    lat, row = torch.zeros(4, 16, 1, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 576, dtype=torch.bfloat16, device="cuda")
    w, freq = torch.zeros(2, 256, 512, dtype=torch.bfloat16, device="cuda"), pkg.rope_inv_freq(64)[0]
    ql, cu = torch.zeros(3, 2, 192, dtype=torch.bfloat16, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    calls = [(pkg.rope, dict(x=q, positions=i, inv_freq=freq), ["x"]),
             (pkg.rope_kv_append, dict(q=q, k_new=k, v_new=k, slots=i, k_cache=bc, v_cache=bc),
              ["k_new", "v_new", "slots", "k_cache", "v_cache"]),
             (pkg.kv_append_fp8, dict(k_new=k, v_new=k, slots=i, k_cache=c, v_cache=c),
              ["k_new", "v_new", "slots", "k_cache", "v_cache"]),
             (pkg.kv_read_fp8, dict(k_cache=c, v_cache=c, indices=i), ["k_cache", "v_cache", "indices"]),
             (pkg.mla_kv_append, dict(latent=row[:, :512], k_rope=row[:, 512:], slots=i, kv_cache=lat),
              ["latent", "k_rope", "slots", "kv_cache"]),
             (pkg.mla_absorb_q, dict(q=ql, w_kv=w), ["q", "w_kv"]),
             (pkg.mla_expand_out, dict(o_latent=ql.new_zeros(3, 2, 512), w_kv=w), ["o_latent", "w_kv"]),
             (pkg.mla_prefill, dict(q=ql, w_kv=w, kv_cache=lat, block_table=i[None], cache_seqlens=i[:1], cu_seqlens_q=cu),
              ["q", "w_kv", "kv_cache", "block_table", "cache_seqlens", "cu_seqlens_q"])]
    for fn, args, required in calls:
        fn(**args)
        for name in required:
            with pytest.raises(TypeError, match=name):
                fn(**dict(args, **{name: None}))
    for offset in (-1, 2 ** 31, 2 ** 32):
        with pytest.raises(ValueError):
            pkg.rope(q, i, freq, rot_offset=offset)
        with pytest.raises(ValueError):
            pkg.rope_kv_append(q, k, k, i, bc, bc, i, freq, rot_offset=offset)
    with pytest.raises(ValueError):
        pkg.mla_prefill(ql, w, lat, i[None], i[:1], cu, max_kv_tokens=1 << 64)
