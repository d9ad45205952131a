"""Timed cases of the serving-side operators around the paged decode: rotary positions, the quantised cache's write
and read, and latent attention's projections (absorbed form) and prompt pass (expanded form).

Each case has a plain form in elementary torch operations in 32 bits (angles in 64) and the library's own call. Sizes
follow the library's shapes: 32 query heads over 4 KV heads of dimension 128 with page size 1, and latent rows of
512 + 64 values with heads of 128 + 64 (keys) and 128 (values).
"""
import math

import torch

own = False

QO, KV, D = 32, 4, 128                    # the paged GQA shape
LAT, ROPE, NOPE, DV = 512, 64, 128, 128   # the latent-attention shape
DQK, ROW = NOPE + ROPE, LAT + ROPE
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: the 32 query and 4 key heads of a fused qkv row, whole heads, half layout
        {"name": "rope step", "op": "rope", "tokens": 64, "heads": 36, "tail": 4, "dim": 128, "offset": 0, "rot": 128,
         "layout": "half", "type": "bf16", "stretch": 1.0, "span": 8192, "inverse": False},
        # a prompt of 32768 tokens, interleaved pairs in the last 64 of 192 values, stretched for a long context
        {"name": "rope prompt", "op": "rope", "tokens": 32768, "heads": 16, "tail": 0, "dim": 192, "offset": 128,
         "rot": 64, "layout": "interleaved", "type": "bf16", "stretch": 16.0, "span": 1048576, "inverse": False},
        # one decode step of 256 sequences into an FP8 cache: Q and K rotated, K and V quantised and stored
        {"name": "append step", "op": "append", "tokens": 256, "pool": 65536, "skip": 7, "rot": 128, "layout": "half",
         "stretch": 1.0, "span": 131072, "cache": "fp8"},
        # a prompt chunk of 16384 tokens into an FP8 cache
        {"name": "append prompt", "op": "append", "tokens": 16384, "pool": 50000, "skip": 0, "rot": 128,
         "layout": "half", "stretch": 4.0, "span": 131072, "cache": "fp8"},
        # the cached prefix of one short request read back (777 tokens scattered over the pool)
        {"name": "read prefix", "op": "read", "tokens": 777, "pool": 20000},
        # the whole batch's cache read back: 262144 tokens
        {"name": "read batch", "op": "read", "tokens": 262144, "pool": 300000},
        # a step of 4 sequences on a 16-head shard: queries into the latent space
        {"name": "absorb step", "op": "absorb", "tokens": 4, "heads": 16, "rotate": True},
        # a step of 128 sequences, 128 heads: queries into the latent space
        {"name": "absorb batch", "op": "absorb", "tokens": 128, "heads": 128, "rotate": True},
        # the same step's latent outputs back to 128 values a head
        {"name": "expand batch", "op": "expand", "tokens": 128, "heads": 128},
        # five short ragged prompts, one of a single token and one empty, 16 heads
        {"name": "prefill ragged", "op": "prefill", "heads": 16, "page": 64, "causal": True,
         "lens": "130/130,1/1,0/0,47/300,333/333"},
        # one prompt of 8192 tokens on a 16-head shard
        {"name": "prefill prompt", "op": "prefill", "heads": 16, "page": 64, "causal": True, "lens": "8192/8192"},
        # a chunk of 1024 tokens behind a cached prefix, 32 heads
        {"name": "prefill chunk", "op": "prefill", "heads": 32, "page": 32, "causal": True, "lens": "1024/16384"},
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "absorb", "expand", "prefill"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        tokens = log_int(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "heads": rng.randint(1, 36), "tail": rng.choice([0, 0, 1, 8]), "dim": dim,
                "offset": rng.choice([0, dim - rot, rng.randint(0, dim - rot)]), "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "type": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "stretch": rng.choice([1.0, 1.0, 8.0, 32.0]), "span": log_int(rng, 4096, 1048576),
                "inverse": rng.random() < 0.25}
    if op == "append":
        tokens = log_int(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "pool": tokens + log_int(rng, 1, 40000), "skip": rng.choice([0, 0, 2, 5]),
                "rot": rng.choice([0, 64, 128, 128, 2 * rng.randint(1, 64)]),
                "layout": rng.choice(["half", "interleaved"]), "stretch": rng.choice([1.0, 8.0]),
                "span": log_int(rng, 4096, 1048576), "cache": rng.choice(["fp8", "fp8", "bf16"])}
    if op == "read":
        tokens = log_int(rng, 1, 262144)
        return {"op": op, "tokens": tokens, "pool": log_int(rng, 1000, 300000)}
    if op in ("absorb", "expand"):
        case = {"op": op, "tokens": log_int(rng, 1, 512), "heads": rng.choice([1, 8, 16, 20, 32, 64, 128])}
        return dict(case, rotate=rng.random() < 0.7) if op == "absorb" else case
    heads = rng.choice([1, 3, 8, 16, 32, 128])
    for _ in range(100):
        lens = []
        for _ in range(rng.randint(1, 6)):
            nq = 0 if rng.random() < 0.1 else log_int(rng, 1, 4096)
            lens.append((nq, nq + (0 if rng.random() < 0.5 else log_int(rng, 1, 12000))))
        mq, mk = max(a for a, _ in lens), max(b for _, b in lens)
        if 0 < mq and len(lens) * heads * mq * mk <= 400_000_000:
            break
    else:
        lens = [(log_int(rng, 1, 512), 512)]
    return {"op": op, "heads": heads, "page": rng.choice([1, 16, 32, 64, 128]), "causal": rng.random() < 0.85,
            "lens": ",".join("%d/%d" % x for x in lens)}


def lengths(case):
    return [tuple(int(x) for x in part.split("/")) for part in case["lens"].split(",")]


def work(case):
    op, n = case["op"], case.get("tokens", 0)
    if op == "rope":
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": 2 * n * case["heads"] * case["dim"] * size + 4 * n, "flops": 3 * n * case["heads"] * case["rot"]}
    if op == "append":
        row = 528 if case["cache"] == "fp8" else 1024
        live = n - (n // case["skip"] if case["skip"] else 0)
        return {"bytes": 2 * n * QO * D * 2 + live * 2 * (1024 + row) + 8 * n, "flops": 3 * n * (QO + KV) * case["rot"]}
    if op == "read":
        return {"bytes": n * (4 + 2 * 528 + 2 * 1024), "flops": 2 * n * KV * D}
    h = case["heads"]
    if op == "absorb":
        return {"bytes": h * NOPE * LAT * 2 + n * h * (DQK + ROW) * 2, "flops": 2 * n * h * NOPE * LAT}
    if op == "expand":
        return {"bytes": h * DV * LAT * 2 + n * h * (LAT + DV) * 2, "flops": 2 * n * h * DV * LAT}
    pairs = sum(nq * nk - nq * (nq - 1) // 2 if case["causal"] else nq * nk for nq, nk in lengths(case))
    tq, tk = (sum(x[i] for x in lengths(case)) for i in (0, 1))
    return {"bytes": tq * h * (DQK + DV) * 2 + tk * ROW * 2 + h * (NOPE + DV) * LAT * 2,
            "flops": 2 * h * (pairs * (DQK + DV) + tk * LAT * (NOPE + DV))}


# ------------------------------------------------------------------------------------------------------------ inputs
def inv_freq(rot, stretch, trained=4096.0):
    """Radians a position of each pair (base 10000); stretched pairs turn `stretch` times slower unless they already
    make 32 turns over the trained length, with a linear ramp down to one turn."""
    got = []
    for i in range(rot // 2):
        f = 10000.0 ** (-2.0 * i / rot)
        turns = trained * f / (2.0 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0)) if stretch > 1 else 1.0
        got.append(f * keep + f / stretch * (1.0 - keep))
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, n = case["op"], case.get("tokens", 0)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    def below(hi, *shape):
        return torch.randint(0, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = dict(case)
    if op == "rope":
        rows = normal(n, case["heads"] + case["tail"], case["dim"], dtype=TYPES[case["type"]])
        s |= {"x": rows[:, :case["heads"]], "positions": below(case["span"], n),
              "inv_freq": inv_freq(case["rot"], case["stretch"]),
              "scale": 1.0 + 0.1 * math.log(case["stretch"])}
    elif op == "append":
        qkv = normal(n, QO + 2 * KV, D)
        # keys carry a few large channels, as trained models' do
        qkv[:, QO:QO + KV, ::32] *= 6
        slots = torch.randperm(case["pool"], generator=g, device="cuda")[:n].to(torch.int32)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1  # padded tokens of the step
        s |= {"q": qkv[:, :QO], "k": qkv[:, QO:QO + KV], "v": qkv[:, QO + KV:], "slots": slots,
              "positions": below(case["span"], n), "scale": 1.0 + 0.1 * math.log(case["stretch"]),
              "inv_freq": inv_freq(case["rot"], case["stretch"]) if case["rot"] else None}
        for name in ("k_cache", "v_cache"):
            if case["cache"] == "fp8":
                c = torch.zeros(case["pool"], 528, dtype=torch.uint8, device="cuda")
                s |= {name: c, name + "_codes": c[:, :512].view(torch.float8_e4m3fn),
                      name + "_scales": c[:, 512:].view(torch.float32)}
            else:
                s[name] = torch.zeros(case["pool"], 1, KV, D, dtype=torch.bfloat16, device="cuda")
    elif op == "read":
        for name in ("k_cache", "v_cache"):
            c = torch.empty(case["pool"], 528, dtype=torch.uint8, device="cuda")
            c[:, :512] = normal(case["pool"], 512, dtype=torch.float32, std=90.0).clamp_(-448, 448) \
                .to(torch.float8_e4m3fn).view(torch.uint8)
            c[:, 512:] = (normal(case["pool"], KV, dtype=torch.float32).abs_().add_(0.1) / 128).view(torch.uint8)
            s[name] = c
        s["indices"] = below(case["pool"], n)
    elif op in ("absorb", "expand"):
        h = case["heads"]
        s["w_kv"] = normal(h, NOPE + DV, LAT, std=LAT ** -0.5)
        if op == "absorb":
            s |= {"q": normal(n, h, DQK), "positions": below(65536, n), "inv_freq": inv_freq(ROPE, 1.0)}
        else:
            s["latent"] = normal(n, h, LAT, std=0.3)
    else:
        h, page, lens = case["heads"], case["page"], lengths(case)
        width = max(1, max(-(-nk // page) for _, nk in lens))
        blocks = sum(-(-nk // page) for _, nk in lens) + 7
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        ids, at = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).cpu(), 0
        for b, (_, nk) in enumerate(lens):
            used = -(-nk // page)
            table[b, :used] = ids[at:at + used]
            at += used
        cu = [0]
        for nq, _ in lens:
            cu.append(cu[-1] + nq)
        s |= {"q": normal(cu[-1], h, DQK), "w_kv": normal(h, NOPE + DV, LAT, std=LAT ** -0.5),
              "kv_cache": normal(blocks, page, 1, ROW), "block_table": table.cuda(),
              "seqlens": torch.tensor([nk for _, nk in lens], dtype=torch.int32, device="cuda"),
              "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"), "total_kv": sum(nk for _, nk in lens),
              "max_q": max(nq for nq, _ in lens), "max_kv": max(1, max(nk for _, nk in lens))}
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def rotated(x, positions, freq, scale, offset, layout, inverse=False):
    """fp32 copy of x [tokens, heads, dim] with the pairs of [offset, offset + 2 len(freq)) turned."""
    angle = positions.double()[:, None] * freq
    cos = (angle.cos() * scale).float()[:, None]
    sin = (angle.sin() * (-scale if inverse else scale)).float()[:, None]
    y, half = x.float(), freq.numel()
    part = y[..., offset:offset + 2 * half]
    a, b = (part[..., :half], part[..., half:]) if layout == "half" else (part[..., ::2], part[..., 1::2])
    pair = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.cat(pair, -1) if layout == "half" else torch.stack(pair, -1).flatten(-2)
    return torch.cat([y[..., :offset], turned, y[..., offset + 2 * half:]], -1)


def quantised(x):
    """e4m3 codes and power-of-two scales of x [tokens, heads, 128] (fp32): the smallest scale that keeps every
    value within 448."""
    top = x.abs().amax(-1)
    mantissa, exponent = torch.frexp(top)
    e = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def plain_append(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["rot"]:
        q = rotated(s["q"], s["positions"], s["inv_freq"], s["scale"], 0, s["layout"])
        k = rotated(s["k"], s["positions"], s["inv_freq"], s["scale"], 0, s["layout"])
    keep = (s["slots"] >= 0) & (s["slots"] < s["pool"])
    to = s["slots"][keep].long()
    if s["cache"] == "bf16":
        s["k_cache"][to, 0] = k[keep].bfloat16()
        s["v_cache"][to, 0] = v[keep].bfloat16()
        return {"q": q.bfloat16(), "k": s["k_cache"], "v": s["v_cache"]}
    kc, ks = quantised(k[keep])
    vc, vs = quantised(v[keep])
    s["k_cache"][to] = torch.cat([kc.flatten(1).view(torch.uint8), ks.view(torch.uint8)], 1)
    s["v_cache"][to] = torch.cat([vc.flatten(1).view(torch.uint8), vs.view(torch.uint8)], 1)
    return appended(s, q.bfloat16())


def appended(s, q):
    if s["cache"] == "bf16":
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    return {"q": q, "k": s["k_cache_codes"], "k_scale": s["k_cache_scales"],
            "v": s["v_cache_codes"], "v_scale": s["v_cache_scales"]}


def plain_read(cache, indices):
    rows = cache[indices.long()]
    codes = rows[:, :512].contiguous().view(torch.float8_e4m3fn).float().view(-1, KV, D)
    return (codes * rows[:, 512:].contiguous().view(torch.float32)[..., None]).bfloat16()


def plain_prefill(s):
    b, t = len(lengths(s)), torch.arange(s["max_kv"], device="cuda")
    page, n = s["page"], s["seqlens"].long()[:, None]
    slot = s["block_table"].long()[:, t // page] * page + t % page
    live = t < n
    rows = s["kv_cache"].view(-1, ROW)[slot.clamp(min=0)].float() * live[..., None]
    w = s["w_kv"].float()
    k = torch.matmul(rows[:, None, :, :LAT], w[:, :NOPE].transpose(1, 2))         # [B, h, t, 128]
    v = torch.matmul(rows[:, None, :, :LAT], w[:, NOPE:].transpose(1, 2))
    k = torch.cat([k, rows[:, None, :, LAT:].expand(-1, s["heads"], -1, -1)], -1)
    i = torch.arange(s["max_q"], device="cuda")
    nq = (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None]
    mine = i < nq
    q = s["q"][(s["cu_q"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    score = torch.matmul(q.transpose(1, 2), k.transpose(2, 3)) * DQK ** -0.5      # [B, h, i, t]
    seen = live[:, None] & ((t <= (n - nq + i)[..., None]) | (not s["causal"]))
    score = score.masked_fill(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.clamp(min=1e-30)
    return out.transpose(1, 2)[mine].bfloat16()


def run(s):
    op = s["op"]
    if own:
        import paged_kv_gqa_split_gb300 as pkg
        if op == "rope":
            return pkg.rope(s["x"], s["positions"], s["inv_freq"], scale=s["scale"], rot_offset=s["offset"],
                            layout=s["layout"], inverse=s["inverse"])
        if op == "append":
            q = pkg.rope_kv_append(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["positions"],
                                   s["inv_freq"], scale=s["scale"], layout=s["layout"])
            return appended(s, q)
        if op == "read":
            return pkg.kv_read_fp8(s["k_cache"], s["v_cache"], s["indices"])
        if op == "absorb":
            turn = s["inv_freq"] if s["rotate"] else None
            return pkg.mla_absorb_q(s["q"], s["w_kv"], s["positions"], turn, layout="interleaved")
        if op == "expand":
            return pkg.mla_expand_out(s["latent"], s["w_kv"])
        return pkg.mla_prefill(s["q"], s["w_kv"], s["kv_cache"], s["block_table"], s["seqlens"], s["cu_q"],
                               causal=s["causal"], max_kv_tokens=s["total_kv"], with_lse=False)[0]
    if op == "rope":
        y = rotated(s["x"], s["positions"], s["inv_freq"], s["scale"], s["offset"], s["layout"], s["inverse"])
        return y.to(s["x"].dtype)
    if op == "append":
        return plain_append(s)
    if op == "read":
        return plain_read(s["k_cache"], s["indices"]), plain_read(s["v_cache"], s["indices"])
    if op == "absorb":
        q = s["q"].float()
        lat = torch.matmul(q[..., :NOPE].transpose(0, 1), s["w_kv"][:, :NOPE].float()).transpose(0, 1)
        turn = s["q"][..., NOPE:]
        turn = rotated(turn, s["positions"], s["inv_freq"], 1.0, 0, "interleaved") if s["rotate"] else turn.float()
        return torch.cat([lat, turn], -1).bfloat16()
    if op == "expand":
        w = s["w_kv"][:, NOPE:].float().transpose(1, 2)
        return torch.matmul(s["latent"].float().transpose(0, 1), w).transpose(0, 1).contiguous().bfloat16()
    return plain_prefill(s)


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def turn64(x, positions, freq, scale, offset, layout, inverse=False):
    y, r = x.double().clone(), freq.numel()
    first = torch.arange(r, device="cuda") + offset if layout == "half" else 2 * torch.arange(r, device="cuda") + offset
    second = first + (r if layout == "half" else 1)
    z = torch.complex(y[..., first], y[..., second])
    a = torch.outer(positions.double(), freq)
    z = z * (torch.polar(torch.full_like(a, scale), -a if inverse else a))[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def e4m3_64(x):
    """Float64 x rounded to the nearest e4m3 value, ties to the even code."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def codes64(x):
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448) - 1e-12))  # log2 of an exact power may come out an ulp high
    scale = torch.where(top > 0, scale, torch.ones_like(scale))
    return e4m3_64(x / scale), scale[..., 0]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        return turn64(s["x"], s["positions"], s["inv_freq"], s["scale"], s["offset"], s["layout"], s["inverse"])
    if op == "append":
        q, k, v = (s[x].double() for x in "qkv")
        if s["rot"]:
            q, k = (turn64(s[x], s["positions"], s["inv_freq"], s["scale"], 0, s["layout"]) for x in "qk")
        got, keep = {"q": q}, s["slots"] >= 0
        for name, x in (("k", k), ("v", v)):
            if case["cache"] == "bf16":
                got[name] = torch.zeros(case["pool"], 1, KV, D, dtype=torch.float64, device="cuda")
                got[name][s["slots"][keep].long(), 0] = x[keep]
                continue
            got[name] = torch.zeros(case["pool"], KV * D, dtype=torch.float64, device="cuda")
            got[name + "_scale"] = torch.zeros(case["pool"], KV, dtype=torch.float64, device="cuda")
            codes, scale = codes64(x[keep])
            got[name][s["slots"][keep].long()] = codes.flatten(1)
            got[name + "_scale"][s["slots"][keep].long()] = scale
        return got
    if op == "read":
        got = []
        for name in ("k_cache", "v_cache"):
            rows = s[name].index_select(0, s["indices"])
            vals = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double().unflatten(1, (KV, D))
            got.append(vals * rows[:, 512:].contiguous().view(torch.float32).double().unsqueeze(-1))
        return tuple(got)
    if op == "absorb":
        lat = torch.einsum("nhd,hdl->nhl", s["q"][..., :NOPE].double(), s["w_kv"][:, :NOPE].double())
        turn = s["q"][..., NOPE:].double()
        if s["rotate"]:
            turn = turn64(s["q"][..., NOPE:], s["positions"], s["inv_freq"], 1.0, 0, "interleaved")
        return torch.cat([lat, turn], -1)
    if op == "expand":
        return torch.einsum("nhl,hdl->nhd", s["latent"].double(), s["w_kv"][:, NOPE:].double())
    h = case["heads"]
    out = torch.zeros(s["q"].shape[0], h, DV, dtype=torch.float64, device="cuda")
    first = 0
    for b, (nq, nk) in enumerate(lengths(case)):
        if nq and nk:
            pages = s["block_table"][b, : -(-nk // case["page"])].long()
            rows = s["kv_cache"][pages].reshape(-1, ROW)[:nk].double()
            for a in range(h):
                full = rows[:, :LAT] @ s["w_kv"][a].double().t()
                key = torch.cat([full[:, :NOPE], rows[:, LAT:]], 1)
                z = (s["q"][first:first + nq, a].double() @ key.t()) / math.sqrt(DQK)
                if case["causal"]:
                    z.masked_fill_(torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1), -math.inf)
                out[first:first + nq, a] = torch.softmax(z, 1) @ full[:, NOPE:]
        first += nq
    return out
