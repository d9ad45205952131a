"""Timed cases of the decode's forms for long and shared contexts over the paged cache: a batch that shares prefixes, the
tokens' blocks bounded, chosen and attended to, attention weights accumulated beside the decode, and the eviction by
them.

Each case has a plain form in elementary torch operations in 32 bits (block scores, whose order decides, in 64) and the
library's own call. Sizes follow the library's shapes: 32 query heads over 4 KV heads of dimension 128, page size 1 for
the CSR page tables, blocks of several tokens for the block tables.
"""
import math
import random

import torch

own = False

QO, KV, D, GROUP = 32, 4, 128, 8
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step of 8 conversations behind one system prompt, their own turns still short
        {"name": "shared step", "op": "shared", "cache": "bf16", "prefixes": "2048", "members": "8", "alone": 0,
         "own": "1-256", "mix": 1},
        # one step of 128 requests about one document of 16384 tokens
        {"name": "shared batch", "op": "shared", "cache": "bf16", "prefixes": "16384", "members": "128", "alone": 0,
         "own": "64-1024", "mix": 2},
        # several prefixes at once in an FP8 cache, one of them empty, some requests with none, some with nothing else
        {"name": "shared groups fp8", "op": "shared", "cache": "fp8", "prefixes": "5000,0,777,32768",
         "members": "37,3,1,20", "alone": 3, "own": "0-600", "mix": 3},
        # the new tokens of one step of 64 requests go into their last blocks' bounds
        {"name": "bounds step", "op": "bounds", "page": 64, "lens": "100-8192", "requests": 64, "fresh": 1, "mix": 4},
        # four prompts of 32768 tokens have just been cached
        {"name": "bounds prompt", "op": "bounds", "page": 32, "lens": "32768-32768", "requests": 4, "fresh": 32768,
         "mix": 5},
        # one step of a single request at 131072 tokens, 4096 of them attended to
        {"name": "blocks long", "op": "blocks", "page": 64, "lens": "131072-131072", "requests": 1, "rows": 1, "top": 64,
         "first": 1, "last": 2, "mix": 6},
        # one step of 128 requests of 1024 to 8192 tokens, 2048 of them attended to
        {"name": "blocks batch", "op": "blocks", "page": 32, "lens": "1024-8192", "requests": 128, "rows": 1, "top": 64,
         "first": 1, "last": 1, "mix": 7},
        # five drafted tokens a request, small blocks, contexts from nothing to longer than what is chosen
        {"name": "blocks drafts", "op": "blocks", "page": 16, "lens": "0-3000", "requests": 11, "rows": 5, "top": 37,
         "first": 0, "last": 3, "mix": 8},
        # one step of 16 short requests whose weights are kept
        {"name": "weigh step", "op": "weigh", "cache": "bf16", "lens": "0-700", "requests": 16, "room": 1024, "decay": 1.0,
         "mix": 9},
        # one step of 64 requests of 512 to 4096 tokens in an FP8 cache, old weights fading
        {"name": "weigh batch", "op": "weigh", "cache": "fp8", "lens": "512-4096", "requests": 64, "room": 4096,
         "decay": 0.98, "mix": 10},
        # 48 requests that have grown past 2048 tokens, or not yet, are cut back
        {"name": "evict step", "op": "evict", "lens": "1900-2300", "requests": 48, "room": 2304, "budget": 2048,
         "first": 4, "last": 256, "mix": 11},
        # two prompts of up to 131072 tokens are cut to 16384
        {"name": "evict prompts", "op": "evict", "lens": "100000-131072", "requests": 2, "room": 131072, "budget": 16384,
         "first": 64, "last": 1000, "mix": 12},
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op, mix = rng.choice(["shared", "shared", "bounds", "blocks", "blocks", "weigh", "evict"]), rng.randrange(1 << 30)
    if op == "shared":
        groups = rng.choice([1, 1, 2, rng.randint(1, 6)])
        members = [log_int(rng, 1, 128 // groups) for _ in range(groups)]
        prefixes = [0 if rng.random() < 0.1 else log_int(rng, 1, 16384) for _ in range(groups)]
        hi = log_int(rng, 1, 1000)
        return {"op": op, "cache": rng.choice(["bf16", "fp8"]), "prefixes": ",".join(map(str, prefixes)),
                "members": ",".join(map(str, members)), "alone": rng.choice([0, 0, 0, 2]),
                "own": "%d-%d" % (rng.randint(0, hi), hi), "mix": mix}
    if op == "bounds":
        requests = log_int(rng, 1, 64)
        hi = log_int(rng, 1, 131072 // requests)
        return {"op": op, "page": rng.choice([1, 8, 16, 32, 48, 64, 128]), "lens": "%d-%d" % (rng.randint(0, hi), hi),
                "requests": requests, "fresh": rng.choice([1, 1, log_int(rng, 1, hi), hi]), "mix": mix}
    if op == "blocks":
        page = rng.choice([8, 16, 16, 32, 32, 64, 64, 128])
        requests, rows = log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
        hi = log_int(rng, 1, min(131072, 262144 // requests))
        first, last = rng.choice([0, 1, 1, 2]), rng.choice([0, 1, 1, 4])
        top = max(1, first + last, log_int(rng, 1, max(1, min(256, 1048576 // (page * requests * rows)))))
        return {"op": op, "page": page, "lens": "%d-%d" % (rng.randint(0, hi), hi), "requests": requests, "rows": rows,
                "top": top, "first": first, "last": last, "mix": mix}
    requests = log_int(rng, 1, 64)
    hi = log_int(rng, 1, 131072 // requests)
    lens, room = "%d-%d" % (rng.randint(0, hi), hi), hi + rng.randint(0, 100)
    if op == "weigh":
        return {"op": op, "cache": rng.choice(["bf16", "fp8"]), "lens": lens, "requests": requests, "room": room,
                "decay": rng.choice([1.0, 0.9, 0.5, 0.0]), "mix": mix}
    budget = log_int(rng, 1, hi)
    first = rng.choice([0, 0, rng.randint(0, budget // 4)])
    return {"op": op, "lens": lens, "requests": requests, "room": room, "budget": budget, "first": first,
            "last": rng.choice([0, rng.randint(0, budget - first), budget // 8]), "mix": mix}


def numbers(text):
    return [int(x) for x in text.split(",")]


def spread(case, what, count):
    """`count` lengths of the case's range, the same for every seed; both ends of it are among them where there are two."""
    lo, hi = (int(x) for x in case[what].split("-"))
    rng = random.Random(case["mix"])
    got = [rng.randint(lo, hi) for _ in range(count)]
    if count > 1:
        got[rng.randrange(count // 2)], got[rng.randrange(count // 2, count)] = lo, hi
    return got


def touched(case):
    """(first new block, blocks) of every request of a bounds case."""
    got = []
    for n in spread(case, "lens", case["requests"]):
        at = max(0, n - case["fresh"]) // case["page"]
        got.append((at, -(-n // case["page"])))
    return got


def row_lens(case):
    """Tokens that each query row sees: the last rows of a request see one more each."""
    return [max(0, n - case["rows"] + 1 + i) for n in spread(case, "lens", case["requests"]) for i in range(case["rows"])]


def work(case):
    op = case["op"]
    if op == "shared":
        row = 1056 if case["cache"] == "fp8" else 2048
        prefixes, members = numbers(case["prefixes"]), numbers(case["members"])
        batch = sum(members) + case["alone"]
        mine = sum(spread(case, "own", batch))
        pairs = mine + sum(p * m for p, m in zip(prefixes, members))
        return {"bytes": (sum(prefixes) + mine) * (row + 4) + batch * (2 * QO * D * 2 + QO * 4), "flops": 4 * QO * D * pairs}
    if op == "bounds":
        lens = spread(case, "lens", case["requests"])
        tokens = sum(max(0, n - at * case["page"]) for n, (at, _) in zip(lens, touched(case)))
        blocks = sum(max(0, end - at) for at, end in touched(case))
        return {"bytes": tokens * KV * D * 2 + blocks * (2 * KV * D * 2 + 4), "flops": 2 * tokens * KV * D}
    if op == "blocks":
        page, top = case["page"], case["top"]
        lens = row_lens(case)
        blocks = [-(-n // page) for n in lens]
        # a request's bounds and chosen rows are read for each of its query rows: their choices differ
        seen = sum(min(n, top * page) for n in lens)
        ahead = sum(-(-n // page) for n in spread(case, "lens", case["requests"]))
        return {"bytes": ahead * (2 * KV * D * 2 + 4) + seen * KV * D * 4 + len(lens) * (2 * QO * D * 2 + QO * 4 + KV * top * 4),
                "flops": 4 * QO * D * (sum(blocks) + seen)}
    lens, width = spread(case, "lens", case["requests"]), case["room"]
    if op == "weigh":
        row = 1056 if case["cache"] == "fp8" else 2048
        return {"bytes": sum(lens) * (row + 4) + case["requests"] * (width * 8 + 2 * QO * D * 2 + QO * 4),
                "flops": 4 * QO * D * sum(lens)}
    return {"bytes": sum(lens) * 8 + sum(lens) * 4 + case["requests"] * (width * 4 + 12), "flops": 8 * sum(lens)}


# ------------------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], dict(case)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def offsets(lens):
        got = [0]
        for n in lens:
            got.append(got[-1] + n)
        return ints(got)

    def shuffled(n, pool):
        return torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)

    def keys(*shape):
        x = normal(*shape)
        x[..., ::32] *= 6  # keys carry a few large channels, as trained models' do
        return x

    def caches(pool, kind):
        for name, x in (("k_cache", keys(pool, KV, D)), ("v_cache", normal(pool, KV, D))):
            if kind == "fp8":
                scale = x.abs().amax(-1) / 448
                c = torch.empty(pool, 528, dtype=torch.uint8, device="cuda")
                c[:, :512] = (x / scale[..., None]).to(torch.float8_e4m3fn).flatten(1).view(torch.uint8)
                c[:, 512:] = scale.view(torch.uint8)
                s[name] = c
            else:
                s[name] = x.to(torch.bfloat16).view(pool, 1, KV, D)

    if op == "shared":
        prefixes, members = numbers(case["prefixes"]), numbers(case["members"])
        batch = sum(members) + case["alone"]
        mine = spread(case, "own", batch)
        total = sum(prefixes) + sum(mine)
        pool = total + 100
        ids = shuffled(total, pool)
        caches(pool, case["cache"])
        s |= {"q": normal(batch, QO, D).to(torch.bfloat16), "prefix_indptr": offsets(prefixes),
              "prefix_indices": ids[:sum(prefixes)].contiguous(), "group_indptr": offsets(members),
              "kv_indptr": offsets(mine), "kv_indices": ids[sum(prefixes):].contiguous(),
              "longest": (max(prefixes), max(members), max(mine))}
    elif op in ("bounds", "blocks"):
        page, lens = case["page"], spread(case, "lens", case["requests"])
        used = [-(-n // page) for n in lens]
        blocks, width = sum(used) + 5, max(1, max(used))
        ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        at, col = offsets(used).long(), torch.arange(width, device="cuda")
        live = col < (at[1:] - at[:-1])[:, None]
        table = torch.where(live, ids[(at[:-1, None] + col).clamp(max=blocks - 1)], -1).to(torch.int32)
        s |= {"block_table": table, "k_cache": keys(blocks, page, KV, D).to(torch.bfloat16), "width": width}
        if op == "bounds":
            s |= {"lens": ints(lens), "first": ints([max(0, n - case["fresh"]) for n in lens]),
                  "bounds": torch.zeros(blocks, 2, KV, D, dtype=torch.bfloat16, device="cuda")}
        else:
            rows = row_lens(case)
            # what the earlier steps have left of the blocks' keys: whole blocks, and the tokens of a request's last one
            held = torch.full((blocks,), page, dtype=torch.int64, device="cuda")
            ends = torch.tensor([n - page * (u - 1) for n, u in zip(lens, used) if u], device="cuda")
            lasts = torch.tensor([sum(used[:i + 1]) - 1 for i, u in enumerate(used) if u], device="cuda")
            if lasts.numel():
                held[ids[lasts.long()].long()] = ends.long()
            inside = (torch.arange(page, device="cuda") < held[:, None])[..., None, None]
            hi = s["k_cache"].masked_fill(~inside, -math.inf).amax(1)
            lo = s["k_cache"].masked_fill(~inside, math.inf).amin(1)
            s |= {"q": normal(len(rows), QO, D).to(torch.bfloat16), "row_lens": ints(rows),
                  "v_cache": normal(blocks, page, KV, D).to(torch.bfloat16),
                  "token_to_req": ints([r for r in range(case["requests"]) for _ in range(case["rows"])]),
                  "bounds": torch.stack([hi, lo], 1)}
    else:
        lens, width = spread(case, "lens", case["requests"]), case["room"]
        total = sum(lens)
        # accumulated weights: a few tokens hold most; the newest have none yet
        weights = torch.exp(normal(len(lens), width, std=2.0))
        place = torch.arange(width, device="cuda")
        weights *= place < ints(lens)[:, None] - 3
        s |= {"weights": weights, "kv_indptr": offsets(lens), "kv_indices": shuffled(total, total + 100)}
        if op == "weigh":
            caches(total + 100, case["cache"])
            s |= {"q": normal(len(lens), QO, D).to(torch.bfloat16), "longest": max(1, max(lens))}
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def rows_of(cache, pages):
    """fp32 rows [..., 4, 128] of a cache's pages."""
    if cache.dtype == torch.uint8:
        rows = cache[pages]
        codes = rows[..., :512].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (KV, D))
        return codes * rows[..., 512:].contiguous().view(torch.float32)[..., None]
    return cache.view(-1, KV, D)[pages].float()


def padded(indptr, width):
    """(positions [n, width] in a CSR list, whether there is one)."""
    at = indptr.long()
    col = torch.arange(width, device="cuda")
    live = col < (at[1:] - at[:-1])[:, None]
    return (at[:-1, None] + col).clamp(max=max(1, int(width) * (indptr.numel() - 1)) - 1).where(live, 0), live


def listed_rows(cache, indices, position):
    if indices.numel() == 0:
        return torch.zeros(*position.shape, KV, D, device="cuda")
    return rows_of(cache, indices.long()[position])


def softmax_parts(score):
    """exp(score - top), its sum and log2 of the sum of exp(score), over the last axis; -inf where it has no term."""
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)) * (1.0 / math.log(2.0))
    return p, total, lse.masked_fill(total == 0, -math.inf)


def own_scores(q, k, live):
    """[b, 4, 8, t] scores of q [b, 32, 128] against k [b, t, 4, 128]."""
    score = torch.matmul(q.unflatten(1, (KV, GROUP)), k.permute(0, 2, 3, 1)) * SCALE
    return score.masked_fill(~live[:, None, None], -math.inf)


def plain_shared(s):
    longest, most, longest_own = s["longest"]
    batch, groups = s["q"].shape[0], s["group_indptr"].numel() - 1
    q = s["q"].float()
    where, live = padded(s["prefix_indptr"], longest)
    kp = listed_rows(s["k_cache"], s["prefix_indices"], where).permute(0, 2, 3, 1)        # [G, 4, 128, P]
    vp = listed_rows(s["v_cache"], s["prefix_indices"], where).transpose(1, 2)            # [G, 4, P, 128]
    member, real = padded(s["group_indptr"], most)                                        # [G, m]
    qg = q[member.clamp(max=batch - 1)].unflatten(2, (KV, GROUP)).permute(0, 2, 1, 3, 4)  # [G, 4, m, 8, 128]
    score = torch.matmul(qg.flatten(2, 3), kp) * SCALE
    score = score.masked_fill(~live[:, None, None], -math.inf).unflatten(2, (most, GROUP))
    # a sequence's group, or none
    b = torch.arange(batch, device="cuda")
    group = torch.searchsorted(s["group_indptr"].long(), b, right=True) - 1
    within = (b - s["group_indptr"].long()[group.clamp(min=0)]).clamp(0, max(most - 1, 0))
    free = (group < 0) | (group >= groups)
    group = group.clamp(0, groups - 1)
    prefix = score[group, :, within].masked_fill(free[:, None, None, None], -math.inf)    # [b, 4, 8, P]
    where, live = padded(s["kv_indptr"], longest_own)
    k, v = (listed_rows(s[x], s["kv_indices"], where) for x in ("k_cache", "v_cache"))
    p, total, lse = softmax_parts(torch.cat([prefix, own_scores(q, k, live)], -1))
    at_prefix = torch.zeros(groups, KV, most, GROUP, longest, device="cuda")
    keep = ~free
    at_prefix[group[keep], :, within[keep]] = p[keep][..., :longest]
    out = torch.matmul(p[..., longest:], v.transpose(1, 2))
    shared = torch.matmul(at_prefix.flatten(2, 3), vp).unflatten(2, (most, GROUP))        # [G, 4, m, 8, 128]
    out = (out + shared[group, :, within] * keep[:, None, None, None]) / total.clamp(min=1e-30)
    return out.flatten(1, 2).bfloat16(), lse.flatten(1)


def plain_bounds(s):
    page = s["page"]
    n, first = s["lens"].long()[:, None], s["first"].long()[:, None]
    block = torch.arange(s["width"], device="cuda")
    fresh = (block >= first // page) & (block * page < n)
    ids = s["block_table"].long()[fresh]
    left = (n - block * page)[fresh]                                                      # tokens of each block
    inside = (torch.arange(page, device="cuda") < left[:, None])[..., None, None]
    k = s["k_cache"][ids]
    hi, lo = k.masked_fill(~inside, -math.inf).amax(1), k.masked_fill(~inside, math.inf).amin(1)
    s["bounds"][ids] = torch.stack([hi, lo], 1)
    return s["bounds"]


def plain_blocks(s):
    page, top = s["page"], s["top"]
    rows, n = s["q"].shape[0], s["row_lens"].long()
    table = s["block_table"].long()[s["token_to_req"].long()]                             # [rows, width]
    block = torch.arange(s["width"], device="cuda")
    count = (n + page - 1) // page
    live = block < count[:, None]
    bounds = s["bounds"][table.clamp(min=0)].double()                                     # [rows, width, 2, 4, 128]
    q = s["q"].double().unflatten(1, (KV, GROUP))
    hi, lo = (bounds[:, :, i].permute(0, 2, 3, 1) for i in (0, 1))                        # [rows, 4, 128, width]
    score = (torch.matmul(q.clamp(min=0), hi) + torch.matmul(q.clamp(max=0), lo)).amax(2)  # [rows, 4, width]
    forced = (block < s["first"]) | (block >= count[:, None] - s["last"])
    score = score.masked_fill(forced[:, None], math.inf).masked_fill(~live[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.where(order < count[:, None, None], order, s["width"]).sort(-1).values
    blocks = torch.full((rows, KV, top), -1, dtype=torch.int32, device="cuda")
    blocks[..., :order.shape[-1]] = torch.where(order < s["width"], order, -1).int()
    t = (blocks.long()[..., None] * page + torch.arange(page, device="cuda")).flatten(2)  # [rows, 4, top * page]
    seen = (t >= 0) & (t < n[:, None, None]) & (blocks >= 0).repeat_interleave(page, -1)
    t = t.where(seen, 0)
    slot = table.gather(1, (t // page).flatten(1)).view_as(t).clamp(min=0) * page + t % page
    head = torch.arange(KV, device="cuda")[:, None]
    k, v = (s[x].view(-1, KV, D)[slot, head].float() for x in ("k_cache", "v_cache"))     # [rows, 4, t, 128]
    score = torch.matmul(s["q"].float().unflatten(1, (KV, GROUP)), k.transpose(2, 3)) * SCALE
    p, total, lse = softmax_parts(score.masked_fill(~seen[:, :, None], -math.inf))
    out = torch.matmul(p, v) / total.clamp(min=1e-30)
    return {"blocks": blocks, "out": out.flatten(1, 2).bfloat16(), "lse": lse.flatten(1)}


def plain_weigh(s):
    where, live = padded(s["kv_indptr"], s["longest"])
    q = s["q"].float()
    score = own_scores(q, listed_rows(s["k_cache"], s["kv_indices"], where), live)
    p, total, lse = softmax_parts(score)
    p = p / total.clamp(min=1e-30)
    out = torch.matmul(p, listed_rows(s["v_cache"], s["kv_indices"], where).transpose(1, 2))
    got = s["weights"].clone()
    got[:, :s["longest"]] = torch.where(live, got[:, :s["longest"]] * s["decay"] + p.sum((1, 2)), got[:, :s["longest"]])
    return {"out": out.flatten(1, 2).bfloat16(), "lse": lse.flatten(1), "weights": got}


def plain_evict(s):
    at = s["kv_indptr"].long()
    n, place = at[1:] - at[:-1], torch.arange(s["room"], device="cuda")
    live = place < n[:, None]
    fixed = (place < s["first"]) | (place >= n[:, None] - s["last"])
    rank = s["weights"].masked_fill(fixed, math.inf).masked_fill(~live, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(live).scatter_(1, order, place.expand_as(order) < s["budget"]) & live
    listed = torch.nonzero(live)                                                          # in the list's order
    kept = keep[listed[:, 0], listed[:, 1]]
    total = s["kv_indices"].numel()
    indices, freed = (torch.full((total,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    mine, gone = s["kv_indices"][kept], s["kv_indices"][~kept]
    indices[:mine.numel()], freed[:gone.numel()] = mine, gone
    left = keep.sum(1)
    weights = torch.zeros_like(s["weights"])
    weights[place < left[:, None]] = s["weights"][keep]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return {"weights": weights, "kv_indptr": torch.cat([zero, left.cumsum(0)]).int(), "kv_indices": indices,
            "freed_indptr": torch.cat([zero, (n - left).cumsum(0)]).int(), "freed": freed}


def run(s):
    op = s["op"]
    if own:
        import paged_kv_gqa_split_gb300 as pkg
        if op == "shared":
            return pkg.shared_run(s["q"], s["k_cache"], s["v_cache"], s["prefix_indptr"], s["prefix_indices"],
                                  s["group_indptr"], s["kv_indptr"], s["kv_indices"])
        if op == "bounds":
            return pkg.block_bounds(s["k_cache"], s["bounds"], s["block_table"], s["lens"], s["first"])
        if op == "blocks":
            blocks = pkg.block_select(s["q"], s["bounds"], s["block_table"], s["token_to_req"], s["row_lens"], s["top"],
                                      s["page"], keep_first=s["first"], keep_last=s["last"])
            out, lse = pkg.block_sparse_run(s["q"], s["k_cache"], s["v_cache"], blocks, s["block_table"],
                                            s["token_to_req"], s["row_lens"])
            return {"blocks": blocks, "out": out, "lse": lse}
        if op == "weigh":
            out, lse, weights = pkg.run_weighted(s["q"], s["k_cache"], s["v_cache"], s["kv_indptr"], s["kv_indices"],
                                                 s["weights"], decay=s["decay"])
            return {"out": out, "lse": lse, "weights": weights}
        weights, indptr, indices, freed_indptr, freed = pkg.kv_evict(
            s["weights"], s["kv_indptr"], s["kv_indices"], s["budget"], keep_first=s["first"], keep_last=s["last"])
        return {"weights": weights, "kv_indptr": indptr, "kv_indices": indices, "freed_indptr": freed_indptr,
                "freed": freed}
    if op == "shared":
        return plain_shared(s)
    if op == "bounds":
        return plain_bounds(s)
    if op == "blocks":
        return plain_blocks(s)
    return plain_weigh(s) if op == "weigh" else plain_evict(s)


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def values64(cache, pages):
    rows = cache.index_select(0, pages)
    if cache.dtype == torch.uint8:
        vals = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double().unflatten(1, (KV, D))
        return vals * rows[:, 512:].contiguous().view(torch.float32).double().unsqueeze(-1)
    return rows.double().view(-1, KV, D)


def attend64(q, k, v):
    """(out [32, 128], lse [32] in base 2, probabilities [4, 8, t]) of one query over rows [t, 4, 128]."""
    if k.shape[0] == 0:
        return q.new_zeros(QO, D).double(), torch.full((QO,), -math.inf, dtype=torch.float64, device="cuda"), None
    z = torch.einsum("ghd,tgd->ght", q.double().view(KV, GROUP, D), k) / math.sqrt(D)
    p = torch.softmax(z, -1)
    return torch.einsum("ght,tgd->ghd", p, v).view(QO, D), torch.logsumexp(z, -1).view(QO) / math.log(2), p


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "shared":
        where, parts = [int(x) for x in s["group_indptr"]], [int(x) for x in s["prefix_indptr"]]
        at, outs, lses = [int(x) for x in s["kv_indptr"]], [], []
        for b in range(s["q"].shape[0]):
            pages = s["kv_indices"][at[b]:at[b + 1]]
            for i in range(len(parts) - 1):
                if where[i] <= b < where[i + 1]:
                    pages = torch.cat([s["prefix_indices"][parts[i]:parts[i + 1]], pages])
            out, lse, _ = attend64(s["q"][b], values64(s["k_cache"], pages), values64(s["v_cache"], pages))
            outs.append(out)
            lses.append(lse)
        return torch.stack(outs), torch.stack(lses)
    if op == "bounds":
        got = torch.zeros(s["bounds"].shape, dtype=torch.float64, device="cuda")
        for r, (n, (at, end)) in enumerate(zip(spread(case, "lens", case["requests"]), touched(case))):
            full = min(end, n // case["page"])
            if full > at:
                ids = s["block_table"][r, at:full].long()
                k = s["k_cache"][ids].double()
                got[ids, 0], got[ids, 1] = k.max(1).values, k.min(1).values
            for i in range(max(at, full), end):
                id_ = int(s["block_table"][r, i])
                k = s["k_cache"][id_, :n - i * case["page"]].double()
                got[id_, 0], got[id_, 1] = k.max(0).values, k.min(0).values
        return got
    if op == "blocks":
        page, top, lens = case["page"], case["top"], row_lens(case)
        picked = torch.full((len(lens), KV, top), -1, dtype=torch.int32, device="cuda")
        outs, lses = [], []
        for r, n in enumerate(lens):
            count, req = -(-n // page), r // case["rows"]
            ids = s["block_table"][req, :count].long()
            hi, lo = s["bounds"][ids, 0].double(), s["bounds"][ids, 1].double()           # [count, 4, 128]
            q = s["q"][r].double().view(KV, 1, GROUP, D)
            for g in range(KV):
                bound = torch.maximum(q[g] * hi[:, g, None], q[g] * lo[:, g, None]).sum(-1).amax(-1)
                bound[:case["first"]] = math.inf
                bound[max(0, count - case["last"]):] = math.inf
                best = torch.sort(-bound, stable=True).indices[:top].sort().values
                picked[r, g, :best.numel()] = best.int()
                t = (best[:, None] * page + torch.arange(page, device="cuda")).flatten()
                t = t[t < n]
                slot = ids[t // page] * page + t % page if n else t
                k, v = (s[x].view(-1, KV, D)[slot][:, g].double() for x in ("k_cache", "v_cache"))
                z = s["q"][r, g * GROUP:(g + 1) * GROUP].double() @ k.t() / math.sqrt(D)
                outs.append(torch.softmax(z, -1) @ v if n else torch.zeros(GROUP, D, dtype=torch.float64, device="cuda"))
                lses.append(torch.logsumexp(z, -1) / math.log(2))
        shape = (len(lens), QO)
        return {"blocks": picked, "out": torch.stack(outs).view(*shape, D), "lse": torch.stack(lses).view(shape)}
    lens, at = spread(case, "lens", case["requests"]), [int(x) for x in s["kv_indptr"]]
    if op == "weigh":
        weights, outs, lses = s["weights"].double(), [], []
        for b, n in enumerate(lens):
            pages = s["kv_indices"][at[b]:at[b + 1]]
            out, lse, p = attend64(s["q"][b], values64(s["k_cache"], pages), values64(s["v_cache"], pages))
            if n:
                weights[b, :n] = weights[b, :n] * case["decay"] + p.sum((0, 1))
            outs.append(out)
            lses.append(lse)
        return {"out": torch.stack(outs), "lse": torch.stack(lses), "weights": weights}
    weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    stay, go = [], []
    for b, n in enumerate(lens):
        w = s["weights"][b, :n].double()
        rank = w.clone()
        rank[:case["first"]] = math.inf
        rank[max(0, n - case["last"]):] = math.inf
        keep = torch.sort(-rank, stable=True).indices[:case["budget"]].sort().values
        drop = torch.ones(n, dtype=torch.bool, device="cuda")
        drop[keep] = False
        weights[b, :keep.numel()] = w[keep]
        pages = s["kv_indices"][at[b]:at[b + 1]]
        stay.append(pages[keep])
        go.append(pages[drop])
    got = {"weights": weights}
    for names, lists in ((("kv_indptr", "kv_indices"), stay), (("freed_indptr", "freed"), go)):
        ends = [0]
        for x in lists:
            ends.append(ends[-1] + x.numel())
        flat = torch.full((at[-1],), -1, dtype=torch.int32, device="cuda")
        flat[:ends[-1]] = torch.cat(lists)
        got |= {names[0]: torch.tensor(ends, dtype=torch.int32, device="cuda"), names[1]: flat}
    return got
