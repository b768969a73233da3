"""The operators of the 4-bit history cache: their plain forms, their calls and the sizes they are measured at.

A serving step with cached user histories makes four calls, and each case is one pass through one of them:
  tables  rocs_kv_block_tables: pages, slots and positions of the step's new history events, from the requests' lengths
  rope    rocs_qk_norm_rope: RMS norm of every query and key head, and the position rotation, in one pass
  store   rocs_kv4_append and rocs_kv4_gather: keys and values to 4 bits in their slots, and back from their slots
  attn    rocs_dca_cross_attn_kv4: grouped attention of query rows against their request's cached keys and values
"""
import numpy as np
import torch

own = False

GROUP = 32              # cache elements that share one scale
TINY, HUGE = 2.0 ** -120, 2.0 ** 120   # the range of a scale


# ---- sizes ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new event for each of 512 requests, the batch of the end-to-end workload; a captured step pads its rows
        dict(name="tables step", op="tables", requests=512, page=64, past=400, past_top=1024, new=1, new_top=1, spare=0, mix=1),
        # whole histories of 512 requests enter an empty cache
        dict(name="tables histories", op="tables", requests=512, page=64, past=0, past_top=0, new=500, new_top=1024, spare=37, mix=2),
        # an offline pass that fills a large cache: many requests, small pages
        dict(name="tables fill", op="tables", requests=40000, page=16, past=60, past_top=1500, new=110, new_top=2000, spare=1000, mix=3),
        # one new event a request: queries and keys of the end-to-end workload's heads
        dict(name="rope step", op="rope", rows=512, q_heads=8, k_heads=8, d=32, rot=32, pairs="halves", top=1025, io="bf16", spare=0, mix=4),
        # whole histories of the end-to-end workload: 512 requests of up to 1024 events
        dict(name="rope histories", op="rope", rows=524288, q_heads=8, k_heads=8, d=32, rot=32, pairs="halves", top=1024, io="bf16", spare=0, mix=5),
        # fp32 activations, shared key heads, half of each head rotated, an odd number of rows with a padded end
        dict(name="rope shared fp32", op="rope", rows=30011, q_heads=16, k_heads=2, d=128, rot=64, pairs="neighbours", top=100000, io="fp32", spare=13, mix=6),
        # the new events of 512 requests, scattered over the cache
        dict(name="store step", op="store", rows=512, heads=8, d=32, page=64, spare=0, mix=7),
        # whole histories of the end-to-end workload
        dict(name="store histories", op="store", rows=262147, heads=8, d=32, page=64, spare=61, mix=8),
        # every request's own query against its history: one row a request
        dict(name="attn request query", op="attn", requests=512, page=64, heads=8, share=1, d=32, kv=500, kv_top=1024, q=1, q_top=1, causal=False, mix=9),
        # candidates against their request's history, the grouped attention of the ranking forward
        dict(name="attn candidates", op="attn", requests=96, page=64, heads=8, share=1, d=32, kv=1000, kv_top=1024, q=400, q_top=2000, causal=False, mix=10),
        # a burst of new events that see the cached history and one another, up to themselves
        dict(name="attn new events", op="attn", requests=48, page=16, heads=4, share=2, d=64, kv=1500, kv_top=4000, q=130, q_top=500, causal=True, mix=11),
        # lifelong histories, one query each, key heads shared by four query heads
        dict(name="attn lifelong", op="attn", requests=3, page=128, heads=8, share=4, d=128, kv=90001, kv_top=131071, q=1, q_top=1, causal=False, mix=12),
    ]


def _between(rng, low, high):
    """A whole number from low to high, spread evenly over its logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "rope", "store", "attn"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        requests = _between(rng, 1, 40000)
        new_top = 1 if rng.random() < 0.3 else _between(rng, 1, max(1, min(20000, 6000000 // requests)))
        past_top = rng.choice([0, _between(rng, 1, max(1, min(20000, 6000000 // requests)))])
        return dict(op=op, requests=requests, page=page, past=past_top // 2, past_top=past_top, new=max(1, new_top // 2), new_top=new_top,
                    spare=rng.choice([0, 1, 17, 300]), mix=mix)
    d = rng.choice([32, 64, 128])
    if op == "rope":
        d = rng.choice([16, 32, 64, 80, 96, 128, 192, 256])
        q_heads, k_heads = rng.choice([(1, 1), (4, 4), (8, 8), (8, 2), (12, 3), (32, 4), (7, 1), (16, 0), (0, 8)])
        io = rng.choice(["bf16", "fp32"])
        rows = _between(rng, 1, max(1, (200000000 if io == "bf16" else 100000000) // ((q_heads + k_heads) * d)))
        return dict(op=op, rows=rows, q_heads=q_heads, k_heads=k_heads, d=d, rot=rng.choice([d, 16 * rng.randint(1, d // 16)]),
                    pairs=rng.choice(["halves", "neighbours"]), top=_between(rng, 10, 100000), io=io, spare=rng.choice([0, 1, 5]) if rows > 8 else 0, mix=mix)
    if op == "store":
        heads = rng.choice([1, 2, 4, 5, 8, 16])
        rows = _between(rng, 1, max(1, 66000000 // (heads * d)))
        return dict(op=op, rows=rows, heads=heads, d=d, page=page, spare=rng.choice([0, 1, 7]) if rows > 16 else 0, mix=mix)
    heads, share = rng.choice([(1, 1), (2, 1), (4, 1), (8, 1), (8, 2), (2, 4), (4, 4), (1, 8), (3, 1)])
    kind = rng.choice(["one", "few", "many", "causal"])
    kv_top = _between(rng, 1, 100000 if kind == "one" else 4000)
    requests = _between(rng, 1, max(1, min(600, 60000000 // (kv_top * heads * d))))
    most = max(1, min(2000, 300000000 // (requests * kv_top * heads * share), 100000000 // (requests * heads * share * d)))
    if kind == "causal":      # the cache holds the new events too
        most = max(1, min(most, int((300000000 // (requests * heads * share)) ** 0.5)))
    q_top = 1 if kind == "one" else _between(rng, 1, min(40, most)) if kind == "few" else _between(rng, 1, most)
    return dict(op=op, requests=requests, page=page, heads=heads, share=share, d=d, kv=max(1, kv_top // 2), kv_top=kv_top, q=max(1, q_top // 2), q_top=q_top,
                causal=kind == "causal", mix=mix)


def _ceil(n, page):
    """The pages that n tokens take."""
    return (n + page - 1) // page


def _lengths(n, mean, top, rng, least=0):
    """n ragged lengths around `mean`, `top` at most: log-normal, as the workloads draw candidate counts."""
    if top <= least:
        return np.full(n, top, np.int64)
    return np.clip(np.round(np.exp(rng.normal(np.log(max(mean, 1)), 1.0, n))), least, top).astype(np.int64)


def _shape(case):
    """What the case's `mix` fixes of its inputs: the lengths, which the work follows from."""
    rng = np.random.default_rng(case["mix"])
    s = dict(case)
    if case["op"] == "tables":
        s["past"] = _lengths(case["requests"], case["past"], case["past_top"], rng)
        s["new"] = _lengths(case["requests"], case["new"], case["new_top"], rng, 0 if case["new_top"] > 1 else 1)
        s["blocks"] = max(1, int(_ceil(s["past"] + s["new"], case["page"]).max()))
        s["need"] = int((_ceil(s["past"] + s["new"], case["page"]) - _ceil(s["past"], case["page"])).sum())
        s["held"] = int(_ceil(s["past"], case["page"]).sum())
        s["rows"] = max(1, int(s["new"].sum()) + case["spare"])
    if case["op"] == "attn":
        s["q"] = _lengths(case["requests"], case["q"], case["q_top"], rng, 0 if case["q_top"] > 1 else 1)
        s["kv"] = _lengths(case["requests"], case["kv"], case["kv_top"], rng, 0)
        if case["causal"]:
            s["kv"] = np.maximum(s["kv"], s["q"])     # the new events are cached before they attend
        s["blocks"] = max(1, int(_ceil(s["kv"], case["page"]).max()))
        s["held"] = int(_ceil(s["kv"], case["page"]).sum())
        s["rows"] = int(s["q"].sum())
        if s["rows"] == 0:
            s["q"][0], s["rows"] = 1, 1
            s["kv"][0] = max(s["kv"][0], 1)
            s["held"] = int(_ceil(s["kv"], case["page"]).sum())
            s["blocks"] = max(1, int(_ceil(s["kv"], case["page"]).max()))
    return s


def work(case):
    s = _shape(case)
    if s["op"] == "tables":
        # lengths, the pages taken and their table entries, a partial page's entry, and each row's slot (8 bytes) and position (4)
        return dict(bytes=4 * (4 * s["requests"] + 2 * s["need"]) + 12 * s["rows"] + 8, flops=4 * s["rows"])
    if s["op"] == "rope":
        size = 2 if s["io"] == "bf16" else 4
        n = (s["rows"] - s["spare"]) * (s["q_heads"] + s["k_heads"]) * s["d"]
        table = min(s["top"], s["rows"] - s["spare"]) * s["rot"] * 4
        return dict(bytes=2 * size * n + table + 4 * s["rows"] + 4 * s["d"] * ((s["q_heads"] > 0) + (s["k_heads"] > 0)), flops=7 * n)
    if s["op"] == "store":
        n = (s["rows"] - s["spare"]) * s["heads"] * s["d"]        # of keys, and of values
        return dict(bytes=2 * (4 * n + 2 * n * 9 // 16) + 16 * s["rows"], flops=2 * 6 * n)
    seen = s["kv"] * s["q"] if not s["causal"] else s["kv"] * s["q"] - s["q"] * (s["q"] - 1) // 2
    heads = s["heads"] * s["share"]
    read = int(s["kv"][s["q"] > 0].sum()) * s["heads"] * s["d"] * 9 // 8
    return dict(bytes=read + 4 * s["rows"] * heads * s["d"] + 4 * (2 * s["requests"] + s["held"]), flops=4 * s["d"] * heads * int(seen.sum()))


# ---- inputs -----------------------------------------------------------------------------------------------------

def _quantize(x):
    """[..., d] to whole numbers in [-7, 7] and [..., d / 32] scales: the smallest number of four significant bits that is no less than
    a 7th of the group's largest magnitude, so that number times scale is a bf16 value; halves away from zero."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    seventh = top / torch.full_like(top, 7)     # a true division: by a plain 7 it would be a product with the rounded reciprocal
    scale = ((seventh.view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(torch.float32).clamp(TINY, HUGE)
    q = torch.floor(g.abs() / scale[..., None] + 0.5).clamp(max=7) * g.sign()
    return q.flatten(-2), scale


def _records(k, v):
    """Keys and values [pages, page, heads, d] as the cache holds them: for each page and head, the keys' codes (d / 2 bytes a token, the
    lower nibble first, 8 standing for 0), their scales (bf16), the values' codes, their scales."""
    parts = []
    for x in (k, v):
        q, scale = _quantize(x.transpose(1, 2))
        n = (q + 8).to(torch.uint8)
        parts += [(n[..., 0::2] | (n[..., 1::2] << 4)).flatten(2), scale.to(torch.bfloat16).flatten(2).view(torch.uint8)]
    return torch.cat(parts, 2).contiguous()


def _values(records, page, d):
    """The keys and values [..., page, d], in 32 bits, that records [..., page * d * 9 / 8] hold."""
    half = []
    for r in records.unflatten(-1, (2, -1)).unbind(-2):
        codes = r[..., : page * d // 2].unflatten(-1, (page, d // 2))
        scale = r[..., page * d // 2:].contiguous().view(torch.bfloat16).unflatten(-1, (page, d // GROUP)).float()
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
        half.append((q.unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2))
    return half


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float32).to(dtype)


def _activations(gen, *shape):
    """Keys or values as projections give them: some channels are much larger than others."""
    x = torch.randn(*shape, device="cuda", generator=gen)
    return (x * torch.exp(0.7 * torch.randn(*shape[1:], device="cuda", generator=gen))).to(torch.bfloat16)


def prepare(case, seed):
    s = _shape(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) + 1000003 * (s["mix"] % 1000003))
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    shuffled = lambda n: torch.randperm(n, device="cuda", generator=gen).to(torch.int32)  # noqa: E731
    if s["op"] == "tables":
        pages = s["held"] + s["need"] + 64
        order = shuffled(pages)
        table = torch.full((s["requests"], s["blocks"]), -1, dtype=torch.int32, device="cuda")
        has = torch.arange(s["blocks"], device="cuda") < i32(_ceil(s["past"], s["page"]))[:, None]
        table[has] = order[: s["held"]]
        rows = s["rows"]
        return dict(s, past_len=i32(s["past"]), new_len=i32(s["new"]), free=order[s["held"]:].contiguous(), pages=pages, table=table,
                    kv_len=torch.empty(s["requests"], dtype=torch.int32, device="cuda"), offsets=torch.empty(s["requests"] + 1, dtype=torch.int32, device="cuda"),
                    slots=torch.empty(rows, dtype=torch.int64, device="cuda"), positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                    taken=torch.empty(1, dtype=torch.int32, device="cuda"))
    if s["op"] == "rope":
        dtype = torch.bfloat16 if s["io"] == "bf16" else torch.float32
        rows, d, nq, nk = s["rows"], s["d"], s["q_heads"], s["k_heads"]
        # queries, keys and values lie side by side, as one projection writes them
        qkv = _normal(gen, rows, (nq + 2 * nk) * d, dtype=dtype)
        at = torch.randint(0, s["top"], (rows,), device="cuda", generator=gen, dtype=torch.int32)
        at[rows - s["spare"]:] = -1          # a padded batch's rows have no position
        angle = torch.arange(s["top"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, s["rot"], 2, device="cuda", dtype=torch.float64) / s["rot"])
        gamma = [torch.rand(d, device="cuda", generator=gen) + 0.5 for _ in range(2)]
        return dict(s, qkv=qkv, positions=at, table=torch.cat((angle.cos(), angle.sin()), 1).float().contiguous(), gamma_q=gamma[0], gamma_k=gamma[1],
                    q_out=torch.zeros(rows, nq * d, device="cuda", dtype=dtype), k_out=torch.zeros(rows, nk * d, device="cuda", dtype=dtype))
    if s["op"] == "store":
        rows, h, d, page = s["rows"], s["heads"], s["d"], s["page"]
        pages = _ceil(rows, page) + 3
        # runs of consecutive slots, as histories fill their pages, in pages that lie anywhere
        at = torch.arange(rows, device="cuda") + 5
        slots = shuffled(pages).long()[at // page] * page + at % page
        slots[rows - s["spare"]:] = -1
        return dict(s, k=_activations(gen, rows, h, d), v=_activations(gen, rows, h, d), slots=slots, pages=pages,
                    cache=torch.zeros(pages, h, page * d * 9 // 8, dtype=torch.uint8, device="cuda"),
                    k_back=torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda"), v_back=torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda"))
    h, d, page = s["heads"], s["d"], s["page"]
    pages = max(1, s["held"]) + 5
    cache = _records(_normal(gen, pages, page, h, d), _normal(gen, pages, page, h, d))
    order = shuffled(pages)
    table = torch.full((s["requests"], s["blocks"]), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(s["blocks"], device="cuda") < i32(_ceil(s["kv"], page))[:, None]] = order[: s["held"]]
    q = _normal(gen, s["rows"], h * s["share"] * d)
    return dict(s, cache=cache, pages=pages, table=table, kv_len=i32(s["kv"]), offsets=i32(np.concatenate(([0], np.cumsum(s["q"])))), q_rows=q, most=int(s["q"].max()),
                out=torch.zeros_like(q))


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _plain_tables(s):
    past, new, page = s["past_len"].long(), s["new_len"].long(), s["page"]
    total = past + new
    before, after = (past + page - 1) // page, (total + page - 1) // page
    ends, starts = new.cumsum(0), (after - before).cumsum(0) - (after - before)
    blocks = torch.arange(s["table"].shape[1], device=past.device)
    fresh = (blocks >= before[:, None]) & (blocks < after[:, None])
    at = (starts[:, None] + blocks - before[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    row = torch.arange(s["rows"], device=past.device)
    r = torch.searchsorted(ends, row, right=True)
    real = r < past.numel()
    r = r.clamp(max=past.numel() - 1)
    position = past[r] + row - (ends[r] - new[r])
    slots = table[r, (position // page).clamp(0, table.shape[1] - 1)].long() * page + position % page
    offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
    return [table, total.int(), offsets.int(), torch.where(real, slots, -1), torch.where(real, position, -1).int(), (after - before).sum().int().reshape(1)]


def _plain_rope(s):
    nq, nk, d, rot = s["q_heads"], s["k_heads"], s["d"], s["rot"]
    rows, at = s["rows"], s["positions"].long()
    cos, sin = s["table"][at.clamp(min=0)][:, None].chunk(2, -1)
    out = []
    for x, gamma, was in ((s["qkv"][:, : nq * d], s["gamma_q"], s["q_out"]), (s["qkv"][:, nq * d: (nq + nk) * d], s["gamma_k"], s["k_out"])):
        x = x.reshape(rows, -1, d).float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma
        a, b = (x[..., : rot // 2], x[..., rot // 2: rot]) if s["pairs"] == "halves" else (x[..., 0:rot:2], x[..., 1:rot:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat((a, b), -1) if s["pairs"] == "halves" else torch.stack((a, b), -1).flatten(-2)
        x = torch.cat((turned, x[..., rot:]), -1).reshape(rows, -1).to(s["qkv"].dtype)
        out.append(torch.where((at >= 0)[:, None], x, was))
    return out


def _plain_store(s):
    page, d, slots = s["page"], s["d"], s["slots"]
    real = slots >= 0
    out = []
    # the cache as [pages, heads, page, ...] views: one index for all of a row's heads
    views = []
    for r in s["cache"].unflatten(-1, (2, -1)).unbind(-2):
        views.append((r[..., : page * d // 2].unflatten(-1, (page, d // 2)), r[..., page * d // 2:].unflatten(-1, (page, d // 16))))
    p, o = slots[real] // page, slots[real] % page
    for x, (codes, scales) in zip((s["k"], s["v"]), views):
        q, scale = _quantize(x[real])
        n = (q + 8).to(torch.uint8)
        codes[p, :, o] = n[..., 0::2] | (n[..., 1::2] << 4)
        scales[p, :, o] = scale.to(torch.bfloat16).view(torch.uint8)
    for was, (codes, scales) in zip((s["k_back"], s["v_back"]), views):
        c, scale = codes[p, :, o], scales[p, :, o].contiguous().view(torch.bfloat16).float()
        q = torch.stack((c & 15, c >> 4), -1).flatten(-2).float() - 8
        back = was.clone()
        back[real] = (q.unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2).to(torch.bfloat16)
        out.append(back)
    return out


def _plain_attn(s):
    h, g, d, page, b, most = s["heads"], s["share"], s["d"], s["page"], s["requests"], s["most"]
    k, v = _values(s["cache"][s["table"].long().clamp(min=0)], page, d)          # [b, blocks, h, page, d]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))                     # [b, h, tokens, d]
    start, count = s["offsets"][:-1].long(), s["offsets"][1:].long() - s["offsets"][:-1].long()
    i = torch.arange(most, device=k.device)
    row = (start[:, None] + i).clamp(max=s["rows"] - 1)                          # [b, most]
    q = s["q_rows"].view(s["rows"], h, g, d)[row].permute(0, 2, 1, 3, 4).flatten(2, 3).float()   # [b, h, most * g, d]
    token = torch.arange(k.shape[2], device=k.device)
    last = s["kv_len"].long()[:, None] - (count[:, None] - i if s["causal"] else 1) + (0 if s["causal"] else 0 * i)
    seen = (token <= last[..., None]) & (token < s["kv_len"][:, None, None])      # [b, most, tokens]
    seen = seen[:, None, :, None].expand(-1, -1, -1, g, -1).flatten(2, 3)
    score = (q @ k.transpose(-1, -2)) * d ** -0.5
    score = torch.where(seen, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
    total = weight.sum(-1, keepdim=True)
    o = (weight @ v) / torch.where(total > 0, total, 1.0)                         # a row that sees nothing is zero
    o = o.unflatten(2, (most, g)).permute(0, 2, 1, 3, 4).flatten(2)               # [b, most, h * g * d]
    return o[i < count[:, None]].to(torch.bfloat16)


# ---- the framework's calls ------------------------------------------------------------------------------------------

_handle = None


def _rocs():
    global _handle
    from request_candidate_sharing_b200 import rocs
    if _handle is None:
        _handle = rocs.Rocs(torch.cuda.current_device())
    return rocs, _handle


def _own_tables(s):
    _, h = _rocs()
    size = h.rocs_kv_block_tables_workspace(s["requests"])
    scratch = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    h.rocs_kv_block_tables(s["past_len"], s["new_len"], s["requests"], s["page"], s["free"], s["free"].numel(), s["pages"], s["table"], s["blocks"],
                           s["kv_len"], s["offsets"], s["slots"], s["positions"], s["rows"], s["taken"], scratch, size, torch.cuda.current_stream().cuda_stream)
    return [s["table"], s["kv_len"], s["offsets"], s["slots"], s["positions"], s["taken"]]


def _own_rope(s):
    rocs, h = _rocs()
    nq, nk, d, qkv = s["q_heads"], s["k_heads"], s["d"], s["qkv"]
    desc = rocs.QkDesc(s["rows"], nq, nk, d, s["rot"], int(s["pairs"] == "neighbours"), s["top"], 1e-6, rocs.dtype_code(qkv))
    ld = qkv.shape[1]
    h.rocs_qk_norm_rope(desc, qkv if nq else None, ld, qkv[:, nq * d:] if nk else None, ld, s["gamma_q"], s["gamma_k"], s["table"], s["positions"],
                        s["q_out"] if nq else None, nq * d, s["k_out"] if nk else None, nk * d, torch.cuda.current_stream().cuda_stream)
    return [s["q_out"], s["k_out"]]


def _own_store(s):
    rocs, h = _rocs()
    desc = rocs.Kv4Desc(s["pages"], s["page"], s["heads"], s["d"])
    ld, stream = s["heads"] * s["d"], torch.cuda.current_stream().cuda_stream
    h.rocs_kv4_append(desc, s["k"], ld, s["v"], ld, s["slots"], s["rows"], s["cache"], stream)
    h.rocs_kv4_gather(desc, s["cache"], s["slots"], s["rows"], s["k_back"], ld, s["v_back"], ld, stream)
    return [s["k_back"], s["v_back"]]


def _own_attn(s):
    rocs, h = _rocs()
    desc = rocs.Kv4Desc(s["pages"], s["page"], s["heads"], s["d"])
    heads = s["heads"] * s["share"]
    size = h.rocs_dca_cross_attn_kv4_workspace(desc, heads, s["requests"], s["rows"], s["blocks"])
    scratch = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    ld = heads * s["d"]
    h.rocs_dca_cross_attn_kv4(desc, s["q_rows"], ld, heads, s["cache"], s["table"], s["blocks"], s["kv_len"], s["offsets"], s["requests"], s["rows"],
                              s["d"] ** -0.5, int(s["causal"]), s["out"], ld, scratch, size, torch.cuda.current_stream().cuda_stream)
    return s["out"]


def run(state):
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "store": _own_store, "attn": _own_attn}[state["op"]](state)
    return {"tables": _plain_tables, "rope": _plain_rope, "store": _plain_store, "attn": _plain_attn}[state["op"]](state)


# ---- the definitions, in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tables":
        return None                  # whole numbers
    if s["op"] == "rope":
        nq, nk, d, rot = s["q_heads"], s["k_heads"], s["d"], s["rot"]
        at = s["positions"].long()
        angle = s["table"].double()[at.clamp(min=0)]
        turn = torch.complex(angle[:, : rot // 2], angle[:, rot // 2:])[:, None]
        out = []
        for first, n, gamma in ((0, nq, s["gamma_q"]), (nq, nk, s["gamma_k"])):
            x = s["qkv"].double()[:, first * d: (first + n) * d].unflatten(1, (n, d)) if n else s["qkv"].double()[:, :0].reshape(s["rows"], 0, d)
            x = x / (x.square().sum(-1, keepdim=True) / d + 1e-6).sqrt() * gamma.double()
            i = torch.arange(rot, device=x.device)
            i = i.view(2, -1) if s["pairs"] == "halves" else i.view(-1, 2).T
            z = torch.complex(x[..., i[0]], x[..., i[1]]) * turn
            y = x.clone()
            y[..., i[0]], y[..., i[1]] = z.real, z.imag
            out.append((y * (at >= 0)[:, None, None]).flatten(1))
        return out
    if s["op"] == "store":
        out = []
        for x in (s["k"], s["v"]):
            g = x.double().unflatten(-1, (-1, GROUP))
            top = g.abs().amax(-1, keepdim=True)
            m, e = torch.frexp(top / torch.full_like(top, 7))
            scale = torch.ldexp(torch.ceil(m * 16) / 16, e).clamp(TINY, HUGE)
            y = torch.sign(g) * torch.floor(g.abs() / scale + 0.5).clamp(max=7) * scale
            out.append(y.flatten(-2) * (s["slots"] >= 0)[:, None, None])
        return out
    h, g, d, page = s["heads"], s["share"], s["d"], s["page"]
    out = torch.zeros(s["rows"], h * g * d, device="cuda", dtype=torch.float64)
    at = 0
    for r, (n, length) in enumerate(zip(s["q"].tolist(), s["kv"].tolist())):
        if n and length:
            rec = s["cache"][s["table"][r, : _ceil(length, page)].long()].permute(1, 0, 2)      # [heads, blocks, record]
            kv = []
            for half in (rec[..., : rec.shape[-1] // 2], rec[..., rec.shape[-1] // 2:]):
                c = half[..., : page * d // 2].reshape(h, -1, d // 2).int()
                scale = half[..., page * d // 2:].contiguous().view(torch.bfloat16).reshape(h, -1, d // GROUP).double()
                x = torch.empty(h, c.shape[1], d, device="cuda", dtype=torch.float64)
                x[..., 0::2], x[..., 1::2] = (c % 16) - 8, (c // 16) - 8
                kv.append((x * scale.repeat_interleave(GROUP, -1))[:, :length])
            q = s["q_rows"][at: at + n].double().view(n, h, g, d)
            score = torch.einsum("nhgd,htd->hgnt", q, kv[0]) / d ** 0.5
            if s["causal"]:
                hidden = torch.arange(length, device="cuda") > (length - n + torch.arange(n, device="cuda"))[:, None]
                score.masked_fill_(hidden, float("-inf"))
            out[at: at + n] = torch.einsum("hgnt,htd->nhgd", torch.softmax(score, -1), kv[1]).reshape(n, -1)
        at += n
    return out
