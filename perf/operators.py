"""Cases of the history-cache and sampling operators: a user's event history held in 8 bits and read by attention,
and the draw of items from their scores.

Four operators, in the order in which a serving step runs them:
  plan       block tables and slot maps from request lengths        hist_plan
  append     new keys and values into the 8-bit cache, read back    hist_append, hist_read
  attention  queries over the 8-bit cache                           hist_attention
  sample     temperature, top-k, top-p and min-p from given noise   sample_scores

`own` chooses between the plain form (torch operations in 32 bits) and the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new event for each of 64 users with up to 2,048 events: the plan before every decode step
        {"name": "plan_decode", "op": "plan", "requests": 64, "cached_lo": 1, "cached_hi": 2047, "new_lo": 1,
         "new_hi": 1, "block": 64},
        # a wave of 4,096 users, some idle, some with a long tail of unseen events: the plan of a mixed batch
        {"name": "plan_mixed", "op": "plan", "requests": 4096, "cached_lo": 0, "cached_hi": 2048, "new_lo": 0,
         "new_hi": 61, "block": 32},
        # one event of 512-d (8 heads of 64) for each of 256 requests, most blocks partly filled
        {"name": "append_decode", "op": "append", "requests": 256, "cached_lo": 0, "cached_hi": 2048, "new_lo": 1,
         "new_hi": 1, "kv_heads": 8, "dim": 64, "block": 64, "dtype": "bf16"},
        # the first pass over 64 users' histories: ragged, up to 2,048 events each
        {"name": "append_prefill", "op": "append", "requests": 64, "cached_lo": 0, "cached_hi": 0, "new_lo": 257,
         "new_hi": 2048, "kv_heads": 8, "dim": 128, "block": 64, "dtype": "bf16"},
        # one user, one event, 8 heads of 64 in fp32 (the table's own type): latency
        {"name": "attn_decode_one", "op": "attention", "requests": 1, "cached_lo": 2047, "cached_hi": 2047,
         "new_lo": 1, "new_hi": 1, "q_heads": 8, "kv_heads": 8, "dim": 64, "block": 64, "dtype": "fp32",
         "causal": True, "window": 0},
        # decode of 256 requests with ragged histories, shared key heads: bound by the cache's bytes
        {"name": "attn_decode_batch", "op": "attention", "requests": 256, "cached_lo": 65, "cached_hi": 8191,
         "new_lo": 1, "new_hi": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "block": 64, "dtype": "bf16",
         "causal": True, "window": 0},
        # two requests with very long histories, one token each: the work is along the length only
        {"name": "attn_decode_long", "op": "attention", "requests": 2, "cached_lo": 98303, "cached_hi": 131071,
         "new_lo": 1, "new_hi": 1, "q_heads": 16, "kv_heads": 2, "dim": 128, "block": 16, "dtype": "fp16",
         "causal": True, "window": 0},
        # a chunk of up to 2,048 new events behind what is cached: causal prefill, bound by the products
        {"name": "attn_prefill", "op": "attention", "requests": 8, "cached_lo": 0, "cached_hi": 2047,
         "new_lo": 1023, "new_hi": 2048, "q_heads": 16, "kv_heads": 4, "dim": 128, "block": 32, "dtype": "bf16",
         "causal": True, "window": 0},
        # 1,024 candidates of each of 64 requests look at the user's history and not at each other
        {"name": "attn_candidates", "op": "attention", "requests": 64, "cached_lo": 0, "cached_hi": 2048,
         "new_lo": 1024, "new_hi": 1024, "q_heads": 8, "kv_heads": 8, "dim": 64, "block": 64, "dtype": "bf16",
         "causal": False, "window": 0},
        # the serving score's own shape: 256 requests x 1,024 candidates, fp32
        {"name": "sample_serving", "op": "sample", "rows": 256, "items": 1024, "dtype": "fp32", "filters": "all"},
        # one request over a middling item set: latency
        {"name": "sample_one", "op": "sample", "rows": 1, "items": 32003, "dtype": "fp32", "filters": "all"},
        # 256 requests over a large item set in bf16 (many equal scores), every filter on
        {"name": "sample_large", "op": "sample", "rows": 256, "items": 131072, "dtype": "bf16", "filters": "all"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "sample", "sample"])
    biggest = {c["name"]: work(c) for c in listed()}
    while True:
        if op == "plan":
            case = {"op": op, "requests": _log_int(rng, 1, 8192), "cached_lo": 0, "cached_hi": _log_int(rng, 1, 4096),
                    "new_lo": rng.choice([0, 1]), "new_hi": _log_int(rng, 1, 300), "block": rng.choice([16, 32, 64, 128])}
            cap = biggest["plan_mixed"]
        elif op == "append":
            case = {"op": op, "requests": _log_int(rng, 1, 512), "cached_lo": 0, "cached_hi": _log_int(rng, 1, 2048),
                    "new_lo": rng.choice([0, 1]), "new_hi": _log_int(rng, 1, 2048), "kv_heads": rng.choice([1, 2, 4, 8]),
                    "dim": rng.choice([32, 64, 128, 256]), "block": rng.choice([16, 32, 64, 128]),
                    "dtype": rng.choice(["bf16", "fp16", "fp32"])}
            cap = biggest["append_prefill"]
        elif op == "attention":
            kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 16])
            new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2048)
            causal = new == 1 or rng.random() < 0.6
            case = {"op": op, "requests": _log_int(rng, 1, 256), "cached_lo": 0,
                    "cached_hi": _log_int(rng, 1, 131071 if new == 1 else 4096), "new_lo": rng.choice([0, 1]),
                    "new_hi": new, "q_heads": kv * group, "kv_heads": kv, "dim": rng.choice([32, 64, 128, 256]),
                    "block": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    "causal": causal, "window": _log_int(rng, 1, 4096) if causal and rng.random() < 0.25 else 0}
            cap = biggest["attn_decode_batch" if new == 1 else "attn_prefill"]
            padded = case["requests"] * (case["cached_hi"] + new)
            if padded * kv * case["dim"] > 2 ** 31 or padded * new * case["q_heads"] > 2 ** 30:
                continue  # the plain form pads every request to the longest
        else:
            case = {"op": op, "rows": _log_int(rng, 1, 512), "items": _log_int(rng, 1, 262144),
                    "dtype": rng.choice(["fp32", "bf16", "fp16"]),
                    "filters": rng.choice(["all", "all", "top_k", "top_p", "min_p", "none"])}
            cap = biggest["sample_large"]
        w = work(case)
        if w["bytes"] <= cap["bytes"] and w["flops"] <= cap["flops"]:
            return case


def _spread(n, lo, hi, turn):
    """n whole numbers over [lo, hi], the same for every seed (so that a case's work is known without one)."""
    if n == 1:
        return [hi]
    return [lo + int((hi - lo + 1) * (((i + 1) * turn) % 1.0)) for i in range(n)]


def _lengths(case):
    """(cached, new) of each request before the seed puts the requests in order."""
    n = case["requests"]
    cached = _spread(n, case["cached_lo"], case["cached_hi"], 0.6180339887498949)
    new = _spread(n, case["new_lo"], case["new_hi"], 0.4142135623730951)
    return cached, new


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _codes(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, g):
    """Scales of blocks of roughly unit-normal values: 3.5/127, spread by a factor of two either way."""
    return torch.randn(shape, generator=g, device="cuda").mul_(0.35).exp_().mul_(3.5 / 127)


def _order(case, seed):
    """The requests' cached and new lengths in the seed's order (int32, on the GPU), and as lists."""
    cached, new = _lengths(case)
    perm = torch.randperm(len(cached), generator=torch.Generator().manual_seed(seed + 1)).tolist()
    cached, new = [cached[i] for i in perm], [new[i] for i in perm]
    on = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return cached, new, on(cached), on(new)


def _table(held, columns, pool, g):
    """A block table [requests, columns] with held[r] random blocks of the pool in row r and -1 after them; and the rest of the pool."""
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    counts = torch.tensor(held, dtype=torch.int64, device="cuda")
    used = int(sum(held))
    first = counts.cumsum(0) - counts
    col = torch.arange(columns, device="cuda")
    table = torch.where(col < counts[:, None], ids[(first[:, None] + col).clamp(max=pool - 1)], -1)
    return table.contiguous(), ids[used:].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "sample":
        return _prepare_sample(s, case, g)
    B = case["block"]
    cached, new, s["cached"], s["new"] = _order(case, seed)
    total, columns = sum(new), max(1, _ceil(case["cached_hi"] + case["new_hi"], B))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "plan":
        held = [_ceil(c, B) for c in cached]
        want = sum(_ceil(c + n, B) for c, n in zip(cached, new)) - sum(held)
        s["table"], s["free"] = _table(held, columns, sum(held) + want + 64, g)
        s["max_tokens"] = max(1, case["requests"] * case["new_hi"])  # what the batch may hold at most
        return s
    kv, D, dtype = case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    held = [_ceil(c + n, B) for c, n in zip(cached, new)]
    pool = sum(held) + 16
    s["table"], _ = _table(held, columns, pool, g)
    s["k_codes"] = _codes((pool, kv, B, D), g)
    s["v_codes"] = _codes((pool, kv, B // 16, D, 16), g)
    s["k_scale"], s["v_scale"] = _scales((pool, kv), g), _scales((pool, kv), g)
    if case["op"] == "append":
        # keys and values are slices of one projection, as a model has them
        qkv = _normal((total, 3, kv, D), g, dtype)
        s["k"], s["v"] = qkv[:, 1], qkv[:, 2]
        pairs = [(r, p) for r in range(len(new)) for p in ((cached[r], cached[r] + new[r]),) if new[r]]
        rows = torch.tensor([r for r, _ in pairs], device="cuda").long()
        lo = torch.tensor([p[0] for _, p in pairs], device="cuda").long()
        hi = torch.tensor([p[1] for _, p in pairs], device="cuda").long()
        s["slots"] = _slots(s["table"], rows, lo, hi, B)
        s["live"] = _slots(s["table"], rows, lo // B * B, hi, B)  # what the touched blocks hold afterwards
        return s
    s["q"] = _normal((total, case["q_heads"], D), g, dtype)
    # causal queries are the newest events, already in the cache; others (candidates) are not in it
    s["lengths"] = s["cached"] + s["new"] if case["causal"] else s["cached"]
    s["max_q"] = max(1, case["new_hi"])
    s["max_len"] = case["cached_hi"] + (case["new_hi"] if case["causal"] else 0)
    # what the plain form pads and masks with
    at = torch.arange(s["max_q"], device="cuda")
    s["pad"] = (s["cu"][:-1, None] + at).clamp(max=max(total - 1, 0)).long()
    s["real"] = at < s["new"][:, None]
    return s


def _slots(table, rows, lo, hi, B):
    n = hi - lo
    owner = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    pos = torch.arange(len(owner), device="cuda") - (n.cumsum(0) - n)[owner] + lo[owner]
    return table[rows[owner], pos // B].long() * B + pos % B


def _prepare_sample(s, case, g):
    R, V, dtype = case["rows"], case["items"], DTYPES[case["dtype"]]
    x = _normal((R, V), g, scale=2.5)
    x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.005, 0.0)  # missed candidates score exactly zero
    x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.01, -math.inf)  # items already seen are masked
    s["scores"] = x.to(dtype)
    s["noise"] = torch.empty((R, V), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    u = torch.rand((4, R), generator=g, device="cuda")
    f = case["filters"]
    s["temperature"] = torch.where(u[0] < 0.1, 0.0, 0.4 + u[0])  # some rows take the best item
    s["top_k"] = (torch.exp(u[1] * math.log(1000.0)).to(torch.int32) if f in ("all", "top_k") else None)
    if f == "all":
        s["top_k"] = torch.where(u[1] < 0.2, 0, s["top_k"])  # 0: no limit
    s["top_p"] = 0.5 + 0.49 * u[2] if f in ("all", "top_p") else None
    s["min_p"] = 0.1 * u[3] * u[3] if f in ("all", "min_p") else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _RUN[s["case"]["op"], bool(own)](s)


def _own_plan(s):
    import hashed_lookup_row_amd as hlr
    slots, cu, lengths, counts = hlr.hist_plan(s["cached"], s["new"], s["table"], s["free"], s["case"]["block"],
                                               s["max_tokens"])
    return {"table": s["table"], "slots": slots, "cu": cu, "lengths": lengths, "counts": counts}


def _own_append(s):
    import hashed_lookup_row_amd as hlr
    cache = s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    hlr.hist_append(*cache, s["k"], s["v"], s["slots"])
    k, v = hlr.hist_read(*cache, s["live"], dtype=s["k"].dtype)
    return {"k": k, "v": v}


def _own_attention(s):
    import hashed_lookup_row_amd as hlr
    out, lse = hlr.hist_attention(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["table"],
                                  s["lengths"], s["cu"], s["max_q"], s["max_len"], causal=s["case"]["causal"],
                                  window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_sample(s):
    import hashed_lookup_row_amd as hlr
    index, logprob = hlr.sample_scores(s["scores"], s["noise"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return {"index": index, "logprob": logprob}


def _plain_plan(s):
    B, table, free = s["case"]["block"], s["table"], s["free"]
    cached, new = s["cached"].long(), s["new"].long()
    lengths = cached + new
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    held, need = (cached + B - 1) // B, (lengths + B - 1) // B
    more = need - held
    first = more.cumsum(0) - more
    col = torch.arange(table.shape[1], device="cuda")
    take = first[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    got = torch.where(take < free.numel(), free[take.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(fresh, got, table))
    t = torch.arange(s["max_tokens"], device="cuda")
    row = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=len(new) - 1)
    pos = cached[row] + t - cu[row]
    block = table[row, (pos // B).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where((t < cu[-1]) & (block >= 0), block * B + pos % B, -1)
    taken = more.sum().clamp(max=free.numel())
    lost = ((t < cu[-1]) & (slots < 0)).sum()
    return {"table": table, "slots": slots, "cu": cu.int(), "lengths": lengths.int(), "counts": torch.stack([taken, lost])}


def _rows_of(codes, scale, transposed):
    """Blocks as fp32 values [blocks, heads, tokens, dim]."""
    x = codes.float()
    if transposed:
        x = x.transpose(-1, -2).flatten(2, 3)
    return x * scale[..., None, None]


def _plain_append_one(codes, scale, x, slots, transposed, B):
    """Quantises x [tokens, heads, dim] into its slots; a block whose scale grows has what it holds rounded again."""
    x = torch.nan_to_num(x.float(), nan=0.0)
    block, at = slots // B, slots % B
    first = torch.full((codes.shape[0],), B, device="cuda").scatter_reduce_(0, block, at, "amin")
    top = torch.zeros_like(scale).index_reduce_(0, block, x.abs().amax(-1), "amax")
    touched = first < B
    old = torch.where((touched & (first > 0))[:, None], scale, torch.zeros_like(scale))
    fresh = top / 127.0
    fresh = torch.maximum(old, torch.where(fresh < 2.0 ** -126, torch.zeros_like(fresh), fresh))
    ids = torch.unique(block)
    inverse = torch.where(fresh > 0, 1.0 / fresh, torch.zeros_like(fresh))
    ratio = torch.where(fresh > old, old * inverse, torch.ones_like(old))[ids]
    q = codes[ids].float()
    if transposed:
        q = q.transpose(-1, -2).flatten(2, 3)
    keep = torch.arange(B, device="cuda") < first[ids][:, None]
    q = torch.where(keep[:, None, :, None], torch.round(q * ratio[..., None, None]), q)
    place = torch.zeros(codes.shape[0], dtype=torch.long, device="cuda")
    place[ids] = torch.arange(len(ids), device="cuda")
    q[place[block], :, at] = torch.round(x * inverse[block][..., None]).clamp(-127, 127)
    if transposed:
        q = q.unflatten(2, (B // 16, 16)).transpose(-1, -2)
    codes[ids] = q.to(torch.int8)
    scale.copy_(torch.where(touched[:, None], fresh, scale))


def _plain_append(s):
    B, out = s["case"]["block"], {}
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        _plain_append_one(codes, scale, s[name], s["slots"], name == "v", B)
        block, at = s["live"] // B, s["live"] % B
        q = codes[block, :, at] if name == "k" else codes[block, :, at // 16, :, at % 16]
        out[name] = (q.float() * scale[block][..., None]).to(s[name].dtype)
    return out


def _plain_attention(s):
    case = s["case"]
    R, kv, D, n = case["requests"], case["kv_heads"], case["dim"], s["max_q"]
    group = case["q_heads"] // kv
    ids = s["table"].clamp(min=0).long()
    k = _rows_of(s["k_codes"][ids].flatten(0, 1), s["k_scale"][ids].flatten(0, 1), False)
    k = k.view(R, -1, kv, case["block"], D).transpose(1, 2).reshape(R, kv, -1, D)[:, :, :s["max_len"]]
    q = s["q"][s["pad"]].float() if s["q"].shape[0] else s["q"].new_zeros((R, n, kv * group, D)).float()
    q = q.view(R, n, kv, group, D).permute(0, 2, 1, 3, 4).reshape(R, kv, n * group, D)
    score = torch.matmul(q * D ** -0.5, k.transpose(-1, -2)).view(R, kv, n, group, -1)
    del k
    pos = torch.arange(score.shape[-1], device="cuda")
    length, fresh = s["lengths"].long()[:, None, None], s["new"].long()[:, None, None]
    at = length - fresh + torch.arange(n, device="cuda")[None, :, None]
    seen = (pos < length).expand(R, n, -1)
    if case["causal"]:
        seen = seen & (pos <= at)
        if case["window"]:
            seen = seen & (pos > at - case["window"])
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.clamp(min=-3e38)).exp_()
    total = score.sum(-1, keepdim=True)
    v = _rows_of(s["v_codes"][ids].flatten(0, 1), s["v_scale"][ids].flatten(0, 1), True)
    v = v.view(R, -1, kv, case["block"], D).transpose(1, 2).reshape(R, kv, -1, D)[:, :, :s["max_len"]]
    out = torch.matmul(score.view(R, kv, n * group, -1), v).view(R, kv, n, group, D) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + total.log(), -math.inf).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[s["real"]]
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)[s["real"]]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_sample(s):
    x = s["scores"].float()
    R, V = x.shape
    t = s["temperature"][:, None]
    x = torch.where(torch.isnan(x), -math.inf, x)
    z = x / torch.where(t > 0, t, 1.0)
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = z[:, :1]
    w = torch.where(z > -math.inf, torch.exp(z - top), 0.0)
    keep = z > -math.inf
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = keep & ((torch.arange(V, device="cuda") < k) | (k <= 0))
    if s["top_p"] is not None:
        kept = torch.where(keep, w, 0.0)
        keep = keep & (kept.cumsum(1) - kept < s["top_p"][:, None] * kept.sum(1, keepdim=True))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"][:, None])
    keep[:, 0] = z[:, 0] > -math.inf
    race = torch.where(keep, z - torch.log(s["noise"].gather(1, order)), -math.inf)
    at = torch.where(t > 0, race.argmax(1, keepdim=True), 0)
    any_left = z[:, :1] > -math.inf
    index = torch.where(any_left, order.gather(1, at), -1).squeeze(1)
    logprob = torch.where(any_left, z.gather(1, at) - top - w.sum(1, keepdim=True).log(), -math.inf).squeeze(1)
    return {"index": index, "logprob": logprob}


_RUN = {("plan", True): _own_plan, ("append", True): _own_append, ("attention", True): _own_attention,
        ("sample", True): _own_sample, ("plan", False): _plain_plan, ("append", False): _plain_append,
        ("attention", False): _plain_attention, ("sample", False): _plain_sample}


# ------------------------------------------------------------------ the work
def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["rows"] * case["items"]
        # every score once; the noise of the items that the filters leave (all of them without a filter)
        noise = 4 * n if case["filters"] == "none" else 4 * case["rows"] * min(case["items"], 64)
        return {"bytes": size * n + noise + 28 * case["rows"], "flops": 4 * n}
    cached, new = _lengths(case)
    B, R, total = case["block"], case["requests"], sum(new)
    if case["op"] == "plan":
        fresh = sum(_ceil(c + n, B) - _ceil(c, B) for c, n in zip(cached, new))
        return {"bytes": 8 * R + 4 * R + 4 * (R + 1) + 8 * max(1, R * case["new_hi"]) + 8 * fresh + 4 * R, "flops": 4 * total + 8 * R}
    kv, D = case["kv_heads"], case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "append":
        live = sum(c + n - c // B * B for c, n in zip(cached, new) if n)
        # new values in, their codes out; the codes of the touched blocks in, their values out
        return {"bytes": 2 * kv * D * (total * (size + 1) + live * (size + 1)) + 8 * (total + live), "flops": 2 * kv * D * (3 * total + live)}
    pairs = 0
    for c, n in zip(cached, new):
        if not case["causal"]:
            pairs += n * c
        elif not case["window"]:
            pairs += n * c + n * (n + 1) // 2
        else:
            pairs += sum(min(case["window"], c + i + 1) for i in range(n))
    if case["causal"] and case["window"]:
        held = sum(min(c + n, case["window"] + n - 1) for c, n in zip(cached, new) if n)
    else:
        held = sum(c + (n if case["causal"] else 0) for c, n in zip(cached, new) if n)
    blocks = sum(_ceil(c + n, B) for c, n in zip(cached, new) if n)
    return {"bytes": 2 * held * kv * D + 8 * blocks * kv + 4 * blocks + total * case["q_heads"] * (2 * size * D + 4),
            "flops": 4 * pairs * case["q_heads"] * D}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](s)


def _token(codes, scale, slot, B, transposed):
    b, i = slot // B, slot % B
    q = codes[b, :, i // 16, :, i % 16] if transposed else codes[b, :, i]
    return q.double() * scale[b].double()[..., None]


def _exact_append(s):
    """Block by block: the scale (a 32-bit number by definition) from the block's largest value, codes in 64 bits."""
    B, out = s["case"]["block"], {}
    slots = s["slots"].cpu()
    block, at = slots // B, slots % B
    starts = [i for i in range(len(slots)) if i == 0 or block[i] != block[i - 1]] + [len(slots)]
    for name in ("k", "v"):
        codes = s[name + "_codes"] if name == "k" else s["v_codes"].transpose(-1, -2).flatten(2, 3).contiguous()
        scale = s[name + "_scale"].double()
        for i, j in zip(starts, starts[1:]):
            b, p = int(block[i]), int(at[i])
            x = s[name][i:j].double().transpose(0, 1)
            new = (x.abs().amax((1, 2)) / 127).float().double()
            if p > 0:
                grown = torch.maximum(new, scale[b])
                codes[b, :, :p] = torch.round(codes[b, :, :p].double() * (scale[b] / grown)[:, None, None]).to(torch.int8)
                new = grown
            scale[b] = new
            codes[b, :, p:p + j - i] = torch.round(x / new[:, None, None]).clamp(-127, 127).to(torch.int8)
        b, i = s["live"] // B, s["live"] % B
        out[name] = codes[b, :, i].double() * scale[b][..., None]
    return out


def _exact_attention(s):
    case = s["case"]
    B, kv, D, dev = case["block"], case["kv_heads"], case["dim"], s["q"].device
    group, cu = case["q_heads"] // kv, s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    for r, length in enumerate(s["lengths"].tolist()):
        lo, hi = cu[r], cu[r + 1]
        if hi == lo or length == 0:
            continue
        pos = torch.arange(length, device=dev)
        slot = s["table"][r].long()[pos // B] * B + pos % B
        k = _token(s["k_codes"], s["k_scale"], slot, B, False)
        v = _token(s["v_codes"], s["v_scale"], slot, B, True)
        at = torch.arange(length - (hi - lo), length, device=dev)[:, None]
        for h in range(case["q_heads"]):
            a = s["q"][lo:hi, h].double() @ k[:, h // group].T / math.sqrt(D)
            if case["causal"]:
                hide = pos[None] > at
                if case["window"]:
                    hide |= pos[None] <= at - case["window"]
                a[hide] = -math.inf
            lse[lo:hi, h] = torch.logsumexp(a, 1)
            out[lo:hi, h] = torch.softmax(a, 1) @ v[:, h // group]
    return {"out": out, "lse": lse}


def _exact_sample(s):
    """Row by row, on the host, from the definition: the items in order of score, cut, raced."""
    x, e = s["scores"].double().cpu(), s["noise"].double().cpu()
    R, V = x.shape
    index, logprob = torch.full((R,), -1), torch.full((R,), -math.inf, dtype=torch.float64)
    par = {k: (s[k].double().tolist() if s[k] is not None else [d] * R)
           for k, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))}
    for r in range(R):
        left = torch.nonzero(x[r] > -math.inf).flatten()
        if not len(left):
            continue
        t = par["temperature"][r]
        z = x[r, left] / (t if t > 0 else 1.0)
        z, by = torch.sort(z, descending=True, stable=True)
        left, total = left[by], torch.logsumexp(z, 0)
        n = len(z)
        if par["top_k"][r] > 0:
            n = min(n, int(par["top_k"][r]))
        p = torch.softmax(z[:n], 0)
        if s["top_p"] is not None:
            n = max(1, int((p.cumsum(0) - p < par["top_p"][r]).sum()))
        n = max(1, min(n, int((torch.exp(z[:n] - z[0]) >= par["min_p"][r]).sum())))
        i = int((z[:n] - torch.log(e[r, left[:n]])).argmax()) if t > 0 else 0
        index[r], logprob[r] = left[i], z[i] - total
    return {"index": index.cuda(), "logprob": logprob.cuda()}
