"""Cases for the paged K/V cache operators: appending new tokens, dense decode
attention over the cached entries (with the attention weight each entry
received, when asked), and eviction by that weight.

Conventions (those of include/qsa_cache.h): a cache is K and V views
[pages, page_size, kv_heads, head_dim]; request b's entry e lives in page
block_tables[b, e // page_size], slot e % page_size; query row b*next_n + j
sees the entries [hi - window, hi), hi = context_lens[b] - next_n + j + 1.

``run`` with ``own`` false is the plain form: elementary torch operations in
binary32 over the padded batch, rounded once at the end.
"""
import math

import torch

own = False

F16, BF16, E4M3 = "float16", "bfloat16", "float8_e4m3fn"
E4M3_MAX = 448.0


def _attend(name, batch, low, high, heads, kv_heads, dim, page, layout, dtype, cache, next_n=1,
            window=0, weights=False):
    return {"name": name, "op": "attend", "batch": batch, "low": low, "high": high, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout, "dtype": dtype,
            "cache": cache, "next_n": next_n, "window": window, "weights": weights}


def _evict(name, batch, low, high, budget, sink, recent, kv_heads, dim, page, layout, cache):
    return {"name": name, "op": "evict", "batch": batch, "low": low, "high": high,
            "budget": budget, "sink": sink, "recent": recent, "kv_heads": kv_heads, "dim": dim,
            "page": page, "layout": layout, "cache": cache}


def _append(name, batch, low, high, tokens, pad, kv_heads, dim, page, layout, dtype, cache):
    return {"name": name, "op": "append", "batch": batch, "low": low, "high": high,
            "tokens": tokens, "pad": pad, "kv_heads": kv_heads, "dim": dim, "page": page,
            "layout": layout, "dtype": dtype, "cache": cache}


def listed():
    return [
        # one interactive request at the decode path's shortest worked size, in its own packed
        # 512-token pages (3 heads of 256 over one K/V head)
        _attend("attend_one_519", 1, 519, 519, 3, 1, 256, 512, "packed", F16, F16),
        # one request far into a long document: few rows, the work has to be split over the length
        _attend("attend_one_131072", 1, 131072, 131072, 32, 8, 128, 64, "split", BF16, BF16),
        # the decode path's mixed batch, 512 to 65536 tokens per request
        _attend("attend_mixed_64", 64, 512, 65536, 3, 1, 256, 512, "packed", F16, F16),
        # the decode path's long context: every request at 131072 tokens
        _attend("attend_long_32", 32, 131072, 131072, 3, 1, 256, 512, "packed", F16, F16),
        # an ordinary serving batch of grouped heads, short and long chats together
        _attend("attend_chat_96", 96, 1, 8191, 32, 8, 128, 64, "split", BF16, BF16),
        # long contexts in an 8-bit cache
        _attend("attend_e4m3_24", 24, 16384, 65536, 64, 8, 128, 64, "split", BF16, E4M3),
        # speculative decoding (a draft of three and the last token) with a sliding window
        _attend("attend_draft_48", 48, 2000, 50000, 16, 4, 64, 16, "heads", F16, F16, next_n=4,
                window=4096),
        # a bounded cache: the step's attention also adds up what weight each entry receives
        _attend("attend_weighed_32", 32, 4097, 16384, 32, 8, 128, 64, "split", F16, F16,
                weights=True),
        # a bounded cache at its budget: a page's worth of entries leaves in each request
        _evict("evict_step_64", 64, 2064, 2064, 2048, 4, 256, 8, 128, 16, "split", F16),
        # prompts read in full, then cut down to the budget before decoding starts
        _evict("evict_prompt_16", 16, 20000, 65536, 8192, 4, 512, 8, 128, 64, "split", BF16),
        # the new tokens of one decode step
        _append("append_step_256", 256, 1, 2048, 256, 0, 1, 256, 512, "packed", F16, F16),
        # the tokens of prompts in an 8-bit cache, the batch padded to a fixed size
        _append("append_prompt_e4m3", 12, 1, 4096, 16384, 40, 8, 128, 64, "split", BF16, E4M3),
    ]


def _between(rng, low, high):
    """A whole number, spread over the range's logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "evict", "append"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 512])
    layout = rng.choice(["packed", "split", "heads"])
    dtype = rng.choice([F16, BF16])
    cache = rng.choice([dtype, dtype, E4M3])
    # cached tokens of the whole batch: at most the longest listed batch's bytes
    per_token = 2 * kv_heads * dim * (1 if cache == E4M3 else 2)
    most = 3_000_000_000 // per_token
    if op == "attend":
        batch = _between(rng, 1, 256)
        high = _between(rng, 16, min(131072, most // batch))
        low = max(1, int(high * rng.choice([0.01, 0.25, 1.0])))
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        next_n = rng.choice([1, 1, 1, 2, 4])
        window = rng.choice([0, 0, 0, _between(rng, 1, high)])
        weights = rng.choice([False, False, True])
        c = _attend("", batch, low, high, group * kv_heads, kv_heads, dim, page, layout, dtype,
                    cache, next_n, window, weights)
    elif op == "evict":
        batch = _between(rng, 1, 64)
        high = _between(rng, 64, min(131072, most // batch))
        low = max(1, int(high * rng.choice([0.1, 0.5, 1.0])))
        budget = max(16, int(high * rng.uniform(0.05, 0.99)))
        c = _evict("", batch, low, high, budget, rng.choice([0, 4]), rng.randint(0, budget // 4),
                   kv_heads, dim, page, layout, cache)
    else:
        tokens = _between(rng, 1, 32768)
        batch = rng.randint(1, min(tokens, 256))
        high = max(_between(rng, 1, 4096), -(-tokens // batch))
        high = min(high, max(most // batch, -(-tokens // batch)))
        c = _append("", batch, 1, high, tokens, rng.randint(0, 63), kv_heads, dim, page, layout,
                    dtype, cache)
    c.pop("name")
    return c


# --- inputs -------------------------------------------------------------------


def _size(name):
    return 1 if name == E4M3 else 2


def _values(shape, dtype, gen):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda").to(dtype)
    return out


def _cache(case, pages, gen):
    """K and V views [pages, page_size, kv_heads, dim] in the case's layout."""
    ps, hk, d = case["page"], case["kv_heads"], case["dim"]
    dt = getattr(torch, case["cache"])
    if case["layout"] == "packed":           # a token's K and V side by side
        kv = _values((pages, ps, 2, hk, d), dt, gen)
        return kv[:, :, 0], kv[:, :, 1]
    if case["layout"] == "heads":            # a page's tokens head by head
        return tuple(_values((pages, hk, ps, d), dt, gen).transpose(1, 2) for _ in range(2))
    return tuple(_values((pages, ps, hk, d), dt, gen) for _ in range(2))


def _lengths(case):
    """Cached tokens of each request: the same for every seed, so that a case is one amount of
    work."""
    cpu = torch.Generator().manual_seed(case["batch"] * 7919 + case["high"])
    n = torch.randint(case["low"], case["high"] + 1, (case["batch"],), generator=cpu)
    n[0] = case["high"]
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, ps, hk, d = case["batch"], case["page"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    cols = -(-case["high"] // ps)
    s = dict(case)
    s["k"], s["v"] = _cache(case, b * cols, gen)
    s["tables"] = torch.randperm(b * cols, generator=gen, device="cuda").to(torch.int32).view(b, cols)
    s["lens"] = lens.to("cuda", torch.int32)
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == E4M3:                # one scale per K/V head, as calibration leaves them
        s["k_scale"] = 0.5 + torch.rand(hk, generator=gen, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(hk, generator=gen, device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        s["q"] = _values((b * case["next_n"], case["heads"], d), getattr(torch, case["dtype"]), gen)
        s["lse"] = torch.empty((b * case["next_n"], case["heads"]), device="cuda")
        if case["weights"]:
            s["sums"] = torch.rand((b, cols * ps), generator=gen, device="cuda")
            s["sums_out"] = torch.zeros((b, cols * ps), device="cuda")
    elif case["op"] == "evict":
        # weights as attention leaves them: a few entries hold most
        s["sums"] = torch.rand((b, cols * ps), generator=gen, device="cuda").pow(8.0)
        # each request's positions in the order its entries were written, a few places swapped by
        # earlier evictions
        pos = torch.arange(cols * ps, device="cuda", dtype=torch.int32).repeat(b, 1)
        half = int(lens.min()) // 2
        if half:
            a = torch.randint(half, (64,), generator=gen, device="cuda").unique()
            pos[:, a], pos[:, a + half] = pos[:, a + half].clone(), pos[:, a].clone()
        s["positions"] = pos
    else:
        t, dt = case["tokens"], getattr(torch, case["dtype"])
        s["new_k"] = _values((t + case["pad"], hk, d), dt, gen)
        s["new_v"] = _values((t + case["pad"], hk, d), dt, gen)
        # the last tokens of each request, the batch's token count dealt out evenly
        count = torch.full((b,), t // b)
        count[:t % b] += 1
        end = torch.maximum(lens, count)
        req = torch.repeat_interleave(torch.arange(b), count)
        entry = torch.arange(t) - torch.repeat_interleave(count.cumsum(0) - end, count)
        none = torch.full((case["pad"],), -1)
        s["requests"] = torch.cat([req, torch.zeros_like(none)]).to("cuda", torch.int32)
        s["entries"] = torch.cat([entry, none]).to("cuda")
        s["positions"] = s["entries"] + 5
        s["entry_positions"] = torch.zeros((b, cols * ps), dtype=torch.int32, device="cuda")
        s["sums"] = torch.rand((b, cols * ps), generator=gen, device="cuda")
    return s


# --- one pass -------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return {"attend": _attend_plain, "evict": _evict_plain, "append": _append_plain}[s["op"]](s)


def _run_own(s):
    import sparse_paged_attention_qsa_gb300 as qsa
    if s["op"] == "attend":
        out = qsa.qsa_paged_attention(
            s["q"], s["k"], s["v"], s["tables"], s["lens"], next_n=s["next_n"],
            window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=s["lse"],
            weight_sums=s.get("sums"), weight_sums_out=s.get("sums_out"), error_word=s["err"])
        return [out, s["lse"]] + ([s["sums_out"]] if s["weights"] else [])
    if s["op"] == "evict":
        got = qsa.qsa_evict_entries(
            s["sums"], s["positions"], s["lens"], s["k"], s["v"], s["tables"], s["budget"],
            num_sink=s["sink"], num_recent=s["recent"], error_word=s["err"])
        return [*got, s["k"], s["v"]]
    qsa.qsa_paged_append(
        s["new_k"], s["new_v"], s["k"], s["v"], s["tables"], s["requests"], s["entries"],
        k_scale=s["k_scale"], v_scale=s["v_scale"], positions=s["positions"],
        entry_positions=s["entry_positions"], weight_sums=s["sums"], error_word=s["err"])
    return [s["k"], s["v"], s["entry_positions"], s["sums"]]


def _entries_of(cache, tables, scale):
    """The requests' entries in order, [batch, columns * page_size, kv_heads, dim] in binary32."""
    x = cache[tables.long()].flatten(1, 2).float()
    return x if scale is None else x * scale[:, None]


def _attend_plain(s):
    b, n, hk, d = s["batch"], s["next_n"], s["kv_heads"], s["dim"]
    q = s["q"].float().view(b, n, hk, -1, d)
    k = _entries_of(s["k"], s["tables"], s["k_scale"])
    v = _entries_of(s["v"], s["tables"], s["v_scale"])
    t = torch.arange(k.shape[1], device="cuda")
    hi = s["lens"][:, None] - n + 1 + torch.arange(n, device="cuda")
    seen = t < hi[..., None]
    if s["window"]:
        seen &= t >= (hi - s["window"])[..., None]
    z = torch.einsum("bnhgd,bthd->bhngt", q, k) / math.sqrt(d)
    z = z.masked_fill(~seen[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    out = torch.einsum("bhngt,bthd->bnhgd", p, v)
    lse = (m + torch.log(total)).permute(0, 2, 1, 3, 4)
    s["lse"].copy_(lse.reshape(b * n, -1))
    got = [out.reshape(b * n, -1, d).to(s["q"].dtype), s["lse"]]
    if s["weights"]:
        sums = s["sums"] + p.sum((1, 2, 3))
        s["sums_out"].copy_(torch.where(t < s["lens"][:, None], sums, s["sums_out"]))
        got.append(s["sums_out"])
    return got


def _evict_plain(s):
    sums, pos, lens, budget = s["sums"], s["positions"], s["lens"][:, None], s["budget"]
    t = torch.arange(sums.shape[1], device="cuda")
    there = t < lens
    newest = torch.where(there, pos, torch.full_like(pos, -1)).amax(1, keepdim=True)
    safe = (pos < s["sink"]) | (pos > newest - s["recent"])
    key = torch.where(safe, torch.full_like(sums, math.inf), sums)
    key = torch.where(there, key, torch.full_like(sums, -math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    keep = torch.zeros_like(there).scatter_(1, order, True) & there
    # the kept entries past the budget, in order, take the places that the evicted ones leave
    moved = torch.sort((~(keep & (t >= budget))).to(torch.int8), dim=1, stable=True).indices
    i = t[:budget]
    hole = ~keep[:, :budget]
    rank = (hole.cumsum(1) - 1).clamp(min=0)
    kept = torch.where(hole, moved.gather(1, rank), i)
    kept = torch.where(i < lens, kept, torch.full_like(kept, -1))
    at = kept.clamp(min=0)
    old = torch.where(kept < 0, i, kept)
    page = s["page"]
    dst = (s["tables"].long()[:, i // page], (i % page).expand_as(at))
    src = (s["tables"].long().gather(1, old // page), old % page)
    for cache in (s["k"], s["v"]):
        x = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        x[dst] = x[src]
    new_sums = torch.where(kept < 0, torch.zeros_like(sums[:, :1]), sums.gather(1, at))
    new_pos = torch.where(kept < 0, torch.full_like(pos[:, :1], -1), pos.gather(1, at))
    return [kept.to(torch.int32), s["lens"].clamp(max=budget), new_sums, new_pos, s["k"], s["v"]]


def _append_plain(s):
    t = s["tokens"]                          # behind them is the batch's padding
    req, entry = s["requests"][:t].long(), s["entries"][:t]
    page, slot = s["tables"][req, entry // s["page"]].long(), entry % s["page"]
    k, v = s["new_k"][:t], s["new_v"][:t]
    if s["cache"] == E4M3:
        k = (k.float() / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v.float() / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        s["k"].view(torch.uint8)[page, slot] = k
        s["v"].view(torch.uint8)[page, slot] = v
    else:
        s["k"][page, slot] = k
        s["v"][page, slot] = v
    s["entry_positions"][req, entry] = s["positions"][:t].to(torch.int32)
    s["sums"][req, entry] = 0.0
    return [s["k"], s["v"], s["entry_positions"], s["sums"]]


# --- the definition in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _attend_exact, "evict": _evict_exact, "append": _append_exact}[case["op"]](s)


def _attend_exact(s):
    b, n, hq, hk, d = s["batch"], s["next_n"], s["heads"], s["kv_heads"], s["dim"]
    out = torch.zeros((b * n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b * n, hq), -math.inf, dtype=torch.float64, device="cuda")
    sums = s["sums_out"].double() if s["weights"] else None
    q = s["q"].double()
    lens = s["lens"].tolist()
    for i in range(b):
        pages = s["tables"][i, :-(-lens[i] // s["page"])].long()
        if sums is not None:
            sums[i, :lens[i]] = s["sums"][i, :lens[i]].double()
        for h in range(hk):
            k = s["k"][pages, :, h].reshape(-1, d)[:lens[i]].double()
            v = s["v"][pages, :, h].reshape(-1, d)[:lens[i]].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            for j in range(n):
                hi = lens[i] - n + j + 1
                lo = max(0, hi - s["window"]) if s["window"] else 0
                if hi <= lo:
                    continue
                z = q[i * n + j, heads] @ k[lo:hi].T * d ** -0.5
                lse[i * n + j, heads] = torch.logsumexp(z, 1)
                w = torch.softmax(z, 1)
                out[i * n + j, heads] = w @ v[lo:hi]
                if sums is not None:
                    sums[i, lo:hi] += w.sum(0)
    return [out, lse] + ([sums] if sums is not None else [])


def _evict_exact(s):
    b, budget = s["batch"], s["budget"]
    kept = torch.full((b, budget), -1, dtype=torch.int64)
    new_sums = torch.zeros((b, budget), dtype=torch.float64)
    new_pos = torch.full((b, budget), -1, dtype=torch.int64)
    lens = s["lens"].tolist()
    for i in range(b):
        n = lens[i]
        w, p = s["sums"][i, :n].double().cpu(), s["positions"][i, :n].long().cpu()
        if n <= budget:
            place = torch.arange(n)
        else:
            rank = w.clone()
            rank[(p < s["sink"]) | (p >= int(p.max()) + 1 - s["recent"])] = math.inf
            chosen = torch.argsort(-rank, stable=True)[:budget].sort().values
            stay = chosen[chosen < budget]
            place = torch.full((budget,), -1)
            place[stay] = stay
            place[place < 0] = chosen[chosen >= budget]
        kept[i, :len(place)] = place
        new_sums[i, :len(place)] = w[place]
        new_pos[i, :len(place)] = p[place]
    return [kept, torch.tensor([min(n, budget) for n in lens]), new_sums, new_pos, None, None]


def _append_exact(s):
    cap = s["tables"].shape[1] * s["page"]
    t = s["tokens"]
    where = s["requests"][:t].long() * cap + s["entries"][:t]
    line = s["tables"].long().view(-1)[where // s["page"]] * s["page"] + where % s["page"]
    got = []
    for new, cache, scale in ((s["new_k"], s["k"], s["k_scale"]), (s["new_v"], s["v"], s["v_scale"])):
        x = cache.double().reshape(-1, *cache.shape[2:])
        y = new[:t].double()
        x[line] = y if scale is None else (y / scale.double()[:, None]).clamp(-448, 448)
        got.append(x.view(cache.shape))
    pos, sums = s["entry_positions"].long().view(-1), s["sums"].double().view(-1)
    pos[where] = s["positions"][:t]
    sums[where] = 0
    return [*got, pos.view(s["batch"], cap), sums.view(s["batch"], cap)]


# --- what a pass cannot do without ------------------------------------------------


def work(case):
    n = _lengths(case).double()
    hk, d, cs = case["kv_heads"], case["dim"], _size(case["cache"])
    entry = 2 * hk * d * cs                                  # K and V of one entry
    if case["op"] == "attend":
        rows, hq, nn = case["batch"] * case["next_n"], case["heads"], case["next_n"]
        j = torch.arange(nn)
        hi = (n[:, None] - nn + j + 1).clamp(min=0)
        lo = (hi - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(hi)
        read = float((hi[:, -1] - lo[:, 0]).sum())
        per = 2 * hq * d * 2 + 4 * hq                        # q, out and lse of a row
        bytes_ = read * entry + rows * per + 4 * read / case["page"] + 4 * case["batch"]
        flops = float((hi - lo).sum()) * hq * d * 4
        if case["weights"]:
            bytes_ += 8 * float(n.sum())
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "evict":
        budget = case["budget"]
        safe = min(budget, case["sink"] + case["recent"])
        over = n[n > budget]
        # entries past the budget that stay: the recent ones, and the others' share of the rest
        share = (budget - safe) / (over - safe)
        moved = float(((over - budget - case["recent"]).clamp(min=0) * share
                       + torch.minimum(over - budget, torch.full_like(over, case["recent"]))).sum())
        return {"bytes": 8 * float(over.sum()) + moved * 2 * entry + 12 * case["batch"] * budget,
                "flops": 0.0}
    t = case["tokens"]
    return {"bytes": t * (2 * hk * d * (2 + cs) + 4 + 8 + 8 + 4 + 4), "flops": 0.0}
