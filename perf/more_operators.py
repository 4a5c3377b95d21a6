"""Cases for the operators of a step around the paged K/V cache: norms of the
new queries and keys with their rotation, attention of ragged chunks of new
tokens (single tokens, drafts, prompts, parts of prompts) with a sliding window
and first tokens that stay visible, and attention of a batch whose requests
share a prefix.

Conventions (those of include/qsa_cache.h and include/qsa_chunk.h): a cache is
K and V views [pages, page_size, kv_heads, head_dim]; entry e of a table's row
lives in page row[e // page_size], slot e % page_size.  Request b's new tokens
are the tokens [query_start_loc[b], query_start_loc[b+1]); its token j of n
sees the entries e < hi = context_lens[b] - n + j + 1 with e >= hi - window
(where there is a window) or e < num_sink, and in the prefix form all entries
below the prefix's length besides.  Tokens behind the last request are padding
and keep what their outputs held.

``run`` with ``own`` false is the plain form: elementary torch operations in
binary32 (angles in binary64), rounded once at the end.
"""
import math

import torch

own = False

F16, BF16, E4M3 = "float16", "bfloat16", "float8_e4m3fn"


def _rope(name, tokens, pad, first, heads, kv_heads, dim, rot, interleaved, base, layout, dtype):
    return {"name": name, "op": "rope", "tokens": tokens, "pad": pad, "first": first,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "base": base, "layout": layout, "dtype": dtype}


def _chunk(name, batch, new, old, heads, kv_heads, dim, page, layout, dtype, cache, window=0,
           sink=0, pad=0):
    return {"name": name, "op": "chunk", "batch": batch, "new_low": new[0], "new_high": new[1],
            "old_low": old[0], "old_high": old[1], "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "layout": layout, "dtype": dtype, "cache": cache,
            "window": window, "sink": sink, "pad": pad, "prefix": 0}


def _prefix(name, batch, prefix, new, old, heads, kv_heads, dim, page, layout, dtype, cache, pad=0):
    c = _chunk(name, batch, new, old, heads, kv_heads, dim, page, layout, dtype, cache, pad=pad)
    return {**c, "op": "prefix", "prefix": prefix}


def listed():
    return [
        # one token of the decode path's attention heads (3 of 256 over one K/V head)
        _rope("rope_one_token", 1, 0, 9214, 3, 1, 256, 64, False, 1e6, "split", F16),
        # the new tokens of an ordinary serving batch, q, k and v side by side as one projection
        # leaves them, far into long documents
        _rope("rope_step_256", 256, 0, 131072, 32, 8, 128, 128, False, 1e6, "fused", BF16),
        # the tokens of prompts, the batch padded to a fixed size, pairs side by side
        _rope("rope_prompt_16384", 16344, 40, 0, 32, 8, 128, 128, True, 1e4, "split", BF16),
        # the step of a streaming chat: one new token a request, a window and four sinks
        _chunk("chunk_step_64", 64, (1, 1), (1, 50000), 32, 8, 128, 64, "split", BF16, BF16,
               window=4096, sink=4),
        # one request's single token in the decode path's packed pages
        _chunk("chunk_one_9215", 1, (1, 1), (9214, 9214), 3, 1, 256, 512, "packed", F16, F16),
        # whole prompts of ordinary lengths, the batch padded
        _chunk("chunk_prompts_12", 12, (1, 4096), (0, 0), 32, 8, 128, 64, "split", BF16, BF16,
               pad=24),
        # one long prompt through layers with a window and sinks, heads of 64
        _chunk("chunk_window_32768", 1, (32768, 32768), (0, 0), 16, 4, 64, 16, "heads", F16, F16,
               window=4096, sink=4),
        # a part of a long prompt in the decode path's packed pages
        _chunk("chunk_part_2048", 1, (2048, 2048), (63488, 63488), 3, 1, 256, 512, "packed", F16,
               F16),
        # prompts in parts beside requests that decode, over an 8-bit cache
        _chunk("chunk_mixed_e4m3", 24, (1, 400), (0, 16384), 32, 8, 128, 64, "split", BF16, E4M3),
        # a few requests behind a short system prompt
        _prefix("prefix_chat_8", 8, 2000, (1, 1), (1, 255), 32, 8, 128, 64, "split", BF16, BF16),
        # many requests over one long document
        _prefix("prefix_document_256", 256, 32768, (1, 1), (1, 1023), 32, 8, 128, 64, "split",
                BF16, BF16),
        # drafts of three and the last token behind a long prefix, the decode path's packed pages
        _prefix("prefix_draft_64", 64, 100000, (4, 4), (0, 511), 3, 1, 256, 512, "packed", F16,
                F16),
    ]


def _between(rng, low, high):
    """A whole number, spread over the range's logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "chunk", "prefix", "prefix"])
    dtype = rng.choice([F16, BF16])
    layout = rng.choice(["packed", "split", "heads"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
        tokens = _between(rng, 1, min(32768, 167_000_000 // (2 * dim * (heads + kv_heads))))
        c = _rope("", tokens, rng.choice([0, rng.randint(0, 63)]), rng.choice([0, _between(rng, 1, 1 << 20)]),
                  heads, kv_heads, dim, rng.choice([dim // 32 * 16, dim // 16 * 16]),
                  rng.random() < 0.5, rng.choice([1e4, 5e5, 1e6]), rng.choice(["split", "fused"]),
                  dtype)
        c.pop("name")
        return c
    while True:
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 16])
        page = rng.choice([16, 32, 64, 128, 512])
        cache = rng.choice([dtype, dtype, E4M3])
        kind = rng.choice(["step", "step", "prompt", "part"])
        pad = rng.choice([0, 0, rng.randint(0, 63)])
        if kind == "step":
            batch = _between(rng, 1, 256)
            new_high = rng.choice([1, 1, 2, 4, 8])
            new_low = rng.choice([1, new_high])
            old_high = _between(rng, 1, 131072 if op == "chunk" else 4096)
        elif kind == "prompt":
            batch = _between(rng, 1, 32)
            new_high = _between(rng, 2, 32768 if op == "chunk" else 2048)
            new_low = max(1, int(new_high * rng.choice([0.01, 0.5, 1.0])))
            old_high = 0
        else:
            batch = _between(rng, 1, 48)
            new_high = _between(rng, 1, 4096)
            new_low = rng.choice([1, new_high])
            old_high = _between(rng, 1, 65536 if op == "chunk" else 4096)
        old = (int(old_high * rng.choice([0.0, 0.25, 1.0])), old_high)
        if op == "chunk":
            window = rng.choice([0, _between(rng, 1, 8192)])
            sink = rng.choice([0, 4, _between(rng, 1, 300)]) if window else 0
            c = _chunk("", batch, (new_low, new_high), old, heads, kv_heads, dim, page, layout,
                       dtype, cache, window, sink, pad)
        else:
            c = _prefix("", batch, _between(rng, 1, 131072), (new_low, new_high), old, heads,
                        kv_heads, dim, page, layout, dtype, cache, pad)
        # no more than the largest listed cases: their products, and their caches
        entry = 2 * kv_heads * dim * _size(cache)
        w = work(c)
        if w["flops"] <= 1.2e12 and w["bytes"] <= 1.2e9 and \
                (batch * (old_high + new_high) + c["prefix"]) * entry <= 8e9:
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
    """(new tokens, cached tokens with them) of each request: the same for every seed, so that a
    case is one amount of work."""
    cpu = torch.Generator().manual_seed(case["batch"] * 7919 + case["old_high"] * 31 + case["new_high"])
    new = torch.randint(case["new_low"], case["new_high"] + 1, (case["batch"],), generator=cpu)
    old = torch.randint(case["old_low"], case["old_high"] + 1, (case["batch"],), generator=cpu)
    new[0], old[0] = case["new_high"], case["old_high"]
    return new, old + new


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_rope if case["op"] == "rope" else _prepare_attend)(case, gen)


def _prepare_rope(case, gen):
    t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    all_t, dt = t + case["pad"], getattr(torch, case["dtype"])
    s = dict(case)
    if case["layout"] == "fused":            # q, k and v of a token side by side
        x = _values((all_t, hq + 2 * hk, d), dt, gen)
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
    else:
        s["q"], s["k"] = _values((all_t, hq, d), dt, gen), _values((all_t, hk, d), dt, gen)
    # learned weights stay near one
    s["q_weight"], s["k_weight"] = ((1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
                                    for _ in range(2))
    r = case["rot"]
    s["inv_freq"] = (case["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(
        "cuda", torch.float32)
    if t <= 1024:                            # a step: every request somewhere in its context
        pos = case["first"] + torch.randint(0, 4096, (t,), generator=gen, device="cuda")
    else:
        pos = case["first"] + torch.arange(t, device="cuda")
    s["positions"] = torch.cat([pos, torch.full((case["pad"],), -1, device="cuda")])
    s["q_out"] = torch.zeros((all_t, hq, d), dtype=dt, device="cuda")
    s["k_out"] = torch.zeros((all_t, hk, d), dtype=dt, device="cuda")
    return s


def _prepare_attend(case, gen):
    b, ps, hk, d = case["batch"], case["page"], case["kv_heads"], case["dim"]
    new, ctx = _lengths(case)
    s = dict(case)
    cols, pcols = -(-int(ctx.max()) // ps), -(-case["prefix"] // ps)
    s["k"], s["v"] = _cache(case, b * cols + pcols, gen)
    pages = torch.randperm(b * cols + pcols, generator=gen, device="cuda").to(torch.int32)
    s["tables"], s["prefix_table"] = pages[:b * cols].view(b, cols), pages[b * cols:]
    s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    s["ctx"] = ctx.to("cuda", torch.int32)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    s["start"] = start.to("cuda", torch.int32)
    # what the host of a serving loop knows of its own batch
    s["new"], s["lens"], s["tokens"] = new.tolist(), ctx.tolist(), int(start[-1])
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == E4M3:                # one scale per K/V head, as calibration leaves them
        s["k_scale"] = 0.5 + torch.rand(hk, generator=gen, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(hk, generator=gen, device="cuda")
    rows, dt = s["tokens"] + case["pad"], getattr(torch, case["dtype"])
    s["q"] = _values((rows, case["heads"], d), dt, gen)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((rows, case["heads"]), device="cuda")
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# --- one pass -------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return (_rope_plain if s["op"] == "rope" else _attend_plain)(s)


def _run_own(s):
    import sparse_paged_attention_qsa_gb300 as qsa
    if s["op"] == "rope":
        qsa.qsa_qk_norm_rope(
            s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"], inv_freq=s["inv_freq"],
            interleaved=s["interleaved"], eps=1e-6, q_out=s["q_out"], k_out=s["k_out"])
        return [s["q_out"], s["k_out"]]
    if s["op"] == "chunk":
        qsa.qsa_chunk_attention(
            s["q"], s["k"], s["v"], s["tables"], s["start"], s["ctx"], window=s["window"],
            num_sink=s["sink"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
            lse=s["lse"], error_word=s["err"])
    else:
        qsa.qsa_prefix_attention(
            s["q"], s["k"], s["v"], s["prefix_table"], s["prefix_len"], s["tables"], s["start"],
            s["ctx"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"],
            error_word=s["err"])
    return [s["out"], s["lse"]]


def _rope_plain(s):
    t, r = s["tokens"], s["rot"]
    angle = s["positions"][:t, None].double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    for x, w, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        y = x[:t].float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if s["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[:t] = torch.cat([z, y[..., r:]], -1).to(out.dtype)
    return [s["q_out"], s["k_out"]]


def _entries(s, table, count):
    """Entries [0, count) of a table's row, K and V as [kv_heads, count, dim] in binary32."""
    pages = table[:-(-count // s["page"])].long()
    got = []
    for cache, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = cache[pages].flatten(0, 1)[:count].float()
        got.append((x if scale is None else x * scale[:, None]).transpose(0, 1))
    return got


def _attend_plain(s):
    hk, d = s["kv_heads"], s["dim"]
    group = s["heads"] // hk
    if s["prefix"]:
        pk, pv = _entries(s, s["prefix_table"], s["prefix"])
    t0 = 0
    for b, (n, ctx) in enumerate(zip(s["new"], s["lens"])):
        k, v = _entries(s, s["tables"][b], ctx)
        e = torch.arange(ctx, device="cuda")
        if s["prefix"]:
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
            e = torch.cat([torch.full((s["prefix"],), -1, device="cuda"), e])
        block = max(1, (1 << 28) // (s["heads"] * k.shape[1]))
        for j0 in range(0, n, block):
            m = min(block, n - j0)
            rows = slice(t0 + j0, t0 + j0 + m)
            q = s["q"][rows].float().view(m, hk, group, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            z = (q @ k.transpose(1, 2)).view(hk, group, m, -1) / math.sqrt(d)
            hi = ctx - n + j0 + 1 + torch.arange(m, device="cuda")[:, None]
            seen = e < hi
            if s["window"]:
                seen &= (e >= hi - s["window"]) | (e < s["sink"])
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            out = (p / total).view(hk, group * m, -1) @ v
            s["out"][rows] = out.view(hk, group, m, d).permute(2, 0, 1, 3).reshape(
                m, -1, d).to(s["out"].dtype)
            s["lse"][rows] = (top + torch.log(total)).permute(2, 0, 1, 3).reshape(m, -1)
        t0 += n
    return [s["out"], s["lse"]]


# --- the definition in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return (_rope_exact if case["op"] == "rope" else _attend_exact)(s)


def _rope_exact(s):
    t, r, d = s["tokens"], s["rot"], s["dim"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"][:t].double(), s["inv_freq"].double()))
    first = torch.arange(0, r, 2) if s["interleaved"] else torch.arange(r // 2)
    second = first + 1 if s["interleaved"] else first + r // 2
    got = []
    for x, w, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        y = x[:t].double()
        y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / d + 1e-6)
        y = y * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        full = out.double()
        full[:t] = y
        got.append(full)
    return got


def _attend_exact(s):
    hq, hk, d, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    group = hq // hk
    out, lse = s["out"].double(), s["lse"].double()

    def wide(cache, scale, table, h, lo, hi):
        x = cache[table[lo // page:-(-hi // page)].long(), :, h].reshape(-1, d).double()
        x = x[lo - lo // page * page:][:hi - lo]
        return x if scale is None else x * scale[h].double()

    t0 = 0
    for b, (n, ctx) in enumerate(zip(s["new"], s["lens"])):
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            for j0 in range(0, n, 2048):
                m = min(2048, n - j0)
                rows = slice(t0 + j0, t0 + j0 + m)
                low, high = ctx - n + j0 + 1, ctx - n + j0 + m     # entries below the first's, last's
                parts = []                                         # (table, from, to)
                if s["prefix"]:
                    parts.append((s["prefix_table"], 0, s["prefix"], None))
                lo = max(0, low - s["window"]) if s["window"] else 0
                if 0 < min(s["sink"], lo):
                    parts.append((s["tables"][b], 0, min(s["sink"], lo), 0))
                parts.append((s["tables"][b], lo, high, 0))
                k = torch.cat([wide(s["k"], s["k_scale"], t, h, x, y) for t, x, y, _ in parts])
                v = torch.cat([wide(s["v"], s["v_scale"], t, h, x, y) for t, x, y, _ in parts])
                at = torch.cat([torch.arange(x, y, device="cuda") if own_ == 0 else
                                torch.full((y - x,), -1, device="cuda") for _, x, y, own_ in parts])
                last = torch.arange(low - 1, high, device="cuda")[:, None]      # the token's own entry
                hide = at > last
                if s["window"]:
                    hide |= (at <= last - s["window"]) & (at >= s["sink"])
                for g in range(group):
                    z = s["q"][rows, h * group + g].double() @ k.T * d ** -0.5
                    z.masked_fill_(hide, -math.inf)
                    total = torch.logsumexp(z, 1)
                    lse[rows, h * group + g] = total
                    out[rows, h * group + g] = torch.exp(z - total[:, None]) @ v
        t0 += n
    return [out, lse]


# --- what a pass cannot do without ------------------------------------------------


def work(case):
    if case["op"] == "rope":
        elements = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4.0 * elements + 8.0 * case["tokens"] + 4.0 * case["dim"]
                + 2.0 * case["rot"], "flops": 7.0 * elements}
    new, ctx = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    tokens, seen, read = int(new.sum()), 0, case["prefix"]
    for n, c in zip(new.tolist(), ctx.tolist()):
        hi = torch.arange(c - n + 1, c + 1)
        lo = (hi - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(hi)
        seen += int((hi - lo + torch.clamp(lo, max=case["sink"])).sum()) + n * case["prefix"]
        read += c - int(lo[0]) + min(int(lo[0]), case["sink"])
    entry = 2 * hk * d * _size(case["cache"])                # K and V of one entry
    bytes_ = read * entry + tokens * (4.0 * hq * d + 4 * hq) + 4.0 * read / case["page"] \
        + 8.0 * case["batch"]
    return {"bytes": bytes_, "flops": 4.0 * seen * hq * d}
