"""Cases that measure the paged-cache operators: the tables built from request lengths, the append
of new keys and values, and the attention of new tokens (chunks or single tokens) over the pages.

Each case runs one operator. Request lengths are part of the case (drawn from its `lens` number by
the functions below), tensor values come from the seed. Where `own` is false the operators are
computed by elementary torch operations, else by the library's calls.
"""
import math
import random

import torch

own = False


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a serving batch: every request appends one token
        dict(name="tables_decode", op="tables", R=256, page=64, new=1, cached=32768, cap=256, lens=11),
        # admission of prompts of mixed lengths in small pages, token rows padded to a fixed capacity
        dict(name="tables_prefill", op="tables", R=36, page=16, new=2048, cached=8192, cap=32768, lens=12),
        # the new token of each of 64 requests, K and V sliced out of a fused projection
        dict(name="append_decode", op="append", R=64, Hq=32, Hkv=8, d=128, page=64, new=1, cached=4096, cap=64,
             dtype="bf16", fused=True, lens=21),
        # ragged prompts written to small pages
        dict(name="append_prefill", op="append", R=24, Hq=32, Hkv=8, d=128, page=16, new=2048, cached=2048, cap=20000,
             dtype="bf16", fused=True, lens=22),
        # the smallest step: one request, one token
        dict(name="decode_one", op="attn", R=1, Hq=32, Hkv=8, d=128, page=64, new=1, cached=4131, fixed=True, cap=1,
             window=0, sinks=0, dtype="bf16", lens=31),
        # the 32k decode shape, a dense layer
        dict(name="decode_32k", op="attn", R=8, Hq=32, Hkv=8, d=128, page=64, new=1, cached=32767, fixed=True, cap=8,
             window=0, sinks=0, dtype="bf16", lens=32),
        # a serving batch: contexts from one token to 16k, small pages, two padded rows
        dict(name="decode_ragged", op="attn", R=62, Hq=64, Hkv=8, d=128, page=16, new=1, cached=16384, cap=64,
             window=0, sinks=0, dtype="bf16", lens=33),
        # the last 2048 tokens of a 32k prompt in the prefill shape
        dict(name="chunk_32k", op="attn", R=1, Hq=64, Hkv=4, d=128, page=64, new=2048, cached=30720, fixed=True, cap=2048,
             window=0, sinks=0, dtype="bf16", lens=34),
        # chunked prefill mixed with decodes in one batch
        dict(name="chunk_mixed", op="attn", R=16, Hq=32, Hkv=8, d=128, page=32, new=1024, cached=8192, cap=5000,
             window=0, sinks=0, dtype="bf16", lens=35),
        # sliding-window layer with sinks, chunks of four prompts
        dict(name="window_chunk", op="attn", R=4, Hq=32, Hkv=8, d=128, page=64, new=2048, cached=14336, fixed=True,
             cap=8192, window=512, sinks=4, dtype="bf16", lens=36),
        # the same kind of layer in a decode step of long contexts
        dict(name="window_decode", op="attn", R=32, Hq=64, Hkv=8, d=128, page=64, new=1, cached=32768, cap=32,
             window=1024, sinks=16, dtype="bf16", lens=37),
        # float32, d = 64: the parity configuration's type and head size
        dict(name="chunk_f32", op="attn", R=3, Hq=8, Hkv=2, d=64, page=16, new=512, cached=4096, cap=1200,
             window=0, sinks=0, dtype="f32", lens=369),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["tables", "append", "decode", "chunk", "chunk", "f32"])
    if kind == "tables":
        R = _log(rng, 1, 512)
        new = rng.choice([1, _log(rng, 1, 2048)])
        return dict(op="tables", R=R, page=page, new=new, cached=_log(rng, 1, 32768), cap=min(32768, R * new + rng.randrange(9)),
                    lens=lens)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    d = rng.choice([64, 128, 128])
    if kind == "append":
        R = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 1, 2048)])
        return dict(op="append", R=R, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, new=new, cached=_log(rng, 1, 2048),
                    cap=min(20000, R * new + rng.randrange(9)), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    fused=rng.random() < 0.5, lens=lens)
    window = rng.choice([0, 0, _log(rng, 64, 2048)])
    sinks = rng.choice([0, rng.randrange(1, 129)]) if window else 0
    if kind == "decode":
        cached = _log(rng, 1, 32768)
        R = _log(rng, 1, max(1, min(64, (1 << 18) // cached)))
        return dict(op="attn", R=R, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, new=1, cached=cached, cap=R + rng.randrange(3),
                    window=window, sinks=sinks, dtype="bf16", lens=lens)
    if kind == "chunk":
        cached, new = _log(rng, 1, 30720), _log(rng, 2, 2048)
        room = (1 << 30) // (Hkv * G * new * (cached + new))
        R = _log(rng, 1, max(1, min(32, room)))
        return dict(op="attn", R=R, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, new=new, cached=cached,
                    cap=R * new + rng.randrange(9), window=window, sinks=sinks, dtype="bf16", lens=lens)
    cached, new = _log(rng, 1, 4096), rng.choice([1, _log(rng, 2, 512)])
    return dict(op="attn", R=_log(rng, 1, 8), Hq=Hkv * G, Hkv=Hkv, d=d, page=page, new=new, cached=cached, cap=8 * new,
                window=window, sinks=sinks, dtype="f32", lens=lens)


def lengths(case):
    """(cached, new) token counts of each request: `fixed` cases take the case's own, the others are
    ragged, spread over the logarithm from nothing cached to the case's limits; the new tokens fit
    the case's token rows."""
    R, rng = case["R"], random.Random(case["lens"])
    if case.get("fixed"):
        return [case["cached"]] * R, [case["new"]] * R
    cached = [int(math.exp(rng.uniform(0, math.log(case["cached"] + 1)))) - (1 if i % 5 == 0 else 0) for i in range(R)]
    if case["new"] == 1:
        return cached, [1] * R
    new = [int(math.exp(rng.uniform(0, math.log(case["new"])))) if i % 3 else case["new"] for i in range(R)]
    room = case["cap"]
    for i in range(R):
        new[i] = min(new[i], room)
        room -= new[i]
    return cached, new


def _pages(case):
    """Pages of each request before and after its new tokens, and the width of the block table."""
    P = case["page"]
    cached, new = lengths(case)
    before = [-(-c // P) for c in cached]
    after = [-(-(c + n) // P) for c, n in zip(cached, new)]
    return before, after, max(1, max(after)) + 1


def work(case):
    P, R = case["page"], case["R"]
    cached, new = lengths(case)
    n = sum(new)
    before, after, _ = _pages(case)
    if case["op"] == "tables":
        taken = sum(after) - sum(before)
        # lengths, the pages taken and each request's open page; table entries, slots, sums, lengths
        return {"bytes": 4 * (2 * R + taken + R + taken + case["cap"] + 2 * R + 5), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "append":
        return {"bytes": 4 * n * Hkv * d * e + 4 * case["cap"], "flops": 0}
    keys = pairs = 0
    W, S = case["window"], case["sinks"]
    for c, m in zip(cached, new):
        if m == 0:
            continue
        seen = c + m
        if W:
            edge = max(0, c - W + 1)          # first key of the first row's window
            seen = c + m - edge + min(S, edge)
        keys += seen
        for t in range(c, c + m):
            lo = max(0, t - W + 1) if W else 0
            pairs += t + 1 - lo + min(S, lo)
    Hq = case["Hq"]
    return {"bytes": 2 * keys * Hkv * d * e + 2 * n * Hq * d * e + 4 * (sum(after) + 2 * R), "flops": 4 * d * Hq * pairs}


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    P, R, cap = case["page"], case["R"], case["cap"]
    cached, new = lengths(case)
    before, after, width = _pages(case)
    first, last = sum(before), sum(after)
    n_pages = last + 7
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=case, n_pages=n_pages, width=width, cached=torch.tensor(cached, **i32), new=torch.tensor(new, **i32))
    # pages are handed out in a random order; the free stack holds the ones no request owns yet
    if case["op"] == "tables":
        table = _table(order, before, width, R, dev)
        free = order[first:].contiguous()
        s.update(table=table, free=free, free_count=torch.tensor([free.numel()], **i32),
                 cu=torch.zeros(R + 1, **i32), kv_len=torch.zeros(R, **i32), slots=torch.zeros(cap, **i32),
                 counts=torch.zeros(4, **i32))
        return s
    table = _table(order, after, width, R, dev)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    s.update(table=table, k_cache=normal(n_pages, Hkv, P, d), v_cache=normal(n_pages, Hkv, P, d))
    if case["op"] == "append":
        if case["fused"]:
            qkv = normal(cap, Hq + 2 * Hkv, d)
            s.update(K=qkv[:, Hq:Hq + Hkv], V=qkv[:, Hq + Hkv:])
        else:
            s.update(K=normal(cap, Hkv, d), V=normal(cap, Hkv, d))
        slots = torch.full((cap,), -1, **i32)
        tab, at = table.cpu().tolist(), 0
        flat = [tab[r][t // P] * P + t % P for r in range(R) for t in range(cached[r], cached[r] + new[r])]
        slots[:len(flat)] = torch.tensor(flat, **i32)
        s.update(slots=slots)
        return s
    # keys of a trained model have channel means of their own per head
    s["k_cache"] += (0.5 * torch.randn((1, Hkv, 1, d), generator=g, device=dev)).to(dt)
    sums = [0]
    for m in new:
        sums.append(sums[-1] + m)
    s.update(Q=normal(cap, Hq, d), O=torch.zeros((cap, Hq, d), dtype=dt, device=dev), cu=torch.tensor(sums, **i32),
             kv_len=torch.tensor([c + m for c, m in zip(cached, new)], **i32))
    return s


def _table(order, pages, width, R, dev):
    table = torch.full((R, width), -1, dtype=torch.int32)
    ids, at = order.cpu(), 0
    for r, m in enumerate(pages):
        table[r, :m] = ids[at:at + m]
        at += m
    return table.to(dev)


# ----------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "tables":
        return _tables(s, case)
    if case["op"] == "append":
        return _append(s, case)
    return _attention(s, case)


def _own(s, case):
    from block_sparse_long_summary_b200 import cobs
    p = s.get("params")
    if p is None:   # what a program makes once: the problem statement and the workspace
        p = s["params"] = cobs.PagedParams(
            R=case["R"], Hq=case.get("Hq", 1), Hkv=case.get("Hkv", 1), d=case.get("d", 128), page=case["page"],
            n_pages=s["n_pages"], max_pages=s["width"], n_tokens=case["cap"], max_new=case["new"],
            window=case.get("window", 0), sinks=case.get("sinks", 0), dtype=case.get("dtype", "bf16"))
        if case["op"] == "attn":
            s["ws"] = cobs.alloc_paged_workspace(p)
    if case["op"] == "tables":
        cobs.cobs_paged_tables(p, s["cached"], s["new"], s["free"], s["free_count"], s["table"], s["cu"], s["kv_len"],
                               s["slots"], s["counts"])
        return s["table"], s["cu"], s["kv_len"], s["slots"], s["counts"]
    if case["op"] == "append":
        cobs.cobs_paged_append(p, s["K"], s["V"], s["slots"], s["k_cache"], s["v_cache"])
        return s["k_cache"], s["v_cache"]
    cobs.cobs_paged_attn(p, s["Q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], s["O"], None, s["ws"])
    return s["O"]


def _tables(s, case):
    P, cap = case["page"], case["cap"]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    R, width = table.shape
    dev = table.device
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    cu = torch.cat([zero, new.cumsum(0)])
    before = (cached + P - 1) // P
    after = (cached + new + P - 1) // P
    first = torch.cat([zero, (after - before).cumsum(0)])
    # entry (r, j) takes the page number first[r] + j - before[r] from the top of the stack
    j = torch.arange(width, device=dev)[None, :]
    k = first[:-1, None] + j - before[:, None]
    fresh = (j >= before[:, None]) & (j < after[:, None])
    at = s["free_count"].long() - 1 - k
    taken = torch.where(at >= 0, free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where(fresh, taken, table)
    # token rows: the request whose range holds the row, its position, its page
    t = torch.arange(cap, device=dev)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=R - 1)
    pos = cached[r] + t - cu[r]
    page = table[r, (pos // P).clamp(max=width - 1)].long()
    slots = torch.where((t < cu[-1]) & (page >= 0), page * P + pos % P, -1)
    need = first[-1:]
    have = s["free_count"].long()
    counts = torch.cat([cu[-1:], need, (have - need).clamp(min=0), (need - have).clamp(min=0)])
    i32 = torch.int32
    return table.to(i32), cu.to(i32), (cached + new).to(i32), slots.to(i32), counts.to(i32)


def _append(s, case):
    P = case["page"]
    slots = s["slots"].long()
    rows = (slots >= 0).nonzero()[:, 0]
    page, off = slots[rows] // P, slots[rows] % P
    s["k_cache"][page, :, off] = s["K"][rows]
    s["v_cache"][page, :, off] = s["V"][rows]
    return s["k_cache"], s["v_cache"]


def _attention(s, case):
    P, d, Hq, Hkv, W, S = case["page"], case["d"], case["Hq"], case["Hkv"], case["window"], case["sinks"]
    G, R, m = Hq // Hkv, case["R"], case["new"]
    Q, cu, kv_len = s["Q"], s["cu"].long(), s["kv_len"].long()
    dev = Q.device
    new = cu[1:] - cu[:-1]
    # every request's keys and values by position, padded to the width of the table
    ids = s["table"].long().clamp(min=0)
    T = ids.shape[1] * P

    def by_position(cache):
        return cache[ids].float().permute(0, 2, 1, 3, 4).reshape(R, Hkv, T, d)

    i = torch.arange(m, device=dev)
    rows = (cu[:-1, None] + i).clamp(max=Q.shape[0] - 1)
    q = Q[rows].float().reshape(R, m, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * m, d)
    x = q @ by_position(s["k_cache"]).transpose(2, 3)
    x *= 1.0 / math.sqrt(d)
    pos = (kv_len - new)[:, None] + i
    j = torch.arange(T, device=dev)
    seen = j <= pos[..., None]
    if W:
        seen &= (pos[..., None] - j < W) | (j < S)
    x = x.reshape(R, Hkv, G, m, T)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    x -= x.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    x = x.exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = x.reshape(R, Hkv, G * m, T) @ by_position(s["v_cache"])
    o = o.reshape(R, Hkv, G, m, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, m, Hq, d).to(Q.dtype)
    live = i < new[:, None]
    O = s["O"]
    O[rows[live]] = o[live]
    return O


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definitions in 64 bits, request by request and head by head."""
    if case["op"] == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    P = case["page"]
    cached, new = lengths(case)
    if case["op"] == "append":
        # every slot of the cache looks up the token row that fills it
        n_slots = s["n_pages"] * P
        source = torch.full((n_slots,), -1, dtype=torch.long)
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                source[slot] = t
        source = source.to(s["K"].device).reshape(-1, 1, P, 1)

        def filled(cache, rows):
            picked = rows.double()[source.clamp(min=0).flatten()].reshape(-1, P, *rows.shape[1:]).transpose(1, 2)
            return torch.where(source >= 0, picked, cache.double())

        return filled(s["k_cache"], s["K"]), filled(s["v_cache"], s["V"])
    Hq, Hkv, d, W, S = case["Hq"], case["Hkv"], case["d"], case["window"], case["sinks"]
    G = Hq // Hkv
    O = s["O"].double()
    at = 0
    for r in range(case["R"]):
        n, L = new[r], cached[r] + new[r]
        if n == 0:
            continue
        pages = s["table"][r, :-(-L // P)].long()
        t = torch.arange(cached[r], L, device=O.device)[:, None]
        j = torch.arange(L, device=O.device)[None, :]
        hidden = j > t
        if W:
            hidden |= (j <= t - W) & (j >= S)
        for h in range(Hkv):
            K = s["k_cache"][pages, h].double().reshape(-1, d)[:L]
            V = s["v_cache"][pages, h].double().reshape(-1, d)[:L]
            for a in range(h * G, (h + 1) * G):
                z = (s["Q"][at:at + n, a].double() @ K.T) / math.sqrt(d)
                z = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1)
                O[at:at + n, a] = z @ V
        at += n
    return O
