"""Inputs and 64-bit references of the paged-cache tests."""
import math
import random

import torch


def cobs():
    from block_sparse_long_summary_b200 import build as B
    B.build()
    from block_sparse_long_summary_b200 import cobs as C
    return C


def tables_reference(p, cached, new, free, table):
    """The tables of one step, by walking every token (plain Python; table is changed in place).
    Lengths that the call leaves out count as 0 and 0."""
    cu, kv_len, slots = [0], [], []
    need = 0
    for r, (c, n) in enumerate(zip(cached, new)):
        if c < 0 or n < 0 or n > p.max_new or c + n > p.max_pages * p.page:
            c = n = 0
        n = min(n, p.n_tokens - cu[-1])
        for t in range(c, c + n):
            if t % p.page == 0:
                need += 1
                table[r][t // p.page] = free[len(free) - need] if need <= len(free) else -1
            page = table[r][t // p.page]
            slots.append(page * p.page + t % p.page if page >= 0 else -1)
        cu.append(cu[-1] + n)
        kv_len.append(c + n)
    used = len(slots)
    slots += [-1] * (p.n_tokens - used)
    return cu, kv_len, slots, [used, need, max(0, len(free) - need), max(0, need - len(free))]


class Batch:
    """A ragged batch in a cache of shuffled pages. Every slot that no request owns holds `junk`,
    so do the pages of keys that no row of the batch sees (their table entries are -1) and the padded
    token rows; outputs start as a sentinel."""

    def __init__(self, C, lens, Hq, Hkv, d, page, dtype="bf16", window=0, sinks=0, pad=3, fused=False, junk=float("nan"),
                 seed=0, scale=1.0, device="cuda", drop_unseen=True, max_new=None):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        R = len(lens)
        self.lens = lens
        cached, new = [c for c, _ in lens], [n for _, n in lens]
        pages = [-(-max(0, c + n) // page) for c, n in lens]
        width = max(1, max(pages))
        n_pages = sum(pages) + 3
        ids = list(range(n_pages))
        rng.shuffle(ids)
        n_tok = sum(new) + pad
        self.p = p = C.PagedParams(R=R, Hq=Hq, Hkv=Hkv, d=d, page=page, n_pages=n_pages, max_pages=width, n_tokens=n_tok,
                                   max_new=max_new or max(1, max(new)), window=window, sinks=sinks, dtype=dtype)
        dt = p.torch_dtype
        self.k_cache = torch.full((n_pages, Hkv, page, d), junk, dtype=dt)
        self.v_cache = torch.full((n_pages, Hkv, page, d), junk, dtype=dt)
        table = torch.full((R, width), -1, dtype=torch.int32)
        self.K, self.V = [], []
        for r, (c, n) in enumerate(lens):
            L = max(0, c + n)
            K = (torch.randn((Hkv, L, d), generator=g) * scale).to(dt)
            V = torch.randn((Hkv, L, d), generator=g).to(dt)
            self.K.append(K)
            self.V.append(V)
            edge = max(0, max(0, c) - window + 1) if window and drop_unseen else 0
            for j in range(pages[r]):
                page_id = ids.pop()
                if n == 0 or (edge >= (j + 1) * page and min(sinks, edge) <= j * page):
                    continue   # no row sees this page: junk, no table entry
                table[r, j] = page_id
                lo, hi = j * page, min(L, (j + 1) * page)
                self.k_cache[page_id, :, :hi - lo] = K[:, lo:hi]
                self.v_cache[page_id, :, :hi - lo] = V[:, lo:hi]
                for t in range(lo, hi):
                    if window and drop_unseen and t < edge and t >= sinks:
                        self.k_cache[page_id, :, t - lo] = junk
                        self.v_cache[page_id, :, t - lo] = junk
        q = (torch.randn((n_tok, Hq, d), generator=g) * scale).to(dt)
        q[sum(new):] = junk
        if fused:
            wide = torch.full((n_tok, Hq + 2 * Hkv, d), junk, dtype=dt)
            wide[:, :Hq] = q
            self.Q = wide.to(device)[:, :Hq]
        else:
            self.Q = q.to(device)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        i32 = dict(dtype=torch.int32, device=device)
        self.cu, self.kv_len = torch.tensor(cu, **i32), torch.tensor([c + n for c, n in lens], **i32)
        self.table = table.to(device)
        self.k_cache, self.v_cache = self.k_cache.to(device), self.v_cache.to(device)
        self.O = torch.full((n_tok, Hq, d), 7.0, dtype=dt, device=device)
        self.lse = torch.full((n_tok, Hq), 7.0, device=device)
        self.ws = C.alloc_paged_workspace(p, device) if device != "cpu" else None
        self.C = C

    def run(self, lse=True, stream=None):
        self.C.cobs_paged_attn(self.p, self.Q, self.k_cache, self.v_cache, self.table, self.cu, self.kv_len, self.O,
                               self.lse if lse else None, self.ws, stream)

    def reference(self):
        """(o, lse, tolerance of o, tolerance of lse) in 64 bits; rows of padding keep the sentinel.

        Tolerances, from the arithmetic: scores are float32 sums of d products (at most d + 2
        roundings of 2^-24 of the sum of |q_c k_c|) and go through a scale and an exponential of
        about 2^-21 relative error, so p_j is off by at most ep = (d + 4) 2^-24 max_j sum |q k| / sqrt(d)
        + 2^-21. The sums over L keys in float32 add L 2^-24. With A = sum p |v| / sum p: the quotient
        is off by A (2 ep + 2 L 2^-24); bf16 rounds every p (2^-8 A, twice for its own second order)
        and the result (2^-8 |o|), float32 only the result (2^-24)."""
        p = self.p
        G, d = p.Hq // p.Hkv, p.d
        dev = self.Q.device
        O = torch.full((p.n_tokens, p.Hq, d), 7.0, dtype=torch.float64, device=dev)
        lse = torch.full((p.n_tokens, p.Hq), 7.0, dtype=torch.float64, device=dev)
        tolO, tolL = torch.zeros_like(O), torch.zeros_like(lse)
        at = 0
        for r, (c, n) in enumerate(self.lens):
            L = max(0, c + n)
            t = torch.arange(c, c + n, device=dev)[:, None]
            j = torch.arange(L, device=dev)[None, :]
            seen = j <= t
            if p.window:
                seen = seen & ((t - j < p.window) | (j < p.sinks))
            for h in range(p.Hkv):
                K, V = self.K[r][h].double().to(dev), self.V[r][h].double().to(dev)
                for a in range(h * G, (h + 1) * G):
                    q = self.Q[at:at + n, a].double()
                    if L == 0 or n == 0:
                        O[at:at + n, a], lse[at:at + n, a] = 0.0, -math.inf
                        continue
                    z = (q @ K.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                    l = torch.logsumexp(z, dim=-1)
                    w = torch.exp(z - torch.where(l > -math.inf, l, 0.0)[:, None])
                    # hidden keys do not enter, whatever they hold
                    Vs = torch.where(torch.isfinite(V), V, 0.0)
                    o = w @ Vs
                    for b in (~torch.isfinite(V)).nonzero()[:, 0].unique().tolist():
                        rows = seen[:, b]
                        o[rows] += w[rows, b:b + 1] * (V[b] - Vs[b])
                    A = w @ Vs.abs()
                    big = (q.abs() @ K.abs().T).masked_fill(~seen, 0.0).amax(dim=-1) / math.sqrt(d)
                    ep = (d + 4) * 2.0 ** -24 * big + 2.0 ** -21
                    acc = 2 * ep + 2 * L * 2.0 ** -24
                    half, pr = (2.0 ** -8, 2.0 ** -8 * (1 + 2.0 ** -7)) if p.dtype == "bf16" else (2.0 ** -24, 0.0)
                    O[at:at + n, a], lse[at:at + n, a] = o, l
                    tolO[at:at + n, a] = half * o.abs() + A * (pr + acc[:, None]) * (1 + half) + 1e-30
                    tolL[at:at + n, a] = ep + L * 2.0 ** -24 + 2.0 ** -22 * (l.abs() + 1)
            at += n
        return O, lse, tolO, tolL

    def check(self, what="", lse=True):
        torch.cuda.synchronize()
        O, L, tO, tL = self.reference()
        for got, ref, tol, name in ((self.O, O, tO, "o"), (self.lse, L, tL, "lse")):
            if name == "lse" and not lse:
                continue
            got = got.double()
            same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
            bad = ~same & ~((got - ref).abs() <= tol)
            if bad.any():
                at = bad.nonzero()[0].tolist()
                raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {got[tuple(at)].item()} "
                                     f"against {ref[tuple(at)].item()} (tolerance {tol[tuple(at)].item():.3g}); rows "
                                     f"{bad.nonzero()[:, 0].unique().tolist()[:20]}")
