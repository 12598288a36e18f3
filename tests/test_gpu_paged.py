"""The paged-cache calls on the GPU: block tables and slot maps against a walk over every token,
the append against plain indexing (bit for bit), the attention against 64 bits."""
import dataclasses
import os
import random
import subprocess
import sys

import pytest
import torch

from paged_common import Batch, cobs, tables_reference

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- tables

def _tables(lens, page, n_free, n_tokens=None, max_pages=None, max_new=None, n_pages=None, seed=0, scratch_free=0):
    """Run the call and the walk on one batch; returns both tables' states."""
    C = cobs()
    rng = random.Random(seed)
    R = len(lens)
    cached, new = [c for c, _ in lens], [n for _, n in lens]
    width = max_pages or max(1, max(-(-max(0, c + n) // page) for c, n in lens))
    owned = sum(-(-max(0, c) // page) for c in cached)
    total = n_pages or owned + n_free + 2
    ids = list(range(total))
    rng.shuffle(ids)
    table = [[-1] * width for _ in range(R)]
    for r, c in enumerate(cached):
        for j in range(min(width, -(-max(0, c) // page))):
            table[r][j] = ids.pop()
    free = [ids.pop() for _ in range(n_free)]
    p = C.PagedParams(R=R, Hq=8, Hkv=2, d=128, page=page, n_pages=total, max_pages=width,
                      n_tokens=sum(new) + 5 if n_tokens is None else n_tokens, max_new=max_new or max(1, max(new)))
    buf = C.alloc_paged(p)
    buf.block_table.copy_(torch.tensor(table, dtype=torch.int32))
    stack = _i32(free + [-9] * scratch_free) if free or scratch_free else torch.empty(0, dtype=torch.int32, device="cuda")
    buf.slot_map.fill_(99)
    C.device_error(reset=True)
    C.cobs_paged_tables(p, _i32(cached), _i32(new), stack, _i32([len(free)]), buf.block_table, buf.cu_new, buf.kv_len,
                        buf.slot_map, buf.counts)
    torch.cuda.synchronize()
    want = tables_reference(p, cached, new, free, table)
    got = (buf.cu_new.tolist(), buf.kv_len.tolist(), buf.slot_map.tolist(), buf.counts.tolist())
    for g, w, name in zip(got, want, ("cu_new", "kv_len", "slot_map", "counts")):
        assert g == w, f"{name}: {g[:40]} against {w[:40]}"
    assert buf.block_table.tolist() == table
    return p, buf


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [
    [(0, 1)], [(1, 1)], [(15, 1), (16, 1), (17, 1)], [(0, 16), (0, 17), (0, 15)], [(0, 0), (5, 0), (0, 3), (7, 0)],
    [(127, 2), (128, 130), (0, 300), (1000, 1)],
])
def test_tables_small(page, lens):
    _tables(lens, page, n_free=40)
    assert cobs().device_error() == 0


@pytest.mark.parametrize("R,new,cached", [(1, 5000, 3000), (700, 1, 4000), (1500, 7, 300), (64, 900, 2000), (513, 0, 100)])
def test_tables_ragged(R, new, cached):
    rng = random.Random(R)
    lens = [(rng.randrange(cached + 1), rng.randrange(new + 1)) for _ in range(R)]
    need = sum(-(-(c + n) // 16) - -(-c // 16) for c, n in lens)
    _tables(lens, 16, n_free=need + 3, scratch_free=4)
    assert cobs().device_error() == 0


def test_tables_at_the_largest_request_count():
    lens = [((7 * r) % 90, r % 3) for r in range(16384)]
    _tables(lens, 32, n_free=16384)
    assert cobs().device_error() == 0


def test_tables_missing_pages_are_counted():
    p, buf = _tables([(10, 40), (0, 100), (16, 1)], 16, n_free=4)
    assert buf.counts.tolist()[3] > 0 and cobs().device_error() == 0
    _tables([(10, 40)], 16, n_free=0)


@pytest.mark.parametrize("lens,kw", [
    ([(3, 4), (-1, 2), (5, 6)], {}),                    # negative cached length
    ([(3, 4), (2, -3), (5, 6)], dict(n_tokens=15)),     # negative new length
    ([(3, 4), (60, 30), (5, 6)], dict(max_pages=4)),    # beyond the table's width
    ([(3, 4), (2, 9), (5, 6)], dict(max_new=8)),        # more than max_new
    ([(3, 4), (2, 9), (5, 6)], dict(n_tokens=10)),      # more tokens than rows: cut off
])
def test_tables_bad_lengths_are_left_out_and_recorded(lens, kw):
    _tables(lens, 16, n_free=20, **kw)
    assert cobs().device_error(reset=True) == 3


def test_tables_bad_free_pages_are_recorded():
    C = cobs()
    p = C.PagedParams(R=1, Hq=1, Hkv=1, d=64, page=16, n_pages=4, max_pages=4, n_tokens=40, max_new=40)
    buf = C.alloc_paged(p)
    C.device_error(reset=True)
    C.cobs_paged_tables(p, _i32([0]), _i32([40]), _i32([2, 9, 1]), _i32([3]), buf.block_table, buf.cu_new, buf.kv_len,
                        buf.slot_map, buf.counts)
    assert C.device_error(reset=True) == 1
    assert buf.block_table.tolist() == [[1, -1, 2, -1]]
    assert buf.slot_map.tolist() == list(range(16, 32)) + [-1] * 16 + list(range(32, 40))
    # a count beyond the array is cut to it
    C.cobs_paged_tables(p, _i32([0]), _i32([40]), _i32([2, 3, 1]), _i32([1000]), buf.block_table, buf.cu_new, buf.kv_len,
                        buf.slot_map, buf.counts)
    assert buf.counts.tolist() == [40, 3, 0, 0] and C.device_error() == 0


def test_tables_no_token_rows():
    C = cobs()
    p = C.PagedParams(R=2, Hq=1, Hkv=1, d=64, page=16, n_pages=4, max_pages=4, n_tokens=0, max_new=1)
    buf = C.alloc_paged(p)
    C.device_error(reset=True)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    C.cobs_paged_tables(p, _i32([3, 17]), _i32([0, 0]), e, _i32([0]), buf.block_table, buf.cu_new, buf.kv_len, buf.slot_map,
                        buf.counts)
    assert buf.cu_new.tolist() == [0, 0, 0] and buf.kv_len.tolist() == [3, 17] and buf.counts.tolist() == [0, 0, 0, 0]
    q = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    C.cobs_paged_append(p, q, q, buf.slot_map, c, c)
    C.cobs_paged_attn(p, q, c, c, buf.block_table, buf.cu_new, buf.kv_len, buf.O, None, buf.ws)
    assert C.device_error() == 0


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,d,page,n,fused", [(1, 64, 16, 1, False), (8, 128, 64, 65, True), (3, 128, 32, 700, True),
                                                (2, 64, 128, 5000, False)])
def test_append_copies_rows_bit_for_bit(dtype, Hkv, d, page, n, fused):
    C = cobs()
    g = torch.Generator(device="cuda").manual_seed(n)
    n_pages = n // page + 3
    p = C.PagedParams(R=1, Hq=2 * Hkv, Hkv=Hkv, d=d, page=page, n_pages=n_pages, max_pages=n_pages, n_tokens=n, max_new=n,
                      dtype=dtype)
    wide = torch.randn((n, 4 * Hkv, d), generator=g, device="cuda").to(p.torch_dtype)
    K, V = (wide[:, 2 * Hkv:3 * Hkv], wide[:, 3 * Hkv:]) if fused else (wide[:, :Hkv].contiguous(), wide[:, Hkv:2 * Hkv].contiguous())
    kc = torch.randn((n_pages, Hkv, page, d), generator=g, device="cuda").to(p.torch_dtype)
    vc = torch.randn((n_pages, Hkv, page, d), generator=g, device="cuda").to(p.torch_dtype)
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    slots[n // 2] = -1
    wk, wv = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            wk[s // page, :, s % page] = K[t]
            wv[s // page, :, s % page] = V[t]
    C.device_error(reset=True)
    C.cobs_paged_append(p, K, V, slots, kc, vc)
    assert C.device_error() == 0
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    slots[0] = n_pages * page   # outside the cache: skipped and recorded
    C.cobs_paged_append(p, K, V, slots, kc, vc)
    assert C.device_error(reset=True) == 1
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


# ----------------------------------------------------------------------------- attention

def _check(lens, Hq, Hkv, d, page, **kw):
    C = cobs()
    C.device_error(reset=True)
    b = Batch(C, lens, Hq, Hkv, d, page, **kw)
    b.run()
    assert C.device_error() == 0
    b.check()
    return b


DTYPES = ["bf16", "f32"]
ONE = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (63, 1), (64, 1), (127, 1), (128, 1), (129, 1), (700, 1), (2047, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(dtype, d, page):
    _check(ONE, 8, 2, d, page, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 11, 16])
def test_group_sizes(dtype, G):
    _check([(300, 1), (77, 1)], 2 * G, 2, 128, 32, dtype=dtype, seed=G)
    _check([(300, 70), (0, 33), (77, 1)], 2 * G, 2, 128, 32, dtype=dtype, seed=G, fused=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new", [(1, 1), (3, 1), (7, 1), (9, 1), (3, 5), (7, 40)])
def test_odd_groups_with_units_cut_at_both_ends_of_a_range(dtype, d, G, new):
    # more units than workers, of unequal lengths: ranges begin and end inside units, so that workers leave two records
    rng = random.Random(100 * G + new)
    _check([(rng.randrange(1, 1500), 1 + rng.randrange(new)) for _ in range(64)], 3 * G, 3, d, 32, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("lens", [
    [(0, 2)], [(0, 128)], [(0, 129), (1, 127)], [(100, 300), (5, 0), (0, 17), (513, 2), (0, 1)], [(2000, 200)],
])
def test_chunks(dtype, d, page, lens):
    _check(lens, 8, 2, d, page, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (100, 130), (512, 4), (128, 128), (4096, 7)])
def test_window_and_sinks(dtype, window, sinks):
    _check(ONE, 8, 2, 128, 16, dtype=dtype, window=window, sinks=sinks)
    _check([(900, 130), (0, 300), (64, 65), (3, 2)], 8, 2, 128, 64, dtype=dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_longest_windows_are_no_windows(dtype):
    top = 2 ** 31 - 1
    for window, sinks in ((top, 0), (top, top), (2 ** 30 + 1, 5), (7, top)):
        _check([(500, 1), (3, 1), (-1, 1)], 4, 2, 64, 16, dtype=dtype, window=window, sinks=sinks)
        _check([(500, 40), (-3, 5), (-40, 41), (-200, 300)], 4, 2, 64, 16, dtype=dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_context_with_few_rows_is_split(dtype):
    _check([(40000, 1)], 4, 1, 128, 64, dtype=dtype)
    _check([(30000, 40)], 4, 1, 64, 16, dtype=dtype)
    _check([(30000, 40), (9, 1), (20000, 1)], 8, 2, 128, 32, dtype=dtype, window=9000, sinks=5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_requests(dtype):
    rng = random.Random(5)
    _check([(int(2 ** rng.uniform(0, 11)), 1) for _ in range(300)], 4, 1, 64, 16, dtype=dtype)
    _check([(int(2 ** rng.uniform(0, 9)), rng.choice([0, 1, 1, 1, 5, 60])) for _ in range(600)], 2, 1, 64, 16, dtype=dtype)


@pytest.mark.parametrize("new", [1, 3])
def test_attention_at_the_largest_request_count(new):
    rng = random.Random(3)
    _check([(rng.randrange(40), rng.randrange(1, new + 1)) for _ in range(16384)], 1, 1, 64, 16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores_keep_the_running_maximum(dtype):
    _check([(3000, 3), (500, 200)], 4, 2, 128, 64, dtype=dtype, scale=4.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_fewer_keys_than_new_tokens_leaves_empty_rows(dtype):
    """kv_len < new tokens: the first rows stand before position 0 and see nothing."""
    _check([(-3, 5), (-7, 7), (20, 3)], 8, 2, 128, 16, dtype=dtype)
    _check([(-1, 1), (9, 1)], 8, 2, 128, 16, dtype=dtype)
    _check([(-200, 300), (9, 1)], 8, 2, 64, 16, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_touch_only_the_rows_that_see_them(dtype, value):
    C = cobs()
    for lens, W, S in ([(100, 60), (0, 200)], 0, 0), ([(100, 160)], 20, 3):
        b = Batch(C, lens, 8, 2, 128, 16, dtype=dtype, window=W, sinks=S, drop_unseen=False)
        for r, t in ((0, 110), (0, 150), (len(lens) - 1, 5)):
            b.V[r][:, t, ::7] = value
            b.v_cache[b.table[r, t // 16].item(), :, t % 16] = b.V[r][:, t].to(b.v_cache.device)
        C.device_error(reset=True)
        b.run()
        assert C.device_error() == 0
        b.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinite_scores(dtype):
    """Keys of -inf score count nothing, a row of nothing else is NaN, as is one with a +inf score."""
    C = cobs()
    b = Batch(C, [(60, 4), (130, 1), (3, 1)], 4, 2, 64, 16, dtype=dtype)
    b.Q.copy_(b.Q.abs())
    for r, t, v in ((0, 5, float("-inf")), (0, 61, float("inf")), (1, 130, float("-inf")), (2, 0, float("-inf")),
                    (2, 1, float("-inf")), (2, 2, float("-inf")), (2, 3, float("-inf"))):
        b.K[r][:, t] = v
        b.k_cache[b.table[r, t // 16].item(), :, t % 16] = v
    b.run()
    torch.cuda.synchronize()
    n = [torch.isnan(b.O[i].float()).all().item() for i in range(6)]
    assert n == [False, True, True, True, False, True], n
    assert torch.isfinite(b.O[0].float()).all() and torch.isfinite(b.O[4].float()).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_pages_count_as_zeros_and_are_recorded(dtype):
    C = cobs()
    for lens in ([(200, 1), (90, 1)], [(200, 30), (90, 1)]):
        b = Batch(C, lens, 4, 2, 128, 32, dtype=dtype)
        for page, j in ((-1, 1), (b.p.n_pages, 3)):
            b.table[0, j] = page
            b.K[0][:, 32 * j:32 * (j + 1)] = 0
            b.V[0][:, 32 * j:32 * (j + 1)] = 0
        C.device_error(reset=True)
        b.run()
        assert C.device_error(reset=True) == 1
        b.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_bad_lengths_leave_the_request_out(dtype):
    C = cobs()
    for what in ("long", "short", "rows", "order", "new"):
        b = Batch(C, [(40, 5), (60, 4), (9, 3)], 4, 2, 64, 16, dtype=dtype, max_new=5 if what != "new" else 4)
        whole = b.reference()
        if what == "long":
            b.kv_len[1] = b.p.max_pages * 16 + 1
        elif what == "short":
            b.kv_len[1] = -1
        elif what == "rows":
            b.cu[3] = b.p.n_tokens + 1
        elif what == "order":
            b.cu[2] = 4
        C.device_error(reset=True)
        b.run()
        assert C.device_error(reset=True) == 3
        kept = {"long": [0, 2], "short": [0, 2], "rows": [0, 1], "order": [0], "new": [1, 2]}[what]
        rows = {0: range(0, 5), 1: range(5, 9), 2: range(9, 12)}
        if what == "order":   # request 2 then starts at row 4 with 8 tokens: more than max_new
            kept = [0]
        for r in range(3):
            for i in rows[r]:
                if r in kept:
                    assert ((b.O[i].double() - whole[0][i]).abs() <= whole[2][i]).all(), (what, r, i)
                else:
                    assert (b.O[i] == 7).all(), (what, r, i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[(5000, 1), (70, 1)], [(900, 90), (70, 1), (0, 200)]])
def test_repeated_calls_agree_bit_for_bit_and_replay_from_a_graph(dtype, lens):
    C = cobs()
    a, b = (Batch(C, lens, 8, 2, 128, 64, dtype=dtype, seed=s) for s in (1, 2))
    b.ws = a.ws   # one workspace, calls in order
    a.run(); b.run()
    want = [x.O.clone() for x in (a, b)]
    for x in (a, b, a):
        x.O.fill_(7.0)
        x.run()
    assert torch.equal(a.O, want[0]) and torch.equal(b.O, want[1])
    s = torch.cuda.Stream()
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.run()
        graphs.append(g)
    for _ in range(3):
        for x in (a, b):
            x.O.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.O, want[0]) and torch.equal(b.O, want[1])
    # the same graph with other lengths: the last request shrinks by a few keys
    a.lens = [(c - 3, n) if i == 0 else (c, n) for i, (c, n) in enumerate(lens)]
    a.kv_len[0] -= 3
    a.K[0], a.V[0] = a.K[0][:, :-3], a.V[0][:, :-3]
    graphs[0].replay()
    a.check()
    assert C.device_error() == 0


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from paged_common import Batch, cobs
C = cobs()
b = Batch(C, [(300, {n}), (77, 1)], 8, 2, 128, 16, dtype={dtype!r}, max_new={n})
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    b.run()
g.replay()
b.check()
assert C.device_error() == 0
"""


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 40), ("f32", 1), ("f32", 40)])
def test_the_first_call_of_a_process_may_be_a_captured_one(dtype, n):
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests, dtype=dtype, n=n)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("lens", [[(2000, 1), (70, 1)], [(900, 90), (70, 1), (0, 200)]])
def test_two_streams_at_once(lens):
    """Calls with workspaces of their own may overlap."""
    C = cobs()
    bs = [Batch(C, lens, 8, 2, 128, 64, seed=s) for s in range(4)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(bs, streams):
            b.run(stream=s)
    for b in bs:
        b.check()
    assert C.device_error() == 0


def test_side_stream_and_no_lse():
    C = cobs()
    b = Batch(C, [(300, 20), (1000, 1)], 8, 2, 128, 16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.run(lse=False, stream=s)
    s.synchronize()
    b.check(lse=False)
    assert (b.lse == 7).all()


def test_binding_checks_tensors():
    C = cobs()
    b = Batch(C, [(30, 4), (5, 1)], 4, 2, 64, 16, junk=0.0)
    p = b.p
    wide = torch.zeros((p.n_tokens, 8, 64), dtype=torch.bfloat16, device="cuda")

    def attn(**kw):
        t = dict(Q=b.Q, k_cache=b.k_cache, v_cache=b.v_cache, block_table=b.table, cu_new=b.cu, kv_len=b.kv_len, O=b.O, lse=None,
                 workspace=b.ws)
        t.update(kw)
        C.cobs_paged_attn(p, *t.values())

    attn()
    attn(Q=wide[:, :4])
    for bad, why in ((dict(Q=wide[:, ::2]), "contiguous"), (dict(Q=wide[:-1, :4]), "must be"), (dict(Q=b.Q.float()), "bfloat16"),
                     (dict(Q=wide[:1, :4].expand(p.n_tokens, 4, 64)), "overlap"), (dict(Q=wide.transpose(0, 1)[:4].transpose(0, 1)[:, :, ::1].cpu()), "CUDA"),
                     (dict(Q=torch.zeros((p.n_tokens, 4, 128), dtype=torch.bfloat16, device="cuda")[:, :, ::2]), "contiguous"),
                     (dict(k_cache=b.k_cache[:-1]), "elements"), (dict(v_cache=b.v_cache.transpose(0, 1)), "contiguous"),
                     (dict(block_table=b.table.long()), "int32"), (dict(cu_new=b.cu[:-1]), "elements"), (dict(O=b.O[:, :2]), "contiguous"),
                     (dict(lse=torch.zeros(3, device="cuda")), "elements"), (dict(workspace=b.ws.float()), "uint8"),
                     (dict(kv_len=b.kv_len.cpu()), "CUDA")):
        with pytest.raises(ValueError, match=why):
            attn(**bad)
    with pytest.raises(C.CobsError, match="workspace"):
        attn(workspace=b.ws[:1024])
    with pytest.raises(AttributeError):
        C.cobs_paged_append(p, wide[:, :2], wide[:, 2:4], torch.full((p.n_tokens,), -1, dtype=torch.int32, device="cuda"), b.k_cache,
                            b.v_cache, stream=5)
    with pytest.raises(ValueError, match="stride"):
        C.cobs_paged_append(p, wide[:, :2], wide[:, 2:4].contiguous(), torch.full((p.n_tokens,), -1, dtype=torch.int32, device="cuda"),
                            b.k_cache, b.v_cache)


def test_steps_of_a_serving_loop():
    """Three requests live through prompt chunks and single tokens; each step's tables, append and
    attention run as one paged_step, checked against a contiguous history."""
    C = cobs()
    Hq, Hkv, d, page = 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    p = C.PagedParams(R=3, Hq=Hq, Hkv=Hkv, d=d, page=page, n_pages=64, max_pages=20, n_tokens=200, max_new=120, window=0)
    kc = torch.full((64, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    buf = C.alloc_paged(p)
    stack = torch.randperm(64, generator=g, device="cuda").to(torch.int32)
    free = _i32([64])
    hist = [(torch.empty((0, Hkv, d), device="cuda"), torch.empty((0, Hkv, d), device="cuda")) for _ in range(3)]
    C.device_error(reset=True)
    cached = [0, 0, 0]
    for step, new in enumerate([[120, 7, 0], [60, 1, 40], [1, 1, 1], [1, 0, 1], [1, 1, 1], [0, 33, 1]]):
        q = dataclasses.replace(p, max_new=max(1, max(new)))
        rows = torch.randn((200, Hq + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        C.paged_step(q, rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], _i32(cached), _i32(new), stack, free, kc, vc, buf)
        free = buf.counts[2:3].clone()
        assert C.device_error() == 0 and buf.counts[3].item() == 0
        at = 0
        for r, n in enumerate(new):
            K = torch.cat([hist[r][0], rows[at:at + n, Hq:Hq + Hkv].float()])
            V = torch.cat([hist[r][1], rows[at:at + n, Hq + Hkv:].float()])
            hist[r] = (K, V)
            for i in range(n):
                t = cached[r] + i + 1
                k, v = (x[:t].double().repeat_interleave(Hq // Hkv, dim=1) for x in (K, V))
                w = torch.softmax(torch.einsum("hd,thd->ht", rows[at + i, :Hq].double(), k) / d ** 0.5, dim=-1)
                o, A = torch.einsum("ht,thd->hd", w, v), torch.einsum("ht,thd->hd", w, v.abs())
                # two roundings to bf16 (p and o) and float32 sums, as in the single-call tests
                tol = 2.0 ** -8 * o.abs() + A * (2.0 ** -8 * 1.01 + 1e-4)
                assert ((buf.O[at + i].double() - o).abs() <= tol).all(), (step, r, i)
            at += n
        cached = [c + n for c, n in zip(cached, new)]


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements per tensor, its last pages in use."""
    C = cobs()
    Hkv, d, page, n_pages = 8, 128, 128, 17000   # 2.2e9 elements, 4.5 GB each
    kc = torch.zeros((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    p = C.PagedParams(R=2, Hq=16, Hkv=Hkv, d=d, page=page, n_pages=n_pages, max_pages=3, n_tokens=200, max_new=150)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((200, 16 + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    buf = C.alloc_paged(p)
    buf.block_table[0] = _i32([16990, 16999, 5])
    buf.block_table[1] = _i32([3, 16998, -1])
    C.device_error(reset=True)
    for new in ([150, 50], [1, 1]):
        q = dataclasses.replace(p, max_new=max(new), n_tokens=sum(new))
        b = C.alloc_paged(q)
        b.block_table.copy_(buf.block_table)
        cached = [0, 0] if new[0] > 1 else [150, 50]
        x = rows[:sum(new)]
        # the tables exist already: only the slots are wanted, no page is taken
        slots = [[16990, 16999, 5][t // 128] * 128 + t % 128 for t in range(cached[0], cached[0] + new[0])]
        slots += [[3, 16998][t // 128] * 128 + t % 128 for t in range(cached[1], cached[1] + new[1])]
        C.cobs_paged_append(q, x[:, 16:24], x[:, 24:], _i32(slots), kc, vc)
        C.cobs_paged_attn(q, x[:, :16], kc, vc, b.block_table, _i32([0, new[0], sum(new)]),
                          _i32([c + n for c, n in zip(cached, new)]), b.O, None, b.ws)
        assert C.device_error() == 0
        for i, (r, t) in enumerate([(0, cached[0] + k) for k in range(new[0])] + [(1, cached[1] + k) for k in range(new[1])]):
            if i % 37 and i != sum(new) - 1:
                continue
            pages = b.block_table[r].long()[:-(-(t + 1) // 128)]
            k, v = (c[pages].transpose(1, 2).reshape(-1, Hkv, d)[:t + 1].double().repeat_interleave(2, dim=1) for c in (kc, vc))
            w = torch.softmax(torch.einsum("hd,thd->ht", x[i, :16].double(), k) / d ** 0.5, dim=-1)
            o, A = torch.einsum("ht,thd->hd", w, v), torch.einsum("ht,thd->hd", w, v.abs())
            tol = 2.0 ** -8 * o.abs() + A * (2.0 ** -8 * 1.01 + 1e-4)
            assert ((b.O[i].double() - o).abs() <= tol).all(), (new, i)
