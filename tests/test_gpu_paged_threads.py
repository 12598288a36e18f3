"""Host threads that make paged calls at the same time, with different numbers of requests."""
import ctypes
import threading

import pytest
import torch

from paged_common import cobs

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _at_once(calls, rounds):
    """Each of `calls` (a function that returns a status) `rounds` times on a thread of its own; the statuses."""
    torch.cuda.synchronize()
    got, gate = [set() for _ in calls], threading.Barrier(len(calls))

    def loop(k):
        gate.wait()
        for _ in range(rounds):
            got[k].add(calls[k]())

    threads = [threading.Thread(target=loop, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return got


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def test_tables_of_different_request_counts():
    C = cobs()
    calls, keep = [], []
    for R in (5000, 16384, 6000, 16384):   # all need more shared memory than a kernel has unasked
        p = C.PagedParams(R=R, Hq=1, Hkv=1, d=64, page=16, n_pages=R, max_pages=1, n_tokens=R, max_new=1)
        buf = C.alloc_paged(p)
        lens, one, free = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.ones(R, dtype=torch.int32, device="cuda"), \
            torch.arange(R, dtype=torch.int32, device="cuda")
        count, cp, stream = _i32(R), p.c(), torch.cuda.Stream()
        keep.append((buf, lens, one, free, count, cp, stream, R))
        calls.append(lambda cp=cp, a=(lens, one, free), R=R, b=(count, buf.block_table, buf.cu_new, buf.kv_len, buf.slot_map, buf.counts),
                     s=stream: C._lib.cobs_paged_tables(ctypes.byref(cp), *map(_ptr, a), R, *map(_ptr, b), ctypes.c_void_p(s.cuda_stream)))
    assert _at_once(calls, 30000) == [{0}] * 4, C._lib.cobs_last_error()
    for buf, *_, R in keep:
        assert torch.equal(buf.cu_new, torch.arange(R + 1, dtype=torch.int32, device="cuda"))
        assert buf.counts.tolist() == [R, R, 0, 0]
    assert C.device_error() == 0


def test_float32_chunks_of_different_request_counts():
    C = cobs()
    calls, keep = [], []
    for R in (3, 16384, 3, 16384):
        p = C.PagedParams(R=R, Hq=1, Hkv=1, d=64, page=16, n_pages=1, max_pages=1, n_tokens=2, max_new=2, dtype="f32")
        q, kv = torch.randn((2, 1, 64), device="cuda"), torch.zeros((1, 1, 16, 64), device="cuda")
        kv[0, 0, 0] = 3.0
        buf = C.alloc_paged(p)
        buf.block_table[0] = 0
        buf.cu_new[1:] = 2
        buf.kv_len[0] = 2
        cp, stream = p.c(), torch.cuda.Stream()
        keep.append((buf, q, kv, cp, stream))
        calls.append(lambda cp=cp, a=(q, kv, kv, buf.block_table, buf.cu_new, buf.kv_len, buf.O), ws=buf.ws, s=stream:
                     C._lib.cobs_paged_attn(ctypes.byref(cp), *map(_ptr, a), None, _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream)))
    assert _at_once(calls, 30000) == [{0}] * 4, C._lib.cobs_last_error()
    for buf, *_ in keep:
        assert (buf.O[0] == 3.0).all() and torch.isfinite(buf.O).all()
    assert C.device_error() == 0
