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


STUB = """
extern int PyGILState_Check(void);
extern int unlocked(void) { return PyGILState_Check() ? -100 : -200; }
"""
CALLS = """
import importlib.util, sys, torch
sys.path.insert(0, {root!r})
from block_sparse_long_summary_b200 import cobs
spec = importlib.util.spec_from_file_location("_paged", {binding!r})
paged = importlib.util.module_from_spec(spec)
spec.loader.exec_module(paged)   # a second copy, which finds the stand-in beside itself
p = cobs.PagedParams(R=1, Hq=1, Hkv=1, d=64, page=16, n_pages=1, max_pages=1, n_tokens=1, max_new=1)
buf = cobs.alloc_paged(p)
i = torch.zeros(1, dtype=torch.int32, device="cuda")
kv, row = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
print(paged.tables(p.address, i, i, i, i, buf.block_table, buf.cu_new, buf.kv_len, buf.slot_map, buf.counts, None),
      paged.append(p.address, row, row, buf.slot_map, kv, kv, None),
      paged.attn(p.address, row, kv, kv, buf.block_table, buf.cu_new, buf.kv_len, buf.O, None, buf.ws, None))
"""


def test_the_library_runs_without_the_interpreter_lock(tmp_path):
    """The binding beside a stand-in for the library that tells whether its caller holds the lock. (The package's
    own library is loaded by its path and keeps its symbols to itself.)"""
    import os
    import shutil
    import subprocess
    import sys

    from block_sparse_long_summary_b200 import build as B
    cobs()
    source = STUB + "".join(f"int {f}(void) {{ return unlocked(); }}\n" for f in ("cobs_paged_tables", "cobs_paged_append", "cobs_paged_attn"))
    (tmp_path / "stub.c").write_text(source)
    subprocess.run([os.environ.get("CC", "gcc"), "-shared", "-fPIC", "-w", str(tmp_path / "stub.c"), "-o", str(tmp_path / "libcobs.so")], check=True)
    binding = shutil.copy(B.binding_path(), tmp_path / "_paged.so")
    r = subprocess.run([sys.executable, "-c", CALLS.format(root=B.ROOT, binding=str(binding))], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["-200"] * 3, r.stdout
