"""Refusals of the paged-cache calls: all on the host, before anything is launched (no GPU needed),
and the tables' walk that the GPU tests compare with, on hand-made cases."""
import copy
import ctypes
import pickle

import pytest
import torch

from block_sparse_long_summary_b200 import build as B
from paged_common import tables_reference


@pytest.fixture(scope="module")
def lib():
    B.build()
    from block_sparse_long_summary_b200 import cobs
    return cobs


def _p(lib, **kw):
    base = dict(R=4, Hq=8, Hkv=2, d=128, page=64, n_pages=100, max_pages=10, n_tokens=16, max_new=4)
    base.update(kw)
    return lib.PagedParams(**base)


FAKE = [ctypes.c_void_p((k + 1) << 24) for k in range(12)]   # never read: validation fails first


def _attn(lib, cp, ptrs=None, ws=1 << 40):
    q = list(FAKE[:9]) if ptrs is None else ptrs
    return lib._lib.cobs_paged_attn(ctypes.byref(cp), *q[:9], ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), -1), (dict(R=16385), -2), (dict(Hq=0), -1), (dict(Hq=7), -1), (dict(Hq=34, Hkv=2), -2), (dict(d=96), -2),
    (dict(page=8), -2), (dict(page=48), -2), (dict(page=256), -2), (dict(n_pages=0), -1), (dict(max_pages=0), -1),
    (dict(n_tokens=-1), -1), (dict(max_new=0), -1), (dict(window=-1), -1), (dict(sinks=-1, window=4), -1),
    (dict(sinks=2), -1), (dict(n_pages=1 << 25), -2), (dict(max_pages=1 << 25), -2), (dict(n_tokens=1 << 28), -2),
    (dict(max_pages=(1 << 24) + 1), -2), (dict(Hq=1, Hkv=1, n_tokens=(1 << 30) + 1), -2),
    (dict(Hq=256, Hkv=256, max_pages=1 << 24), -2),
])
def test_bad_params_are_refused(lib, kw, status):
    p = _p(lib, **kw)
    cp = p.c()
    assert _attn(lib, cp) == status, lib._lib.cobs_last_error()
    assert lib._lib.cobs_paged_append(ctypes.byref(cp), *FAKE[:5], None) == status
    assert lib._lib.cobs_paged_tables(ctypes.byref(cp), FAKE[0], FAKE[1], FAKE[2], 4, *FAKE[3:9], None) == status
    assert lib.paged_workspace_bytes(p) == 0 and lib._lib.cobs_last_error() != b""


@pytest.mark.parametrize("q,kv", [(8 * 128 - 8, 0), (0, 100), (8 * 128 + 4, 0), (0, 2 * 128 + 1), (-1024, 0)])
def test_bad_strides_are_refused(lib, q, kv):
    assert _attn(lib, _p(lib).c(q, kv)) == -1
    assert b"stride" in lib._lib.cobs_last_error()


def test_bad_dtype_is_refused(lib):
    cp = lib.cobs_paged_params(4, 8, 2, 128, 64, 100, 10, 16, 4, 0, 0, 2, 0, 0)
    assert _attn(lib, cp) == -1
    with pytest.raises(ValueError, match="dtype"):
        _p(lib, dtype="f16").c()


@pytest.mark.parametrize("at,name", list(enumerate(["Q", "k_cache", "v_cache", "block_table", "cu_new", "kv_len", "O", None,
                                                    "workspace"])))
def test_null_and_misaligned_pointers_are_refused(lib, at, name):
    cp = _p(lib).c()
    if name is not None:
        assert _attn(lib, cp, FAKE[:at] + [None] + FAKE[at + 1:]) == -1
        assert name.encode() + b" is NULL" in lib._lib.cobs_last_error()
    assert _attn(lib, cp, FAKE[:at] + [ctypes.c_void_p(FAKE[at].value + 2)] + FAKE[at + 1:]) == -1
    assert b"aligned" in lib._lib.cobs_last_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_new", [1, 4, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_records_of_the_workspace_start_at_16_bytes(lib, dtype, max_new, d):
    def records(size, workers):  # bytes of both records of a worker: behind 32 bytes each, 256-byte aligned in all
        return (size - -(-32 * workers // 256) * 256) / workers

    # two heads: two rows of d + 2 floats in each of two records of one worker per SM
    two = lib.paged_workspace_bytes(_p(lib, Hq=2, Hkv=1, d=64, max_new=1))
    sms = next(n for n in range(1, 1024) if records(two, n) == 2 * 2 * 66 * 4)
    for G in range(1, 17):
        size = lib.paged_workspace_bytes(_p(lib, Hq=G, Hkv=1, d=d, max_new=max_new, dtype=dtype))
        both = [records(size, k * sms) for k in (1, 2, 3)]  # float32 chunks have two or three workers per SM
        assert any(b % (2 * 16) == 0 and b >= 2 * 4 * G * (d + 2) for b in both), (G, size, both)


def test_small_workspace_is_refused(lib):
    p = _p(lib)
    need = lib.paged_workspace_bytes(p)
    assert need > 0
    assert _attn(lib, p.c(), ws=need - 1) == -4
    assert b"workspace" in lib._lib.cobs_last_error()


@pytest.mark.parametrize("clash", [(0, 5), (1, 6), (2, 4), (3, 8), (2, 7)])
def test_tables_whose_inputs_overlap_outputs_are_refused(lib, clash):
    ptrs = [ctypes.c_void_p(f.value) for f in FAKE[:9]]   # 0..3 inputs, 4..8 outputs
    ptrs[clash[0]] = ctypes.c_void_p(ptrs[clash[1]].value + 4)
    cp = _p(lib).c()
    r = lib._lib.cobs_paged_tables(ctypes.byref(cp), ptrs[0], ptrs[1], ptrs[2], 4, ptrs[3], *ptrs[4:9], None)
    assert r == -1 and b"overlaps" in lib._lib.cobs_last_error()


def test_tables_pointers_are_checked(lib):
    cp = _p(lib).c()
    for at in range(9):
        ptrs = [None if k == at else f for k, f in enumerate(FAKE[:9])]
        r = lib._lib.cobs_paged_tables(ctypes.byref(cp), ptrs[0], ptrs[1], ptrs[2], 4, ptrs[3], *ptrs[4:9], None)
        assert r == -1 and b"NULL" in lib._lib.cobs_last_error()
    assert lib._lib.cobs_paged_tables(ctypes.byref(cp), FAKE[0], FAKE[1], FAKE[2], -1, *FAKE[3:9], None) == -1


def test_no_token_rows_needs_no_row_pointers(lib):
    cp = _p(lib, n_tokens=0).c()
    assert lib._lib.cobs_paged_append(ctypes.byref(cp), None, None, None, None, None, None) == 0
    assert _attn(lib, cp, [None] * 9, ws=0) == 0


def test_binding_refuses_host_tensors(lib):
    p = _p(lib)
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.cobs_paged_tables(p, z, z, z, z, z, z, z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        lib.cobs_paged_attn(p, z, z, z, z, z, z, z, None, z)
    with pytest.raises(TypeError, match="tensor"):
        lib.cobs_paged_append(p, z, z, z, None, z)


def test_params_of_the_binding(lib):
    import dataclasses
    p = _p(lib)
    c = p.c(5000, 3000)
    assert (c.R, c.n_tokens, c.dtype, c.q_stride, c.kv_stride) == (4, 16, lib.COBS_BF16, 5000, 3000)
    assert p.c().q_stride == 0   # the copy above has not changed the params
    q = dataclasses.replace(p, max_new=7)
    assert q.c().max_new == 7 and q.address != p.address and p.c().max_new == 4
    with pytest.raises(dataclasses.FrozenInstanceError):
        p.R = 5
    for other in (copy.deepcopy(p), copy.copy(p), pickle.loads(pickle.dumps(p))):
        assert other == p and other.address != p.address and bytes(other.c()) == bytes(p.c())


def test_tables_walk_by_hand(lib):
    p = _p(lib, R=3, page=16, max_pages=3, n_tokens=24, max_new=20, n_pages=9)
    table = [[4, -1, -1], [-1, -1, -1], [7, 2, -1]]
    out = tables_reference(p, [15, 0, 32], [2, 17, 0], [8, 6, 5, 3], table)
    assert table == [[4, 3, -1], [5, 6, -1], [7, 2, -1]]
    assert out[0] == [0, 2, 19, 19] and out[1] == [17, 17, 32] and out[3] == [19, 3, 1, 0]
    assert out[2] == [4 * 16 + 15, 3 * 16] + [5 * 16 + i for i in range(16)] + [6 * 16] + [-1] * 5
