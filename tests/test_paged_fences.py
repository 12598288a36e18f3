"""Order of tensor memory between threads in the kernel of bf16 chunks, by reading its source: a tcgen05 load of
columns that another thread stored, or that another thread has waited for, stands behind a barrier with
tcgen05.fence::before_thread_sync in front of it and tcgen05.fence::after_thread_sync behind it. (Without them
the results were right in every run; nothing made them so.)"""
import os
import re

from block_sparse_long_summary_b200 import build as B

MARKS = re.compile(r"rows_sync<|\bmeet\(\)|fence_before_sync|fence_after_sync|wait_warp|mbar_arrive|tc::st32|ld1\(|ld32_to\(")


def _marks(start, end):
    """The marks of the kernel's source between the first occurrence of `start` and the next of `end`."""
    with open(os.path.join(B.CSRC, "paged_chunk.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("paged_chunk_kernel(const"):]
    at = kernel.index(start)
    return MARKS.findall(kernel[at:kernel.index(end, at)])


def test_scores_of_the_other_half_are_read_behind_fences():
    marks = _marks("tc::st32(tS + c, s)", "ld1(tS + j)")   # from the scores' store in place to their reader
    barrier = marks.index("rows_sync<")
    assert "fence_before_sync" in marks[:barrier] and "fence_after_sync" in marks[barrier:], marks


def test_the_other_groups_accumulator_is_read_behind_fences():
    marks = _marks("wait_warp(&barO[g]", "tmem + lanes + kColO + 128 + c")
    meetings = [k for k, m in enumerate(marks) if m == "meet()"]
    assert len(meetings) >= 2
    waited, read = marks.index("wait_warp"), marks.index("ld32_to(")
    assert waited < meetings[0] and meetings[-1] < read
    assert "fence_before_sync" in marks[waited:meetings[0]], marks
    assert "fence_after_sync" in marks[meetings[-1]:read], marks
