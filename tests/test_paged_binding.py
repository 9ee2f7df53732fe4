"""The binding's compiled module next to Python: errors of Python objects, and other threads while a call is in the library."""
import ctypes as C
import os
import subprocess
import threading
import time

import pytest
import torch

PARAM = 5


class NoTruth:
    def __bool__(self):
        raise ValueError("neither true nor false")


@pytest.fixture(scope="module")
def m():
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    from speculative_decoding_logit_gb300 import _binding
    return _binding


def test_interleaved_without_a_truth_value_is_refused(m):
    """Before anything else is looked at."""
    x = torch.zeros(1)
    with pytest.raises(m.AsvError) as e:
        m._paged_ext().paged_kv_append(x, x, x, x, x, x, x, None, None, NoTruth(), None, x, 0)
    assert e.value.status == PARAM


def _small_call():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c, q = torch.zeros(2, 16, 2, 64, **bf), torch.zeros(1, 4, 64, **bf)
    return c, q, torch.zeros(1, 1, **i32), torch.zeros(1, **i32), torch.tensor([0, 1], **i32)


@pytest.mark.gpu
def test_interleaved_of_a_whole_call(m):
    c, q, table, length, indptr = _small_call()
    rot = torch.zeros(4, 64, device="cuda")
    before = c.clone()
    c2 = c.clone()
    with pytest.raises(m.AsvError) as e:
        m.paged_kv_append(q[:, :2] + 1, q[:, :2] + 1, c, c2, table, length, indptr, rotary=rot, interleaved=NoTruth())
    assert e.value.status == PARAM and torch.equal(c, before) and torch.equal(c2, before)
    m.paged_kv_append(q[:, :2], q[:, :2], c, c2, table, length, indptr, rotary=rot, interleaved=1)


SLOW = """
#include <unistd.h>
extern "C" int slow() { usleep(300000); return 0; }
"""


@pytest.mark.gpu
def test_other_threads_run_while_a_call_is_in_the_library(m, tmp_path):
    """A launch blocks when the stream's queue is full, and what drains it may need the interpreter (a host function in
    Python): a stand-in for the library that takes 0.3 s must not stop other threads."""
    src, lib = tmp_path / "slow.cpp", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    slow = C.cast(C.CDLL(str(lib)).slow, C.c_void_p).value
    L = m.library()
    rest = [C.cast(f, C.c_void_p).value for f in (L.asv_status_string, L.asv_last_cuda_error)]
    real = [C.cast(f, C.c_void_p).value for f in (L.paged_attention, L.paged_kv_append)]
    c, q, table, length, indptr = _small_call()
    count, stop = [0], threading.Event()

    def other():
        while not stop.is_set():
            count[0] += 1
            time.sleep(0.001)

    calls = [lambda: m.paged_attention(q, c, c, table, length, indptr),
             lambda: m.paged_kv_append(q[:, :2], q[:, :2], c, c, table, length, indptr)]
    for call in calls:   # workspaces and kernels are there
        call()
    torch.cuda.synchronize()
    thread = threading.Thread(target=other)
    m._paged_ext().bind(m.AsvError, slow, slow, *rest)
    try:
        thread.start()
        for call in calls:
            before = count[0]
            call()
            assert count[0] - before > 20
    finally:
        m._paged_ext().bind(m.AsvError, *real, *rest)
        stop.set()
        thread.join()
