"""The workspaces that the binding keeps for calls without one, without a GPU:
whose they are, and how long they are held."""
import contextlib
import threading

import pytest
import torch

import top_activation_sparse_b200 as qs
from top_activation_sparse_b200 import build as qs_build


@pytest.fixture
def current(monkeypatch):
    """A stand-in for the current stream: its handle, and whether it is being captured."""
    qs_build.build()
    now = {"stream": 7, "capturing": False}
    monkeypatch.setattr(qs, "_current_stream_ptr", lambda dev: now["stream"])
    monkeypatch.setattr(qs, "_call_context", lambda dev, stream, *t: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    return now


def workspace(op):
    """What a call of the op gets (QS_OP_SPARSE_LINEAR stands for the ops before the 4-bit ones)."""
    get = qs._workspace if op == qs.QS_OP_SPARSE_LINEAR else qs._stream_workspace
    return get(None, op, 4, 256, 512, 2, torch.device("cpu"))


OPS = [qs.QS_OP_FP4_SPARSE_LINEAR, qs.QS_OP_MOE_FFN, qs.QS_OP_SPARSE_LINEAR]


@pytest.mark.parametrize("op", OPS)
def test_two_threads_on_one_stream_have_two(current, op):
    got = []
    threads = [threading.Thread(target=lambda: got.append((workspace(op), workspace(op)))) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    got.append((workspace(op), workspace(op)))
    assert all(a is b for a, b in got)                       # kept within a thread
    assert len({a.data_ptr() for a, _ in got}) == len(got)   # and no other thread's
    assert all(int(a.count_nonzero()) == 0 for a, _ in got)


@pytest.mark.parametrize("op", OPS)
def test_two_streams_have_two(current, op):
    first = workspace(op)
    current["stream"] = 8
    second = workspace(op)
    assert second is not first and workspace(op) is second
    current["stream"] = 7
    assert workspace(op) is first


@pytest.mark.parametrize("op", OPS)
def test_a_captured_call_has_one_of_its_own(current, op):
    kept = workspace(op)
    current["capturing"] = True
    a, b = workspace(op), workspace(op)
    current["capturing"] = False
    assert len({w.data_ptr() for w in (kept, a, b)}) == 3
    assert workspace(op) is kept
    assert int(a[:256 + 65536].count_nonzero()) == 0
