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


class _Anything:
    """A library whose functions take anything and succeed."""

    def __getattr__(self, name):
        return lambda *args: 0


def test_a_callers_tensors_are_held_for_the_stream_of_the_call(current, monkeypatch):
    """Every tensor that the enqueued kernels use, the workspace too: a caller who drops it
    after the call must not get its memory again before that stream is done."""
    held = []
    monkeypatch.setattr(qs, "_call_context", lambda dev, stream, *t: held.extend(t) or contextlib.nullcontext())
    monkeypatch.setattr(qs, "_need_cuda", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(qs, "lib", lambda: _Anything())
    monkeypatch.setattr(qs, "qs_fp4_scale_bytes", lambda *a: 512)
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype)  # noqa: E731
    bf = torch.bfloat16
    f = torch.float32

    def check(call, given):
        held.clear()
        call(stream=3, **given)
        assert {n for n, t in given.items() if isinstance(t, torch.Tensor) and not any(t is h for h in held)} == set()

    check(lambda **k: qs.qs_fp4_quantize(**k),
          dict(x=z(2, 64, dtype=bf), tensor_scale=z(1, dtype=f), codes=z(2, 32), scales=z(512), values=z(2, 64, dtype=bf)))
    check(lambda **k: qs.qs_fp4_sparse_linear(k=8, **k),
          dict(x=z(2, 64, dtype=bf), w_codes=z(8, 32), w_scales=z(512), x_scale=z(1, dtype=f), w_scale=z(1, dtype=f),
               y=z(2, 8, dtype=bf), ws=z(1024)))
    check(lambda **k: qs.qs_moe_ffn(top_k=1, act="drelu", **k),
          dict(x=z(2, 32, dtype=bf), w_router=z(3, 32, dtype=bf), w_gate=z(3, 8, 16), w_up=z(3, 8, 16), w_down=z(3, 8, 16),
               s_gate=z(3, 8, 1), s_up=z(3, 8, 1), s_down=z(3, 8, 1), b_gate=z(3, 8, dtype=f), b_up=z(3, 8, dtype=f),
               y=z(2, 32, dtype=bf), experts=z(2, 1, dtype=torch.int32), weights=z(2, 1, dtype=f), ws=z(1024)))
