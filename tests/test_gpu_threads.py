"""Two host threads inside calls on one stream, without a workspace of their own:
every call's result is that of the call alone."""
import threading

import pytest
import torch

import top_activation_sparse_b200 as qs
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def both(calls, same, rounds=60):
    """Each of the two calls in a thread of its own, again and again."""
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(rounds):
            got[i].append(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == rounds
        assert all(same(g, want[i]) for g in got[i])


def rnd(seed, *shape, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * std


@pytest.mark.parametrize("T,k", [(5, 512), (5, 300), (300, 300)])
def test_4bit_projection(T, k):
    need_gpu()
    w = qs.qs_fp4_quantize(rnd(1, 1024, 512), "nv", "tiled")
    xs = [rnd(2 + i, T, 512).to(torch.bfloat16) for i in range(2)]
    both([lambda x=x: qs.qs_fp4_sparse_linear(x, w.codes, w.scales, k, format="nv") for x in xs], torch.equal)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T", [1, 6, 70])
def test_experts(T, fp4):
    need_gpu()
    dm, dff, E = 256, 512, 8
    a = {"w_router": rnd(1, E, dm, std=0.1).to(torch.bfloat16)}
    for i, n in enumerate(("gate", "up", "down")):
        w = rnd(2 + i, E, dff, dm, std=0.06)
        if fp4:
            r = qs.qs_fp4_quantize(w, "mx", "rows")
            a["w_" + n], a["s_" + n] = r.codes, r.scales
        else:
            a["w_" + n] = w.to(torch.bfloat16)
    xs = [rnd(5 + i, T, dm).to(torch.bfloat16) for i in range(2)]
    both([lambda x=x: qs.qs_moe_ffn(x, top_k=2, act="relu2_glu", y_dtype=torch.float32, **a).y for x in xs], torch.equal)


@pytest.mark.parametrize("T", [1, 8])
def test_projection_and_ffn(T):
    """(their float sums are added in an order that is not fixed: bf16 results may round either way)"""
    need_gpu()
    d, dff = 1024, 2048
    near = lambda a, b: bool(((a.float() - b.float()).norm() <= 2.0 ** -7 * b.float().norm()).item())  # noqa: E731
    wt = rnd(1, d, dff, std=0.03).to(torch.bfloat16)
    xs = [rnd(2 + i, T, d).to(torch.bfloat16) for i in range(2)]
    both([lambda x=x: qs.qs_sparse_linear(x, wt, 700) for x in xs], near)
    up, gate, down = (rnd(4 + i, *s, std=0.03).to(torch.bfloat16) for i, s in enumerate(((d, dff), (d, dff), (dff, d))))
    both([lambda x=x: qs.qs_sparse_ffn(x, up, gate, down, "relu2_glu", 700, 1400).y for x in xs], near)


def test_a_dropped_workspace_is_not_handed_out_while_its_call_runs():
    need_gpu()
    dm, dff, E, T = 256, 512, 8, 6
    a = {"x": rnd(1, T, dm).to(torch.bfloat16), "w_router": rnd(2, E, dm, std=0.1).to(torch.bfloat16)}
    a.update({"w_" + n: rnd(3 + i, E, dff, dm, std=0.06).to(torch.bfloat16) for i, n in enumerate(("gate", "up", "down"))})
    call = lambda **k: qs.qs_moe_ffn(top_k=2, act="relu2_glu", y_dtype=torch.float32, **k, **a).y  # noqa: E731
    want = call()
    s = torch.cuda.Stream()
    for _ in range(3):
        ws = qs.new_workspace(qs.QS_OP_MOE_FFN, T, dm, dff, 2, DEV)
        size = ws.numel()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        y = call(ws=ws, stream=s)
        del ws
        other = torch.full((size,), 0x7f, dtype=torch.uint8, device=DEV)     # the memory, if it were free
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del other


@pytest.mark.parametrize("T", [1, 8])
def test_projection_and_ffn_captured_without_a_workspace(T):
    """Two graphs, each call with a workspace of its own: several tokens replayed at once on two streams, one
    token (whose layer may be one kernel that needs its whole grid resident) in turn."""
    need_gpu()
    d, dff = 1024, 2048
    wt = rnd(1, d, dff, std=0.03).to(torch.bfloat16)
    up, gate, down = (rnd(4 + i, *s, std=0.03).to(torch.bfloat16) for i, s in enumerate(((d, dff), (d, dff), (dff, d))))
    x = rnd(2, T, d).to(torch.bfloat16)

    def layer():
        return qs.qs_sparse_linear(x, wt, 700), qs.qs_sparse_ffn(x, up, gate, down, "relu2_glu", 700, 1400).y

    want = layer()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()                              # its workspaces' memory goes to the second layer's
            got = layer()
        graphs.append((graph, got, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, got, s in graphs:
            with torch.cuda.stream(s):
                for g in got:
                    g.zero_()
                graph.replay()
            if T == 1:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for _, got, _ in graphs:
            for g, w in zip(got, want):
                assert (g.float() - w.float()).norm() <= 2.0 ** -7 * w.float().norm()
    after = layer()                              # the eager workspaces are as they were
    assert all((g.float() - w.float()).norm() <= 2.0 ** -7 * w.float().norm() for g, w in zip(after, want))
