"""qs_moe_ffn by the kernels that a call takes: the queue kernel (one token; several tokens of
large bf16 experts) and the tensor-core kernels."""
import pytest
import torch

import top_activation_sparse_b200 as qs
from gpu_common import check_status, need_gpu
from test_gpu_moe import DEV, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dff,fp4", [(3664, False), (256, False), (256, True)])
def test_a_closed_neurons_second_factor_does_not_matter(dff, fp4):
    """Three tokens of one expert; the first opens a neuron whose second factor is not
    finite, for the others it is closed."""
    need_gpu()
    dm, e, j = 4096, 5, 100
    a, vals = make(41, 3, dm, dff, 8, "drelu", False)
    a["x"][:, 0], a["x"][:, 1] = 40.0, -10.0
    a["x"][0, 1] = 10.0
    a["w_router"][:, 0] = 0.0
    a["w_router"][e, 0] = 4.0
    a["w_gate"][e, j] = a["w_up"][e, j] = 0.0
    a["w_gate"][e, j, 1] = 1.0                          # 10 and -10 with a bias near -0.8
    if fp4:
        for n in ("gate", "up", "down"):
            r = qs.qs_fp4_quantize(vals[n], "mx", "rows", values=True)
            a["w_" + n], a["s_" + n], vals[n] = r.codes, r.scales, r.values
    want = reference(a, vals, 1, "drelu")
    if fp4:
        a["s_up"][e, j, 0] = 255                        # a NaN
    else:
        a["w_up"][e, j, 0] = float("inf")
    r = qs.qs_moe_ffn(top_k=1, act="drelu", experts=True, weights=True, **a)
    assert r.experts.flatten().tolist() == [e] * 3
    assert not torch.isfinite(r.y[0]).all()
    check(qs.MoeResult(r.y[1:], r.experts[1:], r.weights[1:]), {k: v[1:] for k, v in want.items()}, dm, torch.bfloat16)


@pytest.mark.parametrize("dff,fp4", [(3664, False), (256, False), (256, True)])
def test_a_down_row_that_is_not_finite_stays_in_its_expert(dff, fp4):
    """The neuron is closed for every token; tokens of other experts have the results they had."""
    need_gpu()
    dm, e = 4096, 2
    a, vals = make(42, 4, dm, dff, 8, "drelu", fp4)
    a["x"][:, 0] = 40.0
    a["w_router"][:, 0] = 0.0
    a["w_router"][e, 0] = a["w_router"][6, 1] = 4.0     # the expert of every token but the last,
    a["x"][3, :2] = torch.tensor([-40.0, 40.0])         # which prefers another
    a["b_gate"][e, 7] = -1000.0
    want = reference(a, vals, 1, "drelu")
    if fp4:
        a["s_down"][e, 7] = 255
    else:
        a["w_down"][e, 7] = float("nan")
    r = qs.qs_moe_ffn(top_k=1, act="drelu", experts=True, weights=True, **a)
    assert r.experts.flatten().tolist() == [e] * 3 + [6]
    check(qs.MoeResult(r.y[3:], r.experts[3:], r.weights[3:]), {k: v[3:] for k, v in want.items()}, dm, torch.bfloat16)
    # skipped or not, a row of NaNs does not come out as anything else
    finite = torch.isfinite(r.y[:3])
    if finite.all():
        check(qs.MoeResult(r.y, r.experts, r.weights), want, dm, torch.bfloat16)
    else:
        assert not finite.any()


@pytest.mark.parametrize("T", [1, 2])
def test_the_least_scale(T):
    """Blocks with the scale 2^-127 in the first and second factors, of inputs large enough to see them:
    products of 2^-127 and 2^126, exact in float32 but for the sums."""
    need_gpu()
    dm, dff, E = 256, 128, 2
    a, _ = make(43, T, dm, dff, E, "relu2_glu", True)
    a["x"] = (a["x"].float().clamp(-3, 3) * 2.0 ** 126).to(torch.bfloat16)
    a["w_router"][:] = 0.0
    vals = {}
    for n in ("gate", "up", "down"):
        if n != "down":
            a["s_" + n][:] = 0
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV, dtype=torch.float64)
        c = a["w_" + n].long()
        vals[n] = torch.stack((lut[c & 15], lut[c >> 4]), -1).flatten(-2) * torch.exp2(
            a["s_" + n].double() - 127).repeat_interleave(32, -1)
    r = qs.qs_moe_ffn(top_k=1, act="relu2_glu", y_dtype=torch.float32, experts=True, weights=True, **a)
    x, d = a["x"].double(), {n: v[0] for n, v in vals.items()}          # equal logits: the first expert
    want = (torch.relu(x @ d["up"].t()) ** 2 * (x @ d["gate"].t())) @ d["down"]
    assert bool((want != 0).any(1).all())
    check(r, dict(y=want.cpu().numpy(), experts=[[0]] * T, weights=[[1.0]] * T), dm, torch.float32)


# ---- the queue kernel ----------------------------------------------------------------------
# several tokens: (T, d_model, d_ff, experts, top_k); the second is routed through the workspace
# (a router that the CTAs do not each evaluate), the third has more than 8 tokens
SEVERAL = [(3, 4096, 1832, 8, 2), (3, 4096, 3664, 20, 1), (20, 2048, 1368, 16, 1)]
bf = torch.bfloat16


def one_kernel(T, dm, dff, E, top_k, fp4=False, y_dtype=bf):
    """These sizes take the queue kernel."""
    assert qs.qs_moe_ffn_kernels(T, dm, dff, E, top_k, fp4, y_dtype) == 1


def queue(a, top_k, act, **kw):
    return qs.qs_moe_ffn(top_k=top_k, act=act, experts=True, weights=True, **kw, **a)


@pytest.mark.parametrize("size", SEVERAL)
@pytest.mark.parametrize("act,bias", [("drelu", -0.8), ("drelu", None), ("drelu", 30.0), ("relu2_glu", None)])
def test_queue_kernel(size, act, bias):
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(50 + T + E, T, dm, dff, E, act, False, bias)
    check(queue(a, top_k, act), reference(a, vals, top_k, act), dm, bf)


@pytest.mark.parametrize("size", [(1, 4128, 200, 4, 2), (1, 8192, 264, 4, 2), (1, 8160, 136, 9, 1), (3, 8192, 920, 8, 2)])
@pytest.mark.parametrize("act,bias", [("drelu", -0.8), ("relu2_glu", None)])
def test_queue_kernel_rows_longer_than_4096(size, act, bias):
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(60 + T + dm, T, dm, dff, E, act, False, bias)
    ws = qs.new_workspace(qs.QS_OP_MOE_FFN, T, dm, dff, top_k, DEV)
    r = queue(a, top_k, act, ws=ws)
    check(r, reference(a, vals, top_k, act), dm, bf)
    assert torch.equal(queue(a, top_k, act, ws=ws).y, r.y)
    assert int(ws[256:256 + 65536].count_nonzero()) == 0


@pytest.mark.parametrize("size", SEVERAL)
def test_queue_kernel_leaves_its_workspace_ready(size):
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(51, T, dm, dff, E, "relu2_glu", False)
    ws = qs.new_workspace(qs.QS_OP_MOE_FFN, T, dm, dff, top_k, DEV)
    first = queue(a, top_k, "relu2_glu", ws=ws)
    for _ in range(6):
        r = queue(a, top_k, "relu2_glu", ws=ws)
        assert torch.equal(r.y, first.y) and torch.equal(r.experts, first.experts)
    check_status(ws)
    assert int(ws[256:256 + 65536].count_nonzero()) == 0


@pytest.mark.parametrize("size", SEVERAL)
def test_queue_kernel_twice_at_once(size):
    """Two calls that share the SMs, each with its stream's own workspace."""
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(52, T, dm, dff, E, "drelu", False)
    want = queue(a, top_k, "drelu").y
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [queue(a, top_k, "drelu", stream=s).y for _ in range(20) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(want, g) for g in got)


@pytest.mark.parametrize("size", SEVERAL)
def test_queue_kernel_captured_and_replayed(size):
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(53, T, dm, dff, E, "drelu", False)
    eager = queue(a, top_k, "drelu").y
    x = a.pop("x")
    static = torch.zeros_like(x)
    graphs = []
    for _ in range(2):                       # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = queue({**a, "x": static}, top_k, "drelu").y
        graphs.append((graph, y))
    static.copy_(x)
    for _ in range(3):
        for graph, y in graphs:
            y.zero_()
            graph.replay()
            assert torch.equal(y, eager)
    assert torch.equal(queue({**a, "x": x}, top_k, "drelu").y, eager)


@pytest.mark.parametrize("size", SEVERAL)
def test_queue_kernel_a_token_that_is_not_finite_stays_alone(size):
    need_gpu()
    T, dm, dff, E, top_k = size
    one_kernel(*size)
    a, vals = make(54, T, dm, dff, E, "drelu", False)
    want = reference(a, vals, top_k, "drelu")
    a["x"][1, 5] = float("nan")
    r = queue(a, top_k, "drelu")
    assert torch.isnan(r.y[1]).all()
    keep = [t for t in range(T) if t != 1]
    check(qs.MoeResult(r.y[keep], r.experts[keep], r.weights[keep]), {k: v[keep] for k, v in want.items()}, dm, bf)


def test_queue_kernel_closed_batches():
    """No neuron is open over many batches in a row (empty lists), then one is, then its second
    factor is 0 as well; rows of y behind the last are left as they were."""
    need_gpu()
    T, dm, dff, E = 3, 512, 40000, 4
    one_kernel(T, dm, dff, E, 1)
    a, vals = make(55, T, dm, dff, E, "drelu", False, bias=-100.0)
    buf = torch.full((T + 2, dm), 7.0, device=DEV, dtype=bf)
    r = queue(a, 1, "drelu", y=buf[:T])
    assert torch.count_nonzero(r.y).item() == 0 and bool((buf[T:] == 7.0).all())
    a["b_gate"][:, 39990] = 50.0                       # open, but the second factor is closed
    assert torch.count_nonzero(queue(a, 1, "drelu").y).item() == 0
    a["b_gate"][:, 17] = a["b_up"][:, 17] = 50.0
    a["b_gate"][:, 20011] = a["b_up"][:, 20011] = 50.0
    check(queue(a, 1, "drelu"), reference(a, vals, 1, "drelu"), dm, bf)


# one token: a router of more than 64 experts, or of more than 128 KB, is not evaluated by
# each CTA: queue items, whose result is handed over through the workspace
@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("act", ["drelu", "relu2_glu"])
@pytest.mark.parametrize("dm,dff,E,top_k", [(4096, 264, 32, 2), (256, 520, 100, 4), (96, 72, 256, 16), (1056, 136, 65, 1)])
def test_one_token_and_a_large_router(dm, dff, E, top_k, act, fp4):
    need_gpu()
    y = torch.float32
    one_kernel(1, dm, dff, E, top_k, fp4, y)
    a, vals = make(56 + E, 1, dm, dff, E, act, fp4)
    ws = qs.new_workspace(qs.QS_OP_MOE_FFN, 1, dm, dff, top_k, DEV)
    first = queue(a, top_k, act, y_dtype=y, ws=ws)
    check(first, reference(a, vals, top_k, act), dm, y)
    for _ in range(4):
        assert torch.equal(queue(a, top_k, act, y_dtype=y, ws=ws).y, first.y)
    check_status(ws)
    assert int(ws[256:256 + 65536].count_nonzero()) == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_one_token_captured_on_two_streams(fp4):
    need_gpu()
    dm, dff, E = 4096, 264, 32
    one_kernel(1, dm, dff, E, 2, fp4)
    a, vals = make(57, 1, dm, dff, E, "drelu", fp4)
    want = queue(a, 2, "drelu").y
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = queue(a, 2, "drelu").y
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):                      # beside the graph, on another stream
        y.zero_()
        graph.replay()
        got = queue(a, 2, "drelu", stream=s).y
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(got, want)
