"""qs_moe_ffn on the GPU against the fp64 oracle.

Tolerance, per token, on the 2-norm of the error over that of y.  h enters the
down projection with an error below 2^-24 of itself (2^-17 is allowed).  A sum over d_model in float32
takes d_model / 16 + 16 additions (matrix instructions of 16, eight partial
sums), each off by at most 2^-23 of a partial sum, independently: about
sqrt(d_model / 16 + 16) 2^-23 of the sum's own size, which enters h twice or
three times and, for dReLU, with the factor by which the bias makes h smaller
than the product of the projections (below 3): 8 in all.  A bf16 result adds
half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import oracle
import top_activation_sparse_b200 as qs
import workloads
from gpu_common import bits, check_status, need_gpu, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(seed, T, dm, dff, E, act, fp4, bias=-0.8):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    a = {"x": rnd(T, dm).to(torch.bfloat16), "w_router": rnd(E, dm, std=2 * dm ** -0.5).to(torch.bfloat16)}
    vals = {}
    for n, std in (("gate", dm ** -0.5), ("up", dm ** -0.5), ("down", dff ** -0.5)):
        w = rnd(E, dff, dm, std=std)
        if fp4:
            r = qs.qs_fp4_quantize(w, "mx", "rows", values=True)
            a["w_" + n], a["s_" + n], vals[n] = r.codes, r.scales, r.values
        else:
            a["w_" + n] = vals[n] = w.to(torch.bfloat16)
    if act == "drelu" and bias is not None:
        a["b_gate"] = torch.full((E, dff), bias, device=DEV) + 0.1 * rnd(E, dff)
        a["b_up"] = torch.full((E, dff), bias, device=DEV) + 0.1 * rnd(E, dff)
    return a, vals


def reference(a, vals, top_k, act):
    n = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    return oracle.moe_ffn(n(a["x"]), n(a["w_router"]), n(vals["gate"]), n(vals["up"]), n(vals["down"]), top_k, act,
                          n(a.get("b_gate")), n(a.get("b_up")))


def check(r, ref, dm, y_dtype):
    np.testing.assert_array_equal(r.experts.cpu().numpy(), ref["experts"])
    np.testing.assert_allclose(r.weights.cpu().numpy(), ref["weights"], rtol=2e-5, atol=1e-7)
    y, want = to_np(r.y).astype(np.float64), ref["y"]
    rel = 2.0 ** -17 + 8 * (dm / 16 + 16) ** 0.5 * 2.0 ** -23 + (2.0 ** -8 if y_dtype == torch.bfloat16 else 0.0)
    err, norm = np.linalg.norm(y - want, axis=1), np.linalg.norm(want, axis=1)
    assert np.all(err <= rel * norm), float((err / norm).max())


def run_check(seed, T, dm, dff, E, top_k, act, fp4, y_dtype=torch.float32, ws=None, bias=-0.8):
    need_gpu()
    a, vals = make(seed, T, dm, dff, E, act, fp4, bias)
    r = qs.qs_moe_ffn(top_k=top_k, act=act, y_dtype=y_dtype, experts=True, weights=True, ws=ws, **a)
    check(r, reference(a, vals, top_k, act), dm, y_dtype)
    return a, vals, r


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("act", ["drelu", "relu2_glu"])
@pytest.mark.parametrize("T,dm,dff,E,top_k", [
    (1, 32, 8, 1, 1), (1, 256, 512, 8, 2), (2, 512, 264, 8, 2), (3, 96, 1000, 5, 5), (5, 544, 1000, 60, 4),
    (8, 160, 328, 4, 3), (9, 1024, 136, 2, 1), (17, 288, 72, 1, 1), (33, 64, 104, 3, 2), (40, 96, 96, 1, 1),
    (64, 512, 256, 8, 2), (64, 64, 40, 256, 16), (65, 128, 64, 6, 2), (150, 96, 48, 16, 3)])
def test_sizes(T, dm, dff, E, top_k, act, fp4):
    run_check(T * 31 + dm + dff, T, dm, dff, E, top_k, act, fp4)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T", [1, 4, 16])
def test_wide_rows(T, fp4):
    """Rows longer than the eight warps' first pieces, several column tiles, more neurons than one round."""
    run_check(T, T, 4096, 1160, 4, 2, "drelu", fp4, torch.bfloat16)
    run_check(T, T, 2080, 520, 4, 2, "relu2_glu", fp4)


@pytest.mark.parametrize("fp4", [False, True])
def test_one_expert_takes_every_token(fp4):
    """64 tokens of one expert: two passes of 32, whose open neurons differ."""
    need_gpu()
    a, vals = make(9, 64, 128, 512, 4, "drelu", fp4, bias=-1.5)
    a["x"][:, 0] = 40.0                     # every token's largest input asks for expert 2
    a["w_router"][:, 0] = 0.0
    a["w_router"][2, 0] = 4.0
    r = qs.qs_moe_ffn(top_k=1, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)
    assert int((r.experts != 2).sum()) == 0
    check(r, reference(a, vals, 1, "drelu"), 128, torch.float32)


def test_every_neuron_closed_gives_zero():
    need_gpu()
    a, vals = make(4, 6, 64, 128, 4, "drelu", False, bias=-100.0)
    r = qs.qs_moe_ffn(top_k=2, act="drelu", **a)
    assert torch.count_nonzero(r.y).item() == 0


def test_every_neuron_open():
    run_check(21, 10, 128, 640, 3, 2, "drelu", False, bias=30.0)
    run_check(21, 10, 128, 640, 3, 2, "drelu", True, bias=30.0)


def test_no_bias():
    run_check(22, 3, 128, 256, 4, 2, "drelu", False, bias=None)


def test_equal_logits_take_the_lower_experts():
    need_gpu()
    a, vals = make(5, 7, 64, 64, 12, "drelu", False)
    a["w_router"][:] = a["w_router"][3]
    r = qs.qs_moe_ffn(top_k=3, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)
    assert r.experts.tolist() == [[0, 1, 2]] * 7
    check(r, reference(a, vals, 3, "drelu"), 64, torch.float32)


def test_scales_of_every_size():
    """Power-of-two scales from 2^-120 to above 2 (where a second factor is needed)."""
    need_gpu()
    T, dm, dff, E = 3, 128, 256, 2
    a, _ = make(6, T, dm, dff, E, "drelu", True, bias=None)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    vals = {}
    for n in ("gate", "up", "down"):
        a["s_" + n] = torch.randint(120, 137, (E, dff, dm // 32), generator=g, device=DEV, dtype=torch.uint8)
        a["s_" + n][:, ::7] = 3                 # whole rows that are next to nothing
        lut = torch.tensor(list(oracle.E2M1) + list(-oracle.E2M1), device=DEV, dtype=torch.float64)
        c = a["w_" + n].long()
        q = torch.stack((lut[c & 15], lut[c >> 4]), -1).flatten(-2)
        vals[n] = q * torch.exp2(a["s_" + n].double() - 127).repeat_interleave(32, -1)
    r = qs.qs_moe_ffn(top_k=2, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)
    nn = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = oracle.moe_ffn(nn(a["x"]), nn(a["w_router"]), nn(vals["gate"]), nn(vals["up"]), nn(vals["down"]), 2, "drelu")
    check(r, ref, dm, torch.float32)


def test_same_bits_each_time_and_workspace_ready():
    need_gpu()
    T, dm, dff, E = 12, 512, 520, 8
    ws = qs.new_workspace(qs.QS_OP_MOE_FFN, T, dm, dff, 2, DEV)
    a, vals, first = run_check(7, T, dm, dff, E, 2, "relu2_glu", False, ws=ws)
    for _ in range(6):
        r = qs.qs_moe_ffn(top_k=2, act="relu2_glu", y_dtype=torch.float32, ws=ws, **a)
        assert torch.equal(r.y, first.y)
    check_status(ws)
    assert int(ws[256:256 + 65536].count_nonzero()) == 0


def test_two_calls_at_once_on_two_streams():
    """Two layers that share the SMs, each with its stream's own workspace."""
    need_gpu()
    a, vals = make(8, 4, 1024, 2048, 8, "drelu", False)
    want = qs.qs_moe_ffn(top_k=2, act="drelu", y_dtype=torch.float32, **a).y
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [qs.qs_moe_ffn(top_k=2, act="drelu", y_dtype=torch.float32, stream=s, **a).y for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, g) for g in got)


def test_captured_and_replayed():
    need_gpu()
    a, vals = make(10, 3, 256, 512, 8, "drelu", False)
    eager = qs.qs_moe_ffn(top_k=2, act="drelu", y_dtype=torch.float32, **a).y
    x = a.pop("x")
    static = torch.zeros_like(x)
    graphs = []
    for _ in range(2):                       # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = qs.qs_moe_ffn(static, top_k=2, act="drelu", y_dtype=torch.float32, **a).y
        graphs.append((graph, y))
    static.copy_(x)
    for _ in range(3):
        for graph, y in graphs:
            y.zero_()
            graph.replay()
            assert torch.equal(y, eager)
    assert torch.equal(qs.qs_moe_ffn(x, top_k=2, act="drelu", y_dtype=torch.float32, **a).y, eager)


def test_rows_behind_the_last_are_left_as_they_were():
    need_gpu()
    a, vals = make(11, 5, 64, 64, 4, "drelu", False)
    buf = torch.full((9, 64), 7.0, device=DEV)
    qs.qs_moe_ffn(top_k=2, act="drelu", y=buf[:5], **a)
    assert bool((buf[5:] == 7.0).all()) and not bool((buf[:5] == 7.0).any())
