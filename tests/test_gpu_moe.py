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
from gpu_common import check_status, need_gpu, to_np

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


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T,dm", [(1, 4128), (1, 8192), (3, 8192), (20, 5120), (64, 8160)])
def test_rows_longer_than_4096(T, dm, fp4):
    run_check(T + dm, T, dm, 200, 4, 2, "drelu", fp4)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dm,dff,E,top_k", [(544, 1000, 4, 2), (4096, 2056, 2, 2), (96, 49152, 1, 1), (2080, 4104, 8, 8)])
def test_one_token(dm, dff, E, top_k, fp4):
    """Rows whose scales the copies cannot bring (d_model not a multiple of 512),
    several batches per CTA, a last batch that is not whole."""
    run_check(dm + dff, 1, dm, dff, E, top_k, "drelu", fp4)
    run_check(dm + dff, 1, dm, dff, E, top_k, "relu2_glu", fp4, torch.bfloat16)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T", [1, 3])
def test_closed_batches(T, fp4):
    """No neuron is open over many batches in a row (empty lists), then one is,
    then its second factor is 0 as well."""
    need_gpu()
    dm, dff, E = 256, 40000, 1
    a, vals = make(31, T, dm, dff, E, "drelu", fp4, bias=-100.0)
    r = qs.qs_moe_ffn(top_k=1, act="drelu", y_dtype=torch.float32, **a)
    assert torch.count_nonzero(r.y).item() == 0
    a["b_gate"][:, 39990] = 50.0                       # open, but the second factor is closed
    r = qs.qs_moe_ffn(top_k=1, act="drelu", y_dtype=torch.float32, **a)
    assert torch.count_nonzero(r.y).item() == 0
    a["b_gate"][:, 17] = a["b_up"][:, 17] = 50.0
    a["b_gate"][:, 20011] = a["b_up"][:, 20011] = 50.0
    r = qs.qs_moe_ffn(top_k=1, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)
    check(r, reference(a, vals, 1, "drelu"), dm, torch.float32)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T", [4, 20])
def test_a_token_that_is_not_finite_stays_alone(T, fp4):
    need_gpu()
    a, vals = make(33, T, 128, 256, 4, "drelu", fp4)
    want = reference(a, vals, 2, "drelu")
    a["x"][2, 5] = float("nan")
    r = qs.qs_moe_ffn(top_k=2, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)
    assert torch.isnan(r.y[2]).all()
    keep = [t for t in range(T) if t != 2]
    part = qs.MoeResult(r.y[keep], r.experts[keep], r.weights[keep])
    check(part, {k: v[keep] for k, v in want.items()}, 128, torch.float32)


def test_inputs_far_from_one():
    """x of 2^-10 and 2^20 (beyond float16, into which 4-bit weights bring x), and zeros."""
    need_gpu()
    for fp4 in (False, True):
        a, vals = make(34, 3, 128, 256, 4, "relu2_glu", fp4)
        a["x"][0] *= 2.0 ** -10
        a["x"][1] *= 2.0 ** 20
        a["x"][2] = 0.0
        r = qs.qs_moe_ffn(top_k=2, act="relu2_glu", y_dtype=torch.float32, experts=True, weights=True, **a)
        want = reference(a, vals, 2, "relu2_glu")
        check(qs.MoeResult(r.y[:2], r.experts[:2], r.weights[:2]), {k: v[:2] for k, v in want.items()}, 128, torch.float32)
        assert torch.count_nonzero(r.y[2]).item() == 0 and r.experts[2].tolist() == [0, 1]


def test_workspace_too_small_and_wrong_shapes_are_refused():
    need_gpu()
    a, _ = make(35, 2, 64, 64, 4, "drelu", False)
    need = qs.qs_workspace_size(qs.QS_OP_MOE_FFN, 2, 64, 64, 2)
    with pytest.raises(qs.QSError):
        qs.qs_moe_ffn(top_k=2, act="drelu", ws=torch.zeros(need - 16, dtype=torch.uint8, device=DEV), **a)
    for bad in (dict(x=a["x"].float()), dict(x=a["x"][:, :32]), dict(w_down=a["w_down"].transpose(1, 2)),
                dict(w_router=a["w_router"][:3]), dict(b_gate=a["b_gate"].half()), dict(s_up=a["w_up"].to(torch.uint8))):
        with pytest.raises(ValueError):
            qs.qs_moe_ffn(top_k=2, act="drelu", **{**a, **bad})
    for top_k in (0, 5):
        with pytest.raises(qs.QSError):
            qs.qs_moe_ffn(top_k=top_k, act="drelu", **a)
    with pytest.raises(qs.QSError):
        qs.qs_moe_ffn(top_k=2, act="drelu", **{**a, "x": a["x"][:0]})


def test_operators_together_eager_and_captured():
    """The layers of one block: weights quantised once, a 4-bit projection of
    sparsified activations, then 4-bit experts on its output; each step against
    the oracle on the step's own input, then the whole replayed."""
    need_gpu()
    T, d, dm, dff, E, K = 6, 512, 256, 320, 6, 2
    a, vals = make(36, T, dm, dff, E, "drelu", True)
    x = a.pop("x")
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(dm, d, generator=g, device=DEV) * d ** -0.5
    wq = qs.qs_fp4_quantize(w, "mx", "tiled")

    def block(x):
        u = qs.qs_fp4_sparse_linear(x, wq.codes, wq.scales, 358)
        return u, qs.qs_moe_ffn(u, top_k=K, act="drelu", y_dtype=torch.float32, experts=True, weights=True, **a)

    u, r = block(x)
    wv = oracle.fp4_quantize(w.cpu().numpy(), "mx")["values"]
    ref = oracle.fp4_sparse_linear(x.float().cpu().numpy(), wv, 358, "mx")
    # block sums in float32, then half a step of bf16
    assert np.all(np.abs(to_np(u) - ref["y"]) <= (d / 32 + 8) * 2.0 ** -23 * ref["mag"] + 2.0 ** -8 * np.abs(ref["y"]))
    check(r, reference({**a, "x": u}, vals, K, "drelu"), dm, torch.float32)

    static = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gu, gr = block(static)
    static.copy_(x)
    for _ in range(3):
        graph.replay()
        assert torch.equal(gu, u) and torch.equal(gr.y, r.y) and torch.equal(gr.experts, r.experts)
    # the same on a stream of its own, while the default one is busy with the graph
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        graph.replay()
        with torch.cuda.stream(s):
            u2, r2 = block(x)
        s.synchronize()
        assert torch.equal(u2, u) and torch.equal(r2.y, r.y)
    torch.cuda.synchronize()
    assert torch.equal(gr.y, r.y)


@pytest.mark.parametrize("T,dm,dff,E,top_k,one", [(3, 4096, 1832, 8, 2, False), (4, 8192, 688, 16, 2, False),
                                                  (20, 2048, 1368, 16, 1, True)])
def test_several_tokens_of_large_bf16_experts(T, dm, dff, E, top_k, one):
    """Experts large enough that only open rows are read; all tokens of one expert
    (two passes); no neuron open."""
    need_gpu()
    a, vals = make(T + dm, T, dm, dff, E, "drelu", False)
    if one:
        a["x"][:, 0] = 40.0
        a["w_router"][:, 0] = 0.0
        a["w_router"][5, 0] = 4.0
    call = lambda: qs.qs_moe_ffn(top_k=top_k, act="drelu", experts=True, weights=True, **a)  # noqa: E731
    r = call()
    check(r, reference(a, vals, top_k, "drelu"), dm, torch.bfloat16)
    if one:
        assert int((r.experts != 5).sum()) == 0
    assert torch.equal(call().y, r.y)
    a["b_gate"][:] = -1000.0
    assert torch.count_nonzero(call().y).item() == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_f32_results_of_long_sums(fp4):
    """h of both signs over 9000 neurons: the error stays that of float32 sums, 2^-24
    sqrt(number of additions) of the result, where sums cut off at every step of the
    matrix instructions would lose 2^-25 per step (here over 500 steps, 1.7e-5)."""
    need_gpu()
    T, dm, dff, E = 6, 512, 9000, 2
    a, vals = make(77, T, dm, dff, E, "relu2_glu", fp4)
    r = qs.qs_moe_ffn(top_k=1, act="relu2_glu", y_dtype=torch.float32, **a)
    want = reference(a, vals, 1, "relu2_glu")["y"]
    err = np.linalg.norm(to_np(r.y) - want, axis=1) / np.linalg.norm(want, axis=1)
    # three factors of h, each a sum over 512, and the sum over 9000, all as float32
    # sums with half a step per addition: 2^-24 (3 sqrt(512) + sqrt(9000)) = 1e-5 at worst,
    # a third of it for signs that cancel
    assert np.all(err <= 2.0 ** -24 * (3 * 512 ** 0.5 + 9000 ** 0.5) / 3), float(err.max())
