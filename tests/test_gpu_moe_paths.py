"""qs_moe_ffn by the kernels that a call takes: the queue kernel (one token; several tokens of
large bf16 experts) and the tensor-core kernels."""
import pytest
import torch

import top_activation_sparse_b200 as qs
from gpu_common import need_gpu
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
