"""Rounding of qs_moe_ffn's float32 results against the formula in 64 bits.

Tolerance, per token, on the 2-norm of the error over that of y: that of float32 sums with
half a step, 2^-24, per addition.  h has three factors (squared ReLU), each a sum over
d_model, and y is a sum over d_ff, of both signs: errors that are independent of each other add up to
2^-24 (3 sqrt(d_model) + sqrt(d_ff)) of the result's size at most if every addition were as
large as the whole; partial sums of both signs are a third of it on average."""
import pytest
import torch

import top_activation_sparse_b200 as qs
from gpu_common import need_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(seed, T, dm, dff, E, fp4):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    a = {"x": torch.randn(T, dm, generator=g, device=DEV).to(torch.bfloat16),
         "w_router": (torch.randn(E, dm, generator=g, device=DEV) * 2 * dm ** -0.5).to(torch.bfloat16)}
    vals = {}
    for n, std in (("gate", dm ** -0.5), ("up", dm ** -0.5), ("down", dff ** -0.5)):
        w = torch.randn(E, dff, dm, generator=g, device=DEV) * std
        if fp4:
            r = qs.qs_fp4_quantize(w, "mx", "rows", values=True)
            a["w_" + n], a["s_" + n], vals[n] = r.codes, r.scales, r.values
        else:
            a["w_" + n] = vals[n] = w.to(torch.bfloat16)
    return a, vals


def formula(a, vals, experts):
    """y in 64 bits, squared ReLU, for the experts chosen."""
    x = a["x"].double()
    e = experts.long()
    p = torch.softmax((x @ a["w_router"].double().t()).gather(1, e), -1)
    y = torch.zeros_like(x)
    for i in e.unique().tolist():
        t, j = (e == i).nonzero(as_tuple=True)
        gate, up, down = (vals[n][i].double() for n in ("gate", "up", "down"))
        y[t] += p[t, j, None] * ((torch.relu(x[t] @ up.t()) ** 2 * (x[t] @ gate.t())) @ down)
    return y


def check_sums(T, dm, dff, E, top_k, fp4, tol=None):
    need_gpu()
    a, vals = layer(T + dm + top_k, T, dm, dff, E, fp4)
    r = qs.qs_moe_ffn(top_k=top_k, act="relu2_glu", y_dtype=torch.float32, experts=True, **a)
    want = formula(a, vals, r.experts)
    err = ((r.y.double() - want).norm(dim=1) / want.norm(dim=1)).max().item()
    assert err <= (tol or 2.0 ** -24 * (3 * dm ** 0.5 + dff ** 0.5) / 3), err


@pytest.mark.parametrize("T,top_k", [(64, 16), (64, 11), (65, 8)])
def test_long_ranges_of_4bit_experts(T, top_k):
    """So many pairs of a token and an expert that an expert's neurons are dealt out in few ranges."""
    check_sums(T, 256, 28672, 16, top_k, True)


@pytest.mark.parametrize("T", [1, 2])
def test_rows_longer_than_4096(T):
    """bf16 experts whose sums go to registers after 128 terms, i.e. eight matrix instructions, each of which
    cuts off up to 2^-23 of the sum so far, half of it on average, the sum so far being half of the whole on
    average: 8 x 2^-25 for each of four sums (three factors and the down projection).  The sums of 128 are
    then added as above."""
    dm, dff = 8192, 28672
    check_sums(T, dm, dff, 1, 1, False, 4 * 8 * 2.0 ** -25 + 2.0 ** -24 * (3 * (dm / 128) ** 0.5 + (dff / 128) ** 0.5) / 3)
