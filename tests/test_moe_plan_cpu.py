"""Which kernels qs_moe_ffn takes, by the host's answer (no GPU needed)."""
import pytest
import torch

import top_activation_sparse_b200 as qs
from top_activation_sparse_b200 import build as qs_build

bf, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    qs_build.build()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("y", [bf, f32])
@pytest.mark.parametrize("E,top_k", [(1, 1), (8, 2), (100, 4), (256, 16)])
def test_one_token_of_at_most_4096_is_one_kernel(fp4, y, E, top_k):
    assert qs.qs_moe_ffn_kernels(1, 4096, 1832, E, top_k, fp4, y) == 1


def test_more_tokens():
    k = qs.qs_moe_ffn_kernels
    # 4-bit weights: everything else on the tensor cores
    assert k(2, 4096, 11008, 8, 2, True) == 4 and k(1, 4128, 11008, 8, 2, True) == 4
    # bf16: the queue kernel where few tokens share large experts, and results are bf16
    assert k(2, 4096, 11008, 8, 2) == 1 and k(2, 4096, 11008, 8, 2, y_dtype=f32) == 4
    assert k(8, 4096, 11008, 8, 2) == 4 and k(5, 544, 1000, 60, 4) == 4
    # rows longer than 4096: f32 results by the kernels with the shorter sums
    assert k(1, 8192, 11008, 4, 2) == 1 and k(1, 8192, 11008, 4, 2, y_dtype=f32) == 4
    # 64 tokens at a time; a last one alone
    assert k(65, 4096, 11008, 8, 2, True) == 5 and k(64, 4096, 11008, 8, 2, True) == 4
    assert k(150, 96, 48, 16, 3) == 12


@pytest.mark.parametrize("bad", [dict(T=0), dict(d_model=33), dict(d_model=8224), dict(d_ff=12), dict(n_experts=257),
                                 dict(top_k=0), dict(top_k=17), dict(n_experts=1)])
def test_invalid_sizes_have_none(bad):
    ok = dict(T=2, d_model=64, d_ff=64, n_experts=32, top_k=2)
    assert qs.qs_moe_ffn_kernels(**ok) == 4
    assert qs.qs_moe_ffn_kernels(**{**ok, **bad}) == 0
