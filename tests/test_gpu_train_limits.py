"""The training entry points where memory ends and values leave the ordinary range: what lies
behind a tensor, infinities, rows far from zero, launches past the grid's limit, every tile
configuration.  Tolerances count roundings as in test_gpu_train.py."""
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_train import bf16

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ what lies behind a tensor

# odd tokens and odd rows: the last value of dy shares its dword with what lies behind it
@pytest.mark.parametrize("M,N,K", [(1, 1, 4), (3, 17, 20), (31, 63, 252), (33, 65, 260), (129, 641, 2564),
                                   (1001, 641, 2560), (2047, 4097, 14340)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_grad_weight_of_a_prefix(M, N, K, dt):
    big = bf16(M + 1, N, seed=M, scale=1e-3, hot=False)
    xq, a = bw.quant_act_pow2(bf16(M, K, seed=K))
    clean = bw.grad_weight(big[:M].clone(), xq, a, out_dtype=dt)
    assert torch.isfinite(clean).all()
    for value in (float("nan"), float("inf"), -float("inf")):
        big[M] = value
        assert torch.equal(bw.grad_weight(big[:M], xq, a, out_dtype=dt), clean), value
        assert torch.equal(bw.grad_weight(big[:M], xq, a, out_dtype=dt, workspace=False),
                           bw.grad_weight(big[:M].clone(), xq, a, out_dtype=dt, workspace=False)), value
