"""Products grouped by expert at the limits of their sizes and their launches, on the GPU."""
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_experts import experts, offsets_of

pytestmark = pytest.mark.gpu


def codes_of(P, K, seed):
    """int8 codes (P, K), made on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-127, 128, (P, K), dtype=torch.int8, device="cuda", generator=g)


def test_offsets_that_make_no_sense_of_many_rows():
    # every second expert claims all of 2^28 + 2^27 rows: more tiles than 31 bits count
    P, E, N, K = (1 << 28) + (1 << 27), 1024, 1, 4
    packed, s = experts(E, N, K, seed=1)
    off = torch.tensor([0, P] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    xq = torch.ones((P, K), dtype=torch.int8, device="cuda")
    out = bw.gemm_experts(xq, torch.ones(P, device="cuda"), off, packed, s, "bf16")
    dx = bw.grad_input_experts(out, off, packed, s)
    torch.cuda.synchronize()
    assert out.shape == (P, N) and dx.shape == (P, K)
