"""Products grouped by expert at the limits of their sizes and their launches, on the GPU."""
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_experts import experts, offsets_of, spread
from test_gpu_train import BF, TINY, U, bf16, check_grad_input, close

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


def test_input_gradient_of_more_tiles_than_a_launch():
    # 2^30 rows, the most there may be, are 2^24 tiles of 64; with one output column of an expert dx is
    # bf16(dy s) times a ternary weight, exactly
    P, E, N, K = 1 << 30, 3, 1, 4
    packed, s = experts(E, N, K, seed=1)
    s = torch.tensor([[0.75], [1.5], [0.3]], device="cuda")
    counts = [5, (1 << 29) + 77, (1 << 29) - 82]
    table = bf16(4093, N, seed=2)
    dy = table.repeat(P // 4093 + 1, 1)[:P]
    dx = bw.grad_input_experts(dy, offsets_of(counts), packed, s)
    at = 0
    for e, c in enumerate(counts):
        w = bw.unpack_weights(packed[e].clone(), K).to(torch.bfloat16)
        scaled = (table.float() * s[e]).to(torch.bfloat16) * w
        for lo in range(at, at + c, 4093 << 12):
            n = min(4093 << 12, at + c - lo)
            want = scaled.roll(-(lo % 4093), 0).repeat(n // 4093 + 1, 1)[:n]
            assert (dx[lo:lo + n] == want).all(), (e, lo)
        at += c


def test_product_of_more_tiles_than_a_launch():
    # four stacks of one column and 2^28 + 2^22 rows: 4.3 million row tiles times four column tiles
    P, E, K = (1 << 28) + (1 << 22), 3, 4
    w = [experts(E, 1, K, seed=i) for i in range(4)]
    counts = [7, 1 << 28, (1 << 22) - 7]
    table = codes_of(4093, K, seed=1)
    xq = table.repeat(P // 4093 + 1, 1)[:P]
    outs = bw.gemm_experts_grouped(xq, torch.ones(P, device="cuda"), offsets_of(counts), [p for p, _ in w],
                                   [s for _, s in w], "i32")
    for g, (packed, _) in enumerate(w):
        at = 0
        for e, c in enumerate(counts):
            want = (table.float() @ bw.unpack_weights(packed[e].clone(), K).float().t().contiguous()).int()
            for lo in range(at, at + c, 4093 << 12):
                n = min(4093 << 12, at + c - lo)
                assert torch.equal(outs[g][lo:lo + n], want.roll(-(lo % 4093), 0).repeat(n // 4093 + 1, 1)[:n])
            at += c


# input gradients of several stacks that go from one to the next in each kernel: sums of several
# steps, with stacks of a part of a step and of nothing between them
SEVERAL = [(1500, 64, (200, 72), 2064), (1500, 64, (201, 77), 2052), (1500, 64, (75, 3, 0, 201), 1540),
           (300, 16, (200, 136), 2560), (300, 16, (201, 3, 77, 130), 2564), (100, 4, (200, 8, 0, 136), 2064),
           (100, 4, (201, 77), 2052), (100, 4, (640, 712), 2064), (100, 4, (641, 5, 0, 713), 2052)]


@pytest.mark.parametrize("P,E,Ns,K", SEVERAL)
@pytest.mark.parametrize("kind", ["even", "skewed"])
def test_input_gradient_across_stacks(P, E, Ns, K, kind):
    counts = spread(P, E, 3, kind)
    off = offsets_of(counts)
    dys = [bf16(P, n, seed=n + i, scale=1e-3, hot=False) for i, n in enumerate(Ns)]
    w = [experts(E, n, K, seed=n + i) if n else (torch.empty((E, 0, K // 4), dtype=torch.uint8, device="cuda"),
                                                 torch.empty((E, 0), device="cuda")) for i, n in enumerate(Ns)]
    got = bw.grad_input_experts_grouped(dys, off, [p for p, _ in w], [s for _, s in w])
    at = 0
    for e, c in enumerate(counts):
        if c:
            check_grad_input([d[at:at + c] for d, n in zip(dys, Ns) if n],
                             [p[e].clone() for (p, _), n in zip(w, Ns) if n],
                             [s[e].clone() for (_, s), n in zip(w, Ns) if n], K, got[at:at + c], f"{kind} expert {e}")
        at += c


# one size for each kernel of the weight gradient
@pytest.mark.parametrize("P,E,N,K", [(700, 8, 300, 516), (300, 3, 257, 1028), (1200, 2, 256, 256), (4100, 4, 33, 64),
                                     (1700, 4, 1280, 4100), (1100, 3, 1281, 1028)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["absmax", "pow2"])
def test_weight_gradient_against_the_codes_values(P, E, N, K, dt, scale):
    # against sum dy xq / a itself.  Of absmax codes each xq / a takes the reciprocal (1 ulp and a Newton
    # step: one rounding), a product and the rounding to bf16; of powers of two none of them rounds
    counts = spread(P, E, P, "skewed")
    dy = bf16(P, N, seed=N, scale=1e-3, hot=False)
    xq, a = (bw.quant_act if scale == "absmax" else bw.quant_act_pow2)(bf16(P, K, seed=K))
    out = bw.grad_weight_experts(dy, xq, a, offsets_of(counts), dt)
    operand = BF * (1 + 3 * U) + 3 * U if scale == "absmax" else 0.0
    at = 0
    for e, c in enumerate(counts):
        if c:
            d = dy[at:at + c].double().t().contiguous()
            x = xq[at:at + c].double() / a[at:at + c].double()[:, None]
            ref, size = d @ x, d.abs() @ x.abs()
            tol = (operand + (c + 64) * U * (1 + operand)) * size + TINY
            if dt == "bf16":
                tol = (1 + BF) * tol + BF * ref.abs()
            close(out[e], ref, tol, f"expert {e}")
        at += c


@pytest.mark.parametrize("P,E,N,K", [(20, 3, 32, 64), (20, 3, 33, 68), (1500, 64, 40, 2064)])
def test_input_gradient_unused_code_is_zero(P, E, N, K):
    counts = spread(P, E, 1, "even")
    packed, s = experts(E, N, K, seed=1)
    dy = bf16(P, N, seed=1, hot=False)
    unused, zero = packed.clone(), packed.clone()
    unused[:, 7], zero[:, 7] = 0xFF, 0x55
    a, b = (bw.grad_input_experts(dy, offsets_of(counts), p, s) for p in (unused, zero))
    assert torch.equal(a, b)
