"""The training entry points where memory ends and values leave the ordinary range: what lies
behind a tensor, infinities, rows far from zero, launches past the grid's limit, every tile
configuration.  Tolerances count roundings as in test_gpu_train.py."""
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_train import (BF, TINY, U, bf16, check_grad_input, check_grad_weight, close, f32,
                            ternary)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ what lies behind a tensor

# odd tokens and odd rows: the last value of dy shares its dword with what lies behind it
@pytest.mark.parametrize("M,N,K", [(1, 1, 4), (3, 17, 20), (31, 63, 252), (33, 65, 260), (129, 641, 2564),
                                   (65, 127, 260), (97, 129, 516), (7, 255, 16384), (9, 257, 16384),
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


# --------------------------------------------------------------------- rows far from zero

def norm_back_xh(dy, x64, w, mean, rstd):
    """dx, dweight in 64 bits and the sizes that roundings relative to xh are counted against."""
    dy, w, mean, rstd = dy.double(), w.double(), mean.double(), rstd.double()
    xh = (x64 - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    size = rstd[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) +
                            xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), size, (dy * xh).abs().sum(0)


# xh = (x - mean) * rstd has one rounding in the difference and one in the product, relative to
# xh itself; from codes (c - a mean) (rstd / a) has three.  Its terms of dweight then add up
# along a path under 128: 131 u.  dx: 64 for a path, g, 3 for xh, 1 / K, two products, xh again
# and the last two sums: under 80 u.  Nothing is relative to the mean.
@pytest.mark.parametrize("K", [252, 1028, 2560, 8192, 14336, 20000])
@pytest.mark.parametrize("kind", ["bf16", "pow2", "absmax"])
def test_norm_backward_far_from_zero(K, kind):
    M = 6
    x = bf16(M, K, seed=K, hot=False)
    for m, shift in enumerate((0.0, 5.0, -50.0, 500.0, 8000.0)):
        x[m] += shift
    x[5] = 3.0
    dy = bf16(M, K, seed=K + 1, scale=1e-3)
    w = f32(K, seed=1, scale=0.2, shift=1.0)
    mean = x.double().mean(1).float()
    rstd = ((x.double() - mean.double()[:, None]).square().mean(1) + 1e-5).rsqrt().float()
    scale = None
    x64, arg = x.double(), x
    if kind != "bf16":
        arg, scale = (bw.quant_act_pow2 if kind == "pow2" else bw.quant_act)(x)
        x64 = arg.double() / scale.double()[:, None]
    for rows in ([0], [1], [2], [3], [4], [5], list(range(M))):
        r = torch.tensor(rows, device="cuda")
        s = None if scale is None else scale[r]
        dx, dw, _ = bw.layernorm_backward(dy[r], arg[r], w, mean[r], rstd[r], x_scale=s)
        rx, rw, size, sw = norm_back_xh(dy[r], x64[r], w, mean[r], rstd[r])
        close(dx, rx, BF * rx.abs() + (1 + BF) * 80 * U * size + TINY, f"{K} {kind} {rows} dx")
        close(dw, rw, 131 * U * sw + TINY, f"{K} {kind} {rows} dweight")


# ---------------------------------------------------------------- values that are not finite

def with_values(M, N, seed):
    """Rows holding an infinity, a negative one, a NaN, all of them, and the largest number."""
    x = bf16(M, N, seed=seed)
    inf = float("inf")
    for m, values in enumerate(([inf], [-inf], [float("nan")], [inf, -inf, float("nan")], [3.38e38])):
        x[m, torch.arange(len(values)) * 2 + 1] = torch.tensor(values, dtype=torch.bfloat16, device="cuda")
    return x


@pytest.mark.parametrize("N", [12, 252, 2560, 6912, 33000])
def test_fused_codes_are_the_separate_ones_where_values_are_not_finite(N):
    g, u = with_values(7, N, 1), with_values(7, N, 2).flip(0).contiguous()
    h, (gq, uq, gs, us) = bw.swiglu(g, u, checkpoint=True)
    same = lambda p, q: torch.equal(p.view(torch.int32), q.view(torch.int32))  # NaN scales too
    for q, s, t in ((gq, gs, g), (uq, us, u)):
        q2, s2 = bw.quant_act_pow2(t)
        assert torch.equal(q, q2) and same(s, s2)
    for scale, f in (("absmax", bw.quant_act), ("pow2", bw.quant_act_pow2)):
        hq, hs = bw.swiglu_quant(g, u, scale=scale)
        q2, s2 = f(h)
        assert torch.equal(hq, q2) and same(hs, s2), scale
        x = with_values(7, N, 3)
        y = bw.layernorm(x)
        xq, a = bw.layernorm_quant(x, scale=scale)
        q2, s2 = f(y)
        assert torch.equal(xq, q2) and same(a, s2), scale


@pytest.mark.parametrize("N", [12, 1024, 2560])
def test_an_infinity_is_not_restored_as_a_number(N):
    # the largest code times the smallest step: beyond bf16's range again
    x = with_values(7, N, 4)
    for q, s in (bw.quant_act_pow2(x), bw.swiglu(x, torch.ones_like(x), checkpoint=True)[1][::2]):
        back = bw.dequant_act(q, s)
        assert back[0, 1] == float("inf") and back[1, 1] == -float("inf")


def ref_codes(x, a):
    """The documented order of a code: product, round half even, clamp (NaN: the lower end)."""
    r = torch.round(x.float() * a[:, None])
    return torch.where(torch.isnan(r), torch.full_like(r, -127.0), r.clamp(-127, 127)).to(torch.int8)


@pytest.mark.parametrize("M,K", [(7, 12), (7, 2560), (600, 1024), (1100, 260), (7, 20004), (2000, 14336)])
def test_codes_of_both_scales_and_of_the_tensor(M, K):
    x = with_values(M, K, K)
    for f in (bw.quant_act, bw.quant_act_pow2, bw.quant_act_per_tensor):
        q, a = f(x)
        assert torch.equal(q, ref_codes(x, a)), f.__name__
        tail = x[5:].clone()
        q, a = f(tail)
        assert torch.equal(q, ref_codes(tail, a)) and torch.isfinite(a).all(), f.__name__


@pytest.mark.parametrize("M,N,K", [(5, 16, 64), (33, 65, 260), (512, 2560, 2560), (2048, 4096, 14336)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weight_gradient_shows_a_token_that_is_not_finite(M, N, K, value):
    # the absmax scale of a token with a NaN is NaN, with an infinity 0: neither may pass
    # for a token of zeros
    dy = bf16(M, N, seed=1, scale=1e-3, hot=False)
    dy[M - 1] = 1e-3
    x = bf16(M, K, seed=2)
    x[M - 1, ::7] = value
    xq, a = bw.quant_act(x)
    dw = bw.grad_weight(dy, xq, a)
    seen = torch.arange(K, device="cuda") % 7 == 0
    if value == float("inf"):
        assert a[M - 1] == 0
        assert torch.isinf(dw[:, seen]).all() and torch.isfinite(dw[:, ~seen]).all()
    else:
        assert torch.isnan(a[M - 1]) and torch.isnan(dw).all()


# ------------------------------------------------------------------- more rows than one launch

def in_parts(f, args, rows):
    """f over blocks of rows, joined."""
    outs = [f(*[a[i: i + rows] for a in args]) for i in range(0, args[0].shape[0], rows)]
    return [torch.cat(p) for p in zip(*[o if isinstance(o, tuple) else (o,) for o in outs])]


def noise(M, K, seed):
    """bf16 rows of any size, quickly: bits of a counter scrambled, exponents near 1."""
    i = torch.arange(M * K, dtype=torch.int32, device="cuda").mul_(-1640531527).add_(seed)
    return ((i >> 16).to(torch.int16) & -28673 | 0x3000).view(torch.bfloat16).view(M, K)


# 2^32 threads are the limit of a launch: 2^24 blocks of 256
@pytest.mark.parametrize("K", [4, 8])
def test_rows_past_one_launch(K):
    M, part = (1 << 24) + 1029, 1 << 22
    x, u, dh = noise(M, K, 1), noise(M, K, 2), noise(M, K, 3)
    q, a = bw.quant_act_pow2(x)
    assert torch.equal(bw.dequant_act(q, a), in_parts(bw.dequant_act, (q, a), part)[0])
    dg, du = bw.swiglu_backward(dh, x, u)
    for got, want in zip((dg, du), in_parts(bw.swiglu_backward, (dh, x, u), part)):
        assert torch.equal(got, want)
    uq, us = bw.quant_act_pow2(u)
    dg, du = bw.swiglu_backward(dh, q, uq, a, us)
    for got, want in zip((dg, du), in_parts(bw.swiglu_backward, (dh, q, uq, a, us), part)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("f", [bw.quant_act, bw.quant_act_pow2, bw.quant_act_per_tensor])
def test_quantized_rows_past_one_launch(f):
    # four rows a block
    M, K = (1 << 26) + 1029, 4
    x = noise(M, K, 5)
    q, a = f(x)
    if f is bw.quant_act_per_tensor:
        scale = torch.tensor(127.0) / x.float().abs().max().cpu()  # divided on the CPU, rounded once
        assert torch.equal(a, scale.cuda().expand(M)) and torch.equal(q, ref_codes(x, a))
    else:
        want = in_parts(f, (x,), 1 << 24)
        assert torch.equal(q, want[0]) and torch.equal(a, want[1])


# ----------------------------------------------------------------- automatic differentiation

def test_inputs_that_want_a_gradient_are_refused():
    # the results carry no graph: a gradient would stop here without a word
    M, K, N = 4, 64, 16
    x, q = bf16(M, K, seed=1), torch.ones((M, K), dtype=torch.int8, device="cuda")
    dy, s = bf16(M, N, seed=2), torch.ones(M, device="cuda")
    w, (p, ws) = torch.ones(K, device="cuda"), ternary(N, K)
    want = lambda t: t.clone().requires_grad_()
    calls = [
        (lambda: bw.quant_act_pow2(want(x)), lambda: bw.quant_act_pow2(x)),
        (lambda: bw.dequant_act(q, want(s)), lambda: bw.dequant_act(q, s)),
        (lambda: bw.layernorm(want(x)), lambda: bw.layernorm(x)),
        (lambda: bw.layernorm(x, want(w)), lambda: bw.layernorm(x, w)),
        (lambda: bw.layernorm(x, torch.nn.Parameter(w), w), lambda: bw.layernorm(x, w, w)),
        (lambda: bw.layernorm_quant(x, w, want(w)), lambda: bw.layernorm_quant(x, w, w)),
        (lambda: bw.layernorm_backward(x, want(x), w, s, s), lambda: bw.layernorm_backward(x, x, w, s, s)),
        (lambda: bw.swiglu(want(x), x), lambda: bw.swiglu(x, x)),
        (lambda: bw.swiglu_quant(x, want(x)), lambda: bw.swiglu_quant(x, x)),
        (lambda: bw.swiglu_backward(want(x), x, x), lambda: bw.swiglu_backward(x, x, x)),
        (lambda: bw.grad_input(want(dy), p, ws), lambda: bw.grad_input(dy, p, ws)),
        (lambda: bw.grad_weight(want(dy), q, s), lambda: bw.grad_weight(dy, q, s)),
        (lambda: bw.bitlinear_backward(dy, q, s, p, want(ws)),
         lambda: bw.bitlinear_backward(dy, q, s, p, ws)),
    ]
    flat = lambda r: [r] if isinstance(r, torch.Tensor) else [
        t for v in r if v is not None for t in flat(v)]
    for bad, good in calls:
        with pytest.raises(ValueError, match="requires grad"):
            bad()
        with torch.no_grad():
            got = flat(bad())
        want_bits = flat(good())
        assert len(got) == len(want_bits) and all(torch.equal(g, r) for g, r in zip(got, want_bits))


def test_as_functions_of_automatic_differentiation():
    # the calls as a user wraps them: both passes of a Function run without a graph
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, mean, rstd = bw.layernorm(x, w, b, return_stats=True)
            ctx.save_for_backward(x, w, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            return bw.layernorm_backward(dy.contiguous(), *ctx.saved_tensors)

    K = 260
    x, dy = bf16(9, K, seed=1), bf16(9, K, seed=2)
    w, b = f32(K, seed=3, shift=1.0), f32(K, seed=4)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = Norm.apply(*leaves)
    y.backward(dy)
    y0, mean, rstd = bw.layernorm(x, w, b, return_stats=True)
    assert torch.equal(y, y0)
    for leaf, g in zip(leaves, bw.layernorm_backward(dy, x, w, mean, rstd)):
        assert torch.equal(leaf.grad, g)


# ------------------------------------------------------------------ every compiled gradient kernel

# (M, K, Ns) and (M, N, K): each tile, with whole rows, odd ones and (dw) odd ends in a single
# column of tiles; all of these split the sum, and run unsplit without their workspace.
# test_train_plans.py holds the list against the plans and the table of tiles.
DX_TILES = [(1, 176, [1248]), (1, 136, [1347]), (33, 4912, [10120]), (36, 1436, [24747]), (1636, 592, [8784]),
            (4271, 148, [4456]), (199, 19696, [2368]), (4637, 156, [7698])]
DW_TILES = [(334, 60, 144), (478, 63, 136), (401, 65, 144), (1909, 60, 148), (2032, 65, 200), (3249, 67, 144),
            (2956, 134, 11200), (2069, 18479, 148), (3441, 143, 12168)]


@pytest.mark.parametrize("M,K,Ns", DX_TILES + [(520, 2052, [4097]), (2048, 4096, [1000, 3001])])
def test_input_gradient_of_every_kernel(M, K, Ns):
    big = [bf16(M + 1, n, seed=n + i, scale=1e-3, hot=False) for i, n in enumerate(Ns)]
    packs, scales = zip(*[ternary(n, K, seed=n + i) for i, n in enumerate(Ns)])
    for t in big:
        t[M] = float("nan")  # behind the rows
    dys = [t[:M] for t in big]
    for workspace in (None, False):
        got = bw.grad_input_grouped(dys, packs, scales, workspace=workspace)
        check_grad_input(dys, packs, scales, K, got, f"{M} {K} {Ns} {workspace}")


@pytest.mark.parametrize("M,N,K", DW_TILES + [(2048, 4096, 14336), (2047, 4097, 14340)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_weight_gradient_of_every_kernel(M, N, K, dt):
    big = bf16(M + 1, N, seed=N, scale=1e-3, hot=False)
    big[M] = float("nan")
    xq, a = bw.quant_act_pow2(bf16(M, K, seed=K))
    for workspace in (None, False):
        got = bw.grad_weight(big[:M], xq, a, out_dtype=dt, workspace=workspace)
        check_grad_weight(big[:M], xq, a, dt, got, f"{M} {N} {K} {dt} {workspace}")


def test_stream_and_device_getters(monkeypatch):
    # the short cuts give what torch's public functions give, and those serve in their place
    from ternary_weight_linear_token_amd import _binding
    x = bf16(5, 260, seed=1)
    want = bw.layernorm(x)
    public_stream = lambda index: torch.cuda.current_stream(index).cuda_stream
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert _binding._raw_stream(x.device.index) == stream.cuda_stream == public_stream(x.device.index)
    assert _binding._raw_device() == torch.cuda.current_device()
    monkeypatch.setattr(_binding, "_raw_stream", public_stream)
    monkeypatch.setattr(_binding, "_raw_device", torch.cuda.current_device)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bw.layernorm(x)
    side.synchronize()
    assert torch.equal(got, want)
