"""The training side of a BitLinear layer on the GPU against plain 64-bit forms.

Tolerances count roundings, u = 2^-24 for fp32 and 2^-8 for bf16 (half a step relative to
the value).  A sum of n fp32 terms whatever their order is off by at most (adds on the
longest path) * u * sum |terms|; the paths of the row kernels (at most 20 terms a lane, six
lane steps, 16 waves) are under 64 long, those of the column sums under 128."""
import numpy as np
import pytest
import torch

import ternary_weight_linear_token_amd as bw

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
TINY = 2.0 ** -120


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(*shape, seed=0, scale=1.0, shift=0.0, hot=True):
    g = gen(seed)
    x = torch.randn(*shape, generator=g) * scale + shift
    if hot and shape[-1] > 8:
        x[..., torch.randperm(shape[-1], generator=g)[: max(1, shape[-1] // 100)]] *= 20.0
    return x.to(torch.bfloat16).cuda()


def f32(*shape, seed=0, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale + shift).cuda()


def ternary(N, K, seed=0):
    w = 0.02 * torch.randn(N, K, generator=gen(seed))
    return bw.pack_weights(w.cuda())


def weights64(packed, w_scale, K):
    return bw.unpack_weights(packed, K).double() * w_scale.double()[:, None]


def pow2_of(amax):
    """2^floor(log2(127 / max(amax, 1e-5))), by exact comparisons."""
    out = []
    for v in amax.double().clamp(min=1e-5).tolist():
        p = int(np.floor(np.log2(127.0 / v)))
        while v * 2.0 ** (p + 1) <= 127.0:
            p += 1
        while v * 2.0 ** p > 127.0:
            p -= 1
        out.append(2.0 ** p)
    return torch.tensor(out, dtype=torch.float64, device=amax.device)


def close(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    assert bool((over <= 0).all()), (
        f"{what}: {int((over > 0).sum())} of {over.numel()} beyond, worst by {over.max().item():.3g}")


# ------------------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("M,K", [(1, 4), (3, 12), (5, 252), (2, 2564), (33, 4096), (2, 20004),
                                 (1500, 640)])
def test_pow2_codes_are_exact(M, K):
    x = bf16(M, K, seed=M + K)
    if M > 2:
        x[0] = 0
        x[1] *= 1e-6
        x[2] *= 1e20
    xq, a = bw.quant_act_pow2(x)
    want = pow2_of(x.double().abs().amax(1))
    assert torch.equal(a.double(), want)
    assert torch.equal(xq.double(), torch.round(x.double() * want[:, None]))
    back = bw.dequant_act(xq, a)
    assert torch.equal(back.double(), xq.double() / want[:, None])


def test_pow2_scale_at_its_borders():
    # 127 * 2^e is the last maximum with its exponent; the next bf16 value takes half the scale
    vals = [127.0, 127.5, 128.0, 63.5, 63.75, 64.0, 1.984375, 1.9921875, 2.0, 1e-5, 1.5e-5, 1.6e-5,
            2.0 ** -126, 3e38]
    x = torch.zeros((len(vals), 8), dtype=torch.bfloat16)
    x[:, 3] = -torch.tensor(vals).to(torch.bfloat16)
    x = x.cuda()
    xq, a = bw.quant_act_pow2(x)
    want = pow2_of(x.double().abs().amax(1))
    assert torch.equal(a.double(), want)
    assert torch.equal(xq.double(), torch.round(x.double() * want[:, None]))


def test_dequant_of_absmax_codes():
    x = bf16(17, 2560, seed=1)
    xq, a = bw.quant_act(x)
    ref = xq.double() / a.double()[:, None]
    # the reciprocal and the product round once each in fp32, (1 + u)^2 < 1 + 3 u, then bf16
    close(bw.dequant_act(xq, a), ref, (BF * (1 + 3 * U) + 3 * U) * ref.abs(), "dequant")


# -------------------------------------------------------------------------- layer norm

NORM_K = [4, 8, 60, 252, 1024, 1028, 2048, 2564, 4096, 4100, 8192, 8196, 16384, 16388, 20000]


def norm64(x, w, b, eps=1e-5):
    x = x.double()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = (xc.square().mean(1) + eps) ** -0.5
    K = x.shape[1]
    w = torch.ones(K, device=x.device) if w is None else w
    b = torch.zeros(K, device=x.device) if b is None else b
    return xc * rstd[:, None] * w.double() + b.double(), mean, rstd


def check_norm(x, w, b, y, mean, rstd, what):
    ref, m64, r64 = norm64(x, w, b)
    big = x.double().abs().amax(1)
    tol_mean = 64 * U * big
    close(mean, m64, tol_mean, what + " mean")
    rel_r = 64 * U + (tol_mean * r64) ** 2
    close(rstd, r64, rel_r * r64, what + " rstd")
    wa = 1.0 if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    # xh: the mean's error and one subtraction, then rstd's and three more roundings
    xh = (x.double() - m64[:, None]).abs() * r64[:, None]
    tol = ((tol_mean + 2 * U * big) * r64)[:, None] + xh * (rel_r[:, None] + 4 * U)
    close(y, ref, BF * ref.abs() + (1 + BF) * (tol * wa + 2 * U * (xh * wa + ba)), what + " y")


@pytest.mark.parametrize("K", NORM_K)
@pytest.mark.parametrize("M", [1, 5])
def test_layernorm_forward(M, K):
    x = bf16(M, K, seed=K, shift=0.5)
    if M > 2:
        x[1] = 0          # a row without variance: y = bias
        x[2] = 3.0
    w, b = f32(K, seed=1, scale=0.2, shift=1.0), f32(K, seed=2)
    y, mean, rstd = bw.layernorm(x, w, b, return_stats=True)
    check_norm(x, w, b, y, mean, rstd, f"{M}x{K}")
    if M > 2:
        assert torch.equal(y[1], b.to(torch.bfloat16))
    y, mean, rstd = bw.layernorm(x, return_stats=True)
    check_norm(x, None, None, y, mean, rstd, f"{M}x{K} plain")
    assert torch.equal(bw.layernorm(x), y)


def test_layernorm_far_from_zero():
    # mean 500 times the spread: the variance from squared differences keeps its digits
    x = bf16(3, 2560, seed=3, scale=1.0, shift=500.0, hot=False)
    y, mean, rstd = bw.layernorm(x, return_stats=True)
    check_norm(x, None, None, y, mean, rstd, "offset")


@pytest.mark.parametrize("M,K", [(10000, 512), (5000, 1536), (2100, 2560), (1030, 8192)])
def test_layernorm_blocks_take_several_rows(M, K):
    x = bf16(M, K, seed=4, shift=-0.25)
    w, b = f32(K, seed=1, shift=1.0), f32(K, seed=2)
    y, mean, rstd = bw.layernorm(x, w, b, return_stats=True)
    check_norm(x, w, b, y, mean, rstd, f"{M}x{K}")


@pytest.mark.parametrize("K", [4, 252, 1028, 2560, 8196, 16384, 20000])
@pytest.mark.parametrize("scale", ["absmax", "pow2"])
def test_layernorm_codes_are_those_of_y(K, scale):
    x = bf16(6, K, seed=K)
    x[3] = 0
    w, b = f32(K, seed=1, shift=1.0), f32(K, seed=2)
    y0 = bw.layernorm(x, w, b)
    xq, a, y, mean, rstd = bw.layernorm_quant(x, w, b, scale=scale, return_y=True, return_stats=True)
    assert torch.equal(y, y0)
    q2, a2 = bw.quant_act(y0) if scale == "absmax" else bw.quant_act_pow2(y0)
    assert torch.equal(a, a2) and torch.equal(xq, q2)
    q3, a3 = bw.layernorm_quant(x, w, b, scale=scale)
    assert torch.equal(q3, q2) and torch.equal(a3, a2)


def norm_back64(dy, x, w, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double(), rstd.double()
    w = torch.ones(x.shape[1], device=x.device).double() if w is None else w.double()
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - m1 - xh * m2)
    # sizes that the roundings are relative to
    xa = (x.abs() + mean.abs()[:, None]) * rstd[:, None]
    size = rstd[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) +
                            xa * (g.abs() * xa).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), size, (dy.abs() * xa).sum(0), dy.abs().sum(0)


def check_norm_back(dy, x, x64, w, mean, rstd, x_scale, what):
    dx, dw, db = bw.layernorm_backward(dy, x, w, mean, rstd, x_scale=x_scale)
    rx, rw, rb, size, sw, sb = norm_back64(dy, x64, w, mean, rstd)
    close(dx, rx, BF * rx.abs() + 72 * U * size + TINY, what + " dx")
    close(dw, rw, 136 * U * sw + TINY, what + " dweight")
    close(db, rb, 128 * U * sb + TINY, what + " dbias")
    again = bw.layernorm_backward(dy, x, w, mean, rstd, x_scale=x_scale)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again)), what + ": not the same twice"


@pytest.mark.parametrize("K", NORM_K)
@pytest.mark.parametrize("M", [1, 37])
@pytest.mark.parametrize("ckpt", [False, True])
def test_layernorm_backward(M, K, ckpt):
    x = bf16(M, K, seed=K, shift=0.5)
    if M > 2:
        x[1] = 0
    dy = bf16(M, K, seed=K + 1, scale=1e-3)
    w = f32(K, seed=1, scale=0.2, shift=1.0)
    _, mean, rstd = bw.layernorm(x, w, None, return_stats=True)
    if ckpt:
        q, a = bw.quant_act_pow2(x)
        check_norm_back(dy, q, q.double() / a.double()[:, None], w, mean, rstd, a, f"{M}x{K} ckpt")
    else:
        check_norm_back(dy, x, x, w, mean, rstd, None, f"{M}x{K}")
        check_norm_back(dy, x, x, None, mean, rstd, None, f"{M}x{K} no weight")


@pytest.mark.parametrize("M,K", [(9001, 512), (3000, 1024), (2500, 2560), (1300, 8192), (700, 16380),
                                 (2200, 17000)])
def test_layernorm_backward_many_rows(M, K):
    x = bf16(M, K, seed=7)
    dy = bf16(M, K, seed=8)
    w = f32(K, seed=1, shift=1.0)
    _, mean, rstd = bw.layernorm(x, return_stats=True)
    check_norm_back(dy, x, x, w, mean, rstd, None, f"{M}x{K}")


def test_layernorm_backward_absmax_codes():
    # 1 / a is rounded once in fp32 where a is no power of two: one more u on x
    x, dy = bf16(40, 2560, seed=9), bf16(40, 2560, seed=10)
    q, a = bw.quant_act(x)
    _, mean, rstd = bw.layernorm(x, return_stats=True)
    check_norm_back(dy, q, q.double() / a.double()[:, None], None, mean, rstd, a, "absmax codes")


def test_layernorm_backward_empty_and_partial():
    K = 260
    e = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    s = torch.empty((0,), device="cuda")
    dx, dw, db = bw.layernorm_backward(e, e, None, s, s)
    assert dx.shape == (0, K) and not dw.any() and not db.any()
    assert bw.layernorm(e).shape == (0, K)
    x, dy = bf16(5, K, seed=1), bf16(5, K, seed=2)
    _, mean, rstd = bw.layernorm(x, return_stats=True)
    full = bw.layernorm_backward(dy, x, None, mean, rstd)
    dx, dw, db = bw.layernorm_backward(dy, x, None, mean, rstd, need_sums=False)
    assert torch.equal(dx, full[0]) and dw is None and db is None


def test_layernorm_gradient_against_differences():
    # central differences of the 64-bit forward along random directions: the kernel's dx is
    # bf16, so <dx, v> is within BF * sum |dx v|; the difference's own error is far smaller
    M, K, h = 7, 516, 1e-4
    x, dy = bf16(M, K, seed=1, hot=False), bf16(M, K, seed=2)
    w, b = f32(K, seed=3, shift=1.0), f32(K, seed=4)
    _, mean, rstd = bw.layernorm(x, w, b, return_stats=True)
    dx, dw, db = bw.layernorm_backward(dy, x, w, mean, rstd)
    loss = lambda xx, ww, bb: (norm64(xx, ww, bb)[0] * dy.double()).sum()
    for seed in range(3):
        v = torch.randn(M, K, generator=gen(seed)).double().cuda()
        num = (loss(x.double() + h * v, w, b) - loss(x.double() - h * v, w, b)) / (2 * h)
        tol = BF * (dx.double() * v).abs().sum() + 1e-5 * num.abs()
        assert (num - (dx.double() * v).sum()).abs() <= tol
        v = torch.randn(K, generator=gen(seed)).double().cuda()
        num = (loss(x, w.double() + h * v, b) - loss(x, w.double() - h * v, b)) / (2 * h)
        assert (num - (dw.double() * v).sum()).abs() <= 1e-5 * (dw.double() * v).abs().sum()
        num = (loss(x, w, b.double() + h * v) - loss(x, w, b.double() - h * v)) / (2 * h)
        assert (num - (db.double() * v).sum()).abs() <= 1e-5 * (db.double() * v).abs().sum()


# ------------------------------------------------------------------------------ SwiGLU

GLU_N = [4, 12, 252, 256, 1020, 2048, 2052, 6912, 8196, 14336, 28672, 32772]


def check_swiglu(g, u, h, what):
    gd, ud = g.double(), u.double()
    ref = gd * torch.sigmoid(gd) * ud
    # exp(-g): its argument -g log2(e) is rounded to |g| u, two more for exp2 and the
    # reciprocal's 1 ulp each (2 u), and three products
    close(h, ref, BF * ref.abs() + (2 * gd.abs() + 12) * U * ref.abs() + TINY * (1 + ud.abs()), what)


@pytest.mark.parametrize("N", GLU_N)
@pytest.mark.parametrize("M", [1, 6])
def test_swiglu_forward(M, N):
    g, u = bf16(M, N, seed=N, scale=3.0), bf16(M, N, seed=N + 1)
    if M > 2:
        g[1], u[1] = 0, 0
        g[2] *= 4
    h, (gq, uq, gs, us) = bw.swiglu(g, u, checkpoint=True)
    check_swiglu(g, u, h, f"{M}x{N}")
    for q, s, t in ((gq, gs, g), (uq, us, u)):
        q2, s2 = bw.quant_act_pow2(t)
        assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(bw.swiglu(g, u), h)
    for scale in ("absmax", "pow2"):
        hq, hs, h2, ck = bw.swiglu_quant(g, u, scale=scale, return_h=True, checkpoint=True)
        q2, s2 = bw.quant_act(h) if scale == "absmax" else bw.quant_act_pow2(h)
        assert torch.equal(h2, h) and torch.equal(hq, q2) and torch.equal(hs, s2)
        assert all(torch.equal(p, q) for p, q in zip(ck, (gq, uq, gs, us)))
        hq2, hs2 = bw.swiglu_quant(g, u, scale=scale)
        assert torch.equal(hq2, hq) and torch.equal(hs2, hs)


def test_swiglu_many_rows():
    g, u = bf16(9000, 640, seed=1), bf16(9000, 640, seed=2)
    h, (gq, uq, gs, us) = bw.swiglu(g, u, checkpoint=True)
    check_swiglu(g, u, h, "9000x640")
    q2, s2 = bw.quant_act_pow2(u)
    assert torch.equal(uq, q2) and torch.equal(us, s2)


def check_swiglu_back(dh, g, u, dg, du, what):
    d, g, u = dh.double(), g.double(), u.double()
    s = torch.sigmoid(g)
    rg, ru = d * u * s * (1 + g * (1 - s)), d * g * s
    rel = (2 * g.abs() + 12) * U  # of s, as in the forward
    # 1 - s and 1 + g (1 - s) may cancel: s's error counts against s (1 + |g|)
    size = (d * u).abs() * s * (1 + g.abs())
    close(dg, rg, BF * rg.abs() + (1 + BF) * (2 * rel + 6 * U) * size + TINY * (1 + (d * u).abs()), what + " dg")
    close(du, ru, BF * ru.abs() + (rel + 4 * U) * ru.abs() + TINY * (1 + d.abs()), what + " du")


@pytest.mark.parametrize("N", [4, 12, 252, 2048, 2052, 6912, 32772])
@pytest.mark.parametrize("M", [1, 7])
def test_swiglu_backward(M, N):
    g, u, dh = bf16(M, N, seed=N, scale=3.0), bf16(M, N, seed=N + 1), bf16(M, N, seed=5, scale=1e-3)
    if M > 2:
        g[1] = 0
        g[2] *= 4
    check_swiglu_back(dh, g, u, *bw.swiglu_backward(dh, g, u), f"{M}x{N} bf16")
    _, (gq, uq, gs, us) = bw.swiglu(g, u, checkpoint=True)
    dg, du = bw.swiglu_backward(dh, gq, uq, gs, us)
    check_swiglu_back(dh, gq.double() / gs.double()[:, None], uq.double() / us.double()[:, None], dg,
                      du, f"{M}x{N} ckpt")


def test_swiglu_extremes():
    # exp overflows or vanishes: silu(g) is 0 or g, and nothing is NaN
    g = torch.tensor([[-3e38, -1e4, -90.0, -1.0, 0.0, 1.0, 90.0, 1e4]], dtype=torch.bfloat16).cuda()
    u, dh = torch.ones_like(g), torch.ones_like(g)
    check_swiglu(g[:, 1:], u[:, 1:], bw.swiglu(g, u)[:, 1:], "extremes")
    h, (dg, du) = bw.swiglu(g, u), bw.swiglu_backward(dh, g, u)
    assert h[0, 0] == 0 and du[0, 0] == 0 and dg[0, 0] == 0 and dg[0, 7] == 1
    check_swiglu_back(dh[:, 1:], g[:, 1:], u[:, 1:], dg[:, 1:], du[:, 1:], "extremes")


def test_swiglu_gradient_against_differences():
    g, u, dh = (bf16(3, 60, seed=s, hot=False) for s in (1, 2, 3))
    dg, du = bw.swiglu_backward(dh, g, u)
    f = lambda gg, uu: (gg * torch.sigmoid(gg) * uu * dh.double()).sum()
    h = 1e-5
    v = torch.randn(3, 60, generator=gen(4)).double().cuda()
    num = (f(g.double() + h * v, u.double()) - f(g.double() - h * v, u.double())) / (2 * h)
    assert (num - (dg.double() * v).sum()).abs() <= 1.01 * BF * (dg.double() * v).abs().sum() + 1e-7
    num = (f(g.double(), u.double() + h * v) - f(g.double(), u.double() - h * v)) / (2 * h)
    assert (num - (du.double() * v).sum()).abs() <= 1.01 * BF * (du.double() * v).abs().sum() + 1e-7


# --------------------------------------------------------------------- product gradients

def check_grad_input(dys, packs, scales, K, got, what):
    """Against the sum of the kernel's operands (dy * s rounded to bf16, w) in 64 bits:
    what remains is the fp32 sum and the output's rounding; and against the exact sum."""
    ref = exact = size = 0.0
    n = 0
    for dy, p, s in zip(dys, packs, scales):
        w = bw.unpack_weights(p, K).double()
        a = (dy.float() * s).to(torch.bfloat16).double()
        ref = ref + a @ w
        size = size + a.abs() @ w.abs()
        exact = exact + (dy.double() * s.double()) @ w
        n += dy.shape[1]
    close(got, ref, BF * ref.abs() + (n + 64) * U * size + TINY, what)
    # each dy * s is off by at most BF of itself
    close(got, exact, BF * exact.abs() + (BF + (n + 64) * U) * size * (1 + BF) + TINY, what + " exact")


# M, K, Ns: every tile configuration, with and without slices, odd row lengths (two-byte
# loads), columns off the 16-weight words, groups that end inside a step
GRAD_INPUT = [(1, 4, [1]), (1, 2560, [2560]), (3, 20, [17]), (4, 2560, [2560]), (16, 4096, [640]),
              (31, 252, [63]), (33, 256, [64]), (40, 1024, [2561]), (64, 2560, [640, 640]),
              (129, 2564, [641]), (200, 640, [100, 33, 7, 1]), (300, 260, [1000]),
              (512, 2560, [2560, 640, 640]), (257, 6912, [514]), (520, 2048, [4096]),
              (1030, 4112, [1300, 1302]), (2048, 4096, [2048])]


@pytest.mark.parametrize("M,K,Ns", GRAD_INPUT)
def test_grad_input(M, K, Ns):
    dys = [bf16(M, n, seed=n + i, scale=1e-3, hot=False) for i, n in enumerate(Ns)]
    packs, scales = zip(*[ternary(n, K, seed=n + i) for i, n in enumerate(Ns)])
    got = bw.grad_input_grouped(dys, packs, scales)
    check_grad_input(dys, packs, scales, K, got, f"{M} {K} {Ns}")
    assert torch.equal(bw.grad_input_grouped(dys, packs, scales), got)
    plain = bw.grad_input_grouped(dys, packs, scales, workspace=False)
    check_grad_input(dys, packs, scales, K, plain, f"{M} {K} {Ns} unsplit")


def test_grad_input_one_group_and_empty():
    p, s = ternary(640, 1024)
    dy = bf16(10, 640, seed=1)
    one = bw.grad_input(dy, p, s)
    check_grad_input([dy], [p], [s], 1024, one, "one")
    e, pe, se = dy[:, :0].contiguous(), p[:0], s[:0]
    assert torch.equal(bw.grad_input_grouped([e, dy], [pe, p], [se, s]), one)
    assert not bw.grad_input(e, pe, se).any()
    assert bw.grad_input(dy[:0], p, s).shape == (0, 1024)


def test_grad_input_unused_code_is_zero():
    p, s = ternary(32, 64)
    dy = bf16(5, 32, seed=1)
    p2 = p.clone()
    p2[7] = 0xFF  # the unused code in the whole row
    p3 = p.clone()
    p3[7] = 0x55  # weight 0
    assert torch.equal(bw.grad_input(dy, p2, s), bw.grad_input(dy, p3, s))


def test_grad_input_does_not_read_past_the_rows():
    # an odd row length ends inside a 16-byte load: the neighbour row's values (here NaN
    # and infinity in the next tensor rows' place) must not enter
    M, N, K = 5, 33, 64
    p, s = ternary(N, K)
    dy = bf16(M, N, seed=3, hot=False)
    clean = bw.grad_input(dy, p, s)
    bad = dy.clone()
    bad[3] = float("nan")
    got = bw.grad_input(bad, p, s)
    keep = [0, 1, 2, 4]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[3]).all()


def check_grad_weight(dy, xq, a, dt, got, what):
    x = (xq.float() * (1.0 / a)[:, None]).to(torch.bfloat16).double()  # exact for powers of two
    d = dy.double().t().contiguous()
    ref, size = d @ x, d.abs() @ x.abs()
    tol = (dy.shape[0] + 64) * U * size + TINY
    if dt == "bf16":
        tol = (1 + BF) * tol + BF * ref.abs()
    close(got, ref, tol, what)


GRAD_WEIGHT = [(1, 1, 4), (1, 2560, 2560), (3, 17, 20), (16, 640, 2560), (31, 63, 252), (33, 64, 256),
               (64, 257, 1028), (129, 641, 2564), (333, 300, 516), (512, 2560, 2560), (512, 640, 2560),
               (1000, 130, 260), (2048, 128, 256), (4100, 33, 64), (700, 6912, 2560), (520, 4096, 4112)]


@pytest.mark.parametrize("M,N,K", GRAD_WEIGHT)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_grad_weight(M, N, K, dt):
    dy = bf16(M, N, seed=N, scale=1e-3, hot=False)
    xq, a = bw.quant_act_pow2(bf16(M, K, seed=K))
    got = bw.grad_weight(dy, xq, a, out_dtype=dt)
    check_grad_weight(dy, xq, a, dt, got, f"{M} {N} {K} {dt}")
    assert torch.equal(bw.grad_weight(dy, xq, a, out_dtype=dt), got)
    check_grad_weight(dy, xq, a, dt, bw.grad_weight(dy, xq, a, out_dtype=dt, workspace=False), "unsplit")


def test_grad_weight_absmax_codes():
    dy = bf16(100, 320, seed=1, hot=False)
    xq, a = bw.quant_act(bf16(100, 640, seed=2))
    check_grad_weight(dy, xq, a, "f32", bw.grad_weight(dy, xq, a), "absmax")


def test_grad_weight_empty():
    dy = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    xq = torch.empty((0, 68), dtype=torch.int8, device="cuda")
    a = torch.empty((0,), device="cuda")
    out = torch.full((40, 68), 7.0, device="cuda")
    assert not bw.grad_weight(dy, xq, a, out=out).any()
    dy, xq, a = bf16(3, 4, seed=1)[:, :0].contiguous(), *bw.quant_act_pow2(bf16(3, 68, seed=2))
    assert bw.grad_weight(dy, xq, a).shape == (0, 68)


def test_grad_weight_leaves_its_neighbours():
    # ragged output inside a larger buffer: nothing is written past it
    M, N, K = 50, 37, 132
    dy = bf16(M, N, seed=1)
    xq, a = bw.quant_act_pow2(bf16(M, K, seed=2))
    buf = torch.full((N * K + 64,), 3.0, device="cuda")
    bw.grad_weight(dy, xq, a, out=buf[: N * K].view(N, K))
    assert bool((buf[N * K:] == 3.0).all())
    dyi = bf16(N, 65, seed=3)
    p, s = ternary(65, K)
    buf = torch.full((N * K + 64,), 3.0, device="cuda", dtype=torch.bfloat16)
    bw.grad_input(dyi, p, s, out=buf[: N * K].view(N, K))
    assert bool((buf[N * K:] == 3.0).all())


def test_product_gradients_against_differences():
    # loss = sum dy * (x W^T) is bilinear: a difference along v is exact up to rounding
    M, N, K = 9, 130, 260
    x, dy = bf16(M, K, seed=1, hot=False), bf16(M, N, seed=2)
    p, s = ternary(N, K)
    xq, a = bw.quant_act_pow2(x)
    W, X = weights64(p, s, K), xq.double() / a.double()[:, None]
    dx, dw = bw.bitlinear_backward(dy, xq, a, p, s)
    loss = lambda xx, ww: ((xx @ ww.t()) * dy.double()).sum()
    v = torch.randn(M, K, generator=gen(3)).double().cuda()
    num = (loss(X + v, W) - loss(X - v, W)) / 2
    size = dy.double().abs() @ W.abs()
    assert (num - (dx.double() * v).sum()).abs() <= 2.1 * BF * (size * v.abs()).sum()
    v = torch.randn(N, K, generator=gen(4)).double().cuda()
    num = (loss(X, W + v) - loss(X, W - v)) / 2
    size = dy.double().abs().t().contiguous() @ X.abs()
    assert (num - (dw.double() * v).sum()).abs() <= (M + 64) * U * (size * v.abs()).sum()


def test_offsets_past_32_bits():
    # more than 2^31 elements: the last rows come out as they do alone
    M, N, K, T = 1_100_003, 2048, 64, 5
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    tail = bf16(T, N, seed=1, hot=False)
    dy[-T:] = tail
    xq = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    a = torch.ones((M,), device="cuda")
    tq, ta = bw.quant_act_pow2(bf16(T, K, seed=2))
    xq[-T:], a[-T:] = tq, ta
    # zero rows add exact zeros: the sum of five products in some order
    check_grad_weight(tail, tq, ta, "f32", bw.grad_weight(dy, xq, a), "dw")
    p, s = ternary(N, K)
    dx = bw.grad_input(dy, p, s)
    check_grad_input([tail], [p], [s], K, dx[-T:], "dx")
    assert not dx[:-T].any()
    del dx
    # dy as a norm's input, and as SwiGLU's
    y, mean, rstd = bw.layernorm(dy, return_stats=True)
    check_norm(tail, None, None, y[-T:], mean[-T:], rstd[-T:], "norm")
    assert not y[:-T].any()
    gx, gw, gb = bw.layernorm_backward(y, dy, None, mean, rstd)
    rx, rw, rb, size, sw, sb = norm_back64(y[-T:], tail, None, mean[-T:], rstd[-T:])
    close(gx[-T:], rx, BF * rx.abs() + 72 * U * size + TINY, "norm dx")
    # 1.1 million rows over 512 blocks: 2149 more additions, of zeros, on the path
    close(gw, rw, 136 * U * sw + TINY, "norm dweight")
    del gx, y
    h, (gq, uq, gs, us) = bw.swiglu(dy, dy, checkpoint=True)
    check_swiglu(tail, tail, h[-T:], "swiglu")
    dg, du = bw.swiglu_backward(dy, gq, uq, gs, us)
    v = gq[-T:].double() / gs[-T:].double()[:, None]
    check_swiglu_back(tail, v, v, dg[-T:], du[-T:], "swiglu backward")
    q, sc = bw.quant_act_pow2(dy)
    assert torch.equal(bw.dequant_act(q, sc)[-T:].double(), q[-T:].double() / sc[-T:].double()[:, None])


# ------------------------------------------------------------------- the set as it is used

def mlp_step(x, dy, w, b, gate, up, down, outs=None):
    """One training step through norm -> gate, up -> SwiGLU -> down and back."""
    xq, xa, mean, rstd = bw.layernorm_quant(x, w, b, scale="pow2", return_stats=True)
    g, u = bw.gemm_grouped(xq, xa, [gate[0], up[0]], [gate[1], up[1]], "bf16")
    hq, ha, ck = bw.swiglu_quant(g, u, scale="pow2", checkpoint=True)
    y = bw.gemm(hq, ha, *down, "bf16")
    dh, dw_down = bw.bitlinear_backward(dy, hq, ha, *down)
    dg, du = bw.swiglu_backward(dh, *ck)
    dw_gate, dw_up = bw.grad_weight(dg, xq, xa), bw.grad_weight(du, xq, xa)
    dxn = bw.grad_input_grouped([dg, du], [gate[0], up[0]], [gate[1], up[1]])
    dx, dgamma, dbeta = bw.layernorm_backward(dxn, x, w, mean, rstd)
    return y, dx, dgamma, dbeta, dw_gate, dw_up, dw_down


def mlp_inputs(M=96, H=512, F=1028, seed=0):
    x, dy = bf16(M, H, seed=seed, hot=False), bf16(M, H, seed=seed + 1, scale=1e-2, hot=False)
    w, b = f32(H, seed=2, scale=0.1, shift=1.0), f32(H, seed=3, scale=0.1)
    return x, dy, w, b, ternary(F, H, seed=4), ternary(F, H, seed=5), ternary(H, F, seed=6)


def test_mlp_training_step():
    x, dy, w, b, gate, up, down = mlp_inputs()
    y, *got = mlp_step(x, dy, w, b, gate, up, down)
    # the same step in 64 bits with straight-through quantizers, by automatic differentiation
    H, F = x.shape[1], gate[0].shape[0]

    class Round(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            a = pow2_of(t.abs().amax(1))[:, None]
            return torch.round(t * a) / a

        @staticmethod
        def backward(ctx, d):
            return d

    leaf = lambda t: t.detach().double().requires_grad_()
    x64, w64, b64 = leaf(x), leaf(w), leaf(b)
    wg, wu, wd = (leaf(weights64(p, s, k)) for (p, s), k in ((gate, H), (up, H), (down, F)))
    mean = x64.mean(1, keepdim=True)
    xh = (x64 - mean) * ((x64 - mean).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    xn = Round.apply(xh * w64 + b64)
    g, u = xn @ wg.t(), xn @ wu.t()
    out = Round.apply(g * torch.sigmoid(g) * u) @ wd.t()
    out.backward(dy.double())
    # bf16 activations between the stages and 8-bit g and u in the backward: 1/254 of a
    # row's maximum (some four standard deviations) per checkpointed value, twice, and
    # codes that fall to the other side; 5% in the 2-norm covers three such terms
    refs = [x64.grad, w64.grad, b64.grad, wg.grad, wu.grad, wd.grad]
    for k, (p, q) in enumerate(zip([y] + got, [out.detach()] + refs)):
        rel = ((p.double() - q).norm() / q.norm()).item()
        assert rel <= 0.05, f"output {k}: {rel:.3g}"


def test_mlp_training_step_in_graphs():
    # two captured steps of different sizes, replayed in turn with eager work between
    steps = []
    for M, seed in ((96, 0), (33, 50)):
        args = mlp_inputs(M=M, seed=seed)
        want = [t.clone() for t in mlp_step(*args)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            mlp_step(*args)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = mlp_step(*args)
        steps.append((args, want, graph, outs))
    for rep in range(3):
        for args, want, graph, outs in steps:
            for t in outs:
                t.zero_()
            graph.replay()
            eager = mlp_step(*args)
            torch.cuda.synchronize()
            for k, (p, q, r) in enumerate(zip(outs, want, eager)):
                assert torch.equal(p, q), f"replay {rep} output {k}"
                assert torch.equal(r, q), f"eager {rep} output {k}"
        # new inputs in the captured buffers
        args, want, graph, outs = steps[0]
        args[0].copy_(args[0].flip(0).clone())
        steps[0] = (args, [t.clone() for t in mlp_step(*args)], graph, outs)


def test_two_streams_at_once():
    args = [mlp_inputs(seed=s) for s in (0, 9)]
    want = [[t.clone() for t in mlp_step(*a)] for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for s, a in zip(streams, args):
        with torch.cuda.stream(s):
            got.append([mlp_step(*a) for _ in range(3)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for run in g:
            assert all(torch.equal(p, q) for p, q in zip(run, w))


def test_refusals_on_the_device():
    x = bf16(4, 256, seed=1)
    q, a = bw.quant_act_pow2(x)
    p, s = ternary(16, 256)
    with pytest.raises(TypeError):
        bw.layernorm(x.float())
    with pytest.raises(ValueError):
        bw.layernorm(x[:, ::2])                       # not contiguous
    with pytest.raises(ValueError):
        bw.layernorm(x, torch.ones(255, device="cuda"))
    with pytest.raises(ValueError):
        bw.layernorm(x, torch.ones(256))              # weight on the host
    with pytest.raises(bw.BitnetError):
        bw.layernorm(x, eps=0.0)
    with pytest.raises(TypeError):
        bw.layernorm_backward(x, q, None, a, a)       # codes without their scales
    with pytest.raises(bw.BitnetError):
        bw.layernorm_backward(x, x, None, a, a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        bw.swiglu_backward(x, q, q, a, None)
    with pytest.raises(ValueError):
        bw.grad_input(bf16(4, 17, seed=1), p, s)      # 16 rows of weights
    with pytest.raises(ValueError):
        bw.grad_weight(bf16(5, 16, seed=1), q, a)     # 4 tokens of codes
    with pytest.raises(ValueError):
        bw.grad_weight(bf16(4, 16, seed=1), q, a, out_dtype="i32")
