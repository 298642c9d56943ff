"""Root-mean-square norm (forward with the residual's addition and int8 codes, backward) and the
gradients' global norm and clipping on the GPU against plain 64-bit forms.

Tolerances count roundings: u = 2^-24 for fp32, 2^-8 for bf16 (half a step relative to the
value).  A sum of n fp32 terms is off by at most (additions on the longest path) * u * sum
|terms|; the paths of the row kernels (at most 20 terms a lane, six lane steps, 16 waves) are
under 64 long."""
import numpy as np
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_train import BF, TINY, U, bf16, close, f32, pow2_of

pytestmark = pytest.mark.gpu

EPS = 1e-5
NORM_K = [4, 8, 60, 252, 1024, 1028, 2048, 2564, 4096, 4100, 8192, 8196, 16384, 16388, 20000]


def rms64(s, w):
    s = s.double()
    rstd = (s.square().mean(1) + EPS) ** -0.5
    w = torch.ones(s.shape[1], device=s.device) if w is None else w
    return s * rstd[:, None] * w.double(), rstd


def check_rms(s, w, y, rstd, what):
    ref, r64 = rms64(s, w)
    # the sum's 64 roundings count half under the root; the root and its argument round once each
    close(rstd, r64, 64 * U * r64, what + " rstd")
    # the statistics', then two products, then bf16
    close(y, ref, (BF + (1 + BF) * 67 * U) * ref.abs() + TINY, what + " y")


@pytest.mark.parametrize("K", NORM_K)
@pytest.mark.parametrize("M", [1, 5])
def test_rmsnorm_forward(M, K):
    x, res = bf16(M, K, seed=K), bf16(M, K, seed=K + 1, scale=3.0, hot=False)
    if M > 2:
        x[1] = 0
        res[1] = 0        # a row of zeros: y = 0, rstd = eps^-1/2
        x[2], res[2] = 7.0, -7.0
    w = f32(K, seed=1, scale=0.2, shift=1.0)
    want = (x.float() + res.float()).to(torch.bfloat16)
    y, s, rstd = bw.rmsnorm(x, w, residual=res, return_stats=True)
    assert torch.equal(s, want)
    check_rms(s, w, y, rstd, f"{M}x{K} residual")
    if M > 2:
        assert not y[1].any() and not y[2].any()
    y2, rstd2 = bw.rmsnorm(s, w, return_stats=True)  # the norm of the stored sum
    assert torch.equal(y2, y) and torch.equal(rstd2, rstd)
    y, rstd = bw.rmsnorm(x, return_stats=True)
    check_rms(x, None, y, rstd, f"{M}x{K} plain")
    assert torch.equal(bw.rmsnorm(x), y)
    y, s2 = bw.rmsnorm(x, w, residual=res)
    assert torch.equal(s2, want) and torch.equal(y, y2)


@pytest.mark.parametrize("K", [4, 2564, 8192, 16388, 20000])
def test_sum_in_place(K):
    for which in range(2):
        x, res = bf16(5, K, seed=K), bf16(5, K, seed=K + 1)
        y, s = bw.rmsnorm(x, residual=res)
        t = (x, res)[which]
        y2, s2 = bw.rmsnorm(x, residual=res, sum_out=t)
        assert s2 is t and torch.equal(t, s) and torch.equal(y2, y)


@pytest.mark.parametrize("M,K", [(10000, 512), (5000, 1536), (2100, 2560), (1030, 8192), (520, 16384),
                                 (1030, 16400)])
def test_blocks_take_several_rows(M, K):
    x, res = bf16(M, K, seed=4), bf16(M, K, seed=5)
    w = f32(K, seed=1, shift=1.0)
    y, s, rstd = bw.rmsnorm(x, w, residual=res, return_stats=True)
    assert torch.equal(s, (x.float() + res.float()).to(torch.bfloat16))
    check_rms(s, w, y, rstd, f"{M}x{K}")
    xq, a, _ = bw.rmsnorm_quant(x, w, residual=res)
    q2, a2 = bw.quant_act(y)
    assert torch.equal(xq, q2) and torch.equal(a, a2)


@pytest.mark.parametrize("K", [4, 252, 1028, 2560, 8196, 16384, 20000])
@pytest.mark.parametrize("scale", ["absmax", "pow2"])
def test_codes_are_those_of_y(K, scale):
    x, res = bf16(6, K, seed=K), bf16(6, K, seed=K + 9)
    x[3] = 0
    res[3] = 0
    w = f32(K, seed=1, shift=1.0)
    y0, s0, r0 = bw.rmsnorm(x, w, residual=res, return_stats=True)
    xq, a, s, y, rstd = bw.rmsnorm_quant(x, w, residual=res, scale=scale, return_y=True,
                                         return_stats=True)
    assert torch.equal(y, y0) and torch.equal(s, s0) and torch.equal(rstd, r0)
    q2, a2 = bw.quant_act(y0) if scale == "absmax" else bw.quant_act_pow2(y0)
    assert torch.equal(a, a2) and torch.equal(xq, q2)
    q3, a3 = bw.rmsnorm_quant(s0, w, scale=scale)
    assert torch.equal(q3, q2) and torch.equal(a3, a2)


def test_rows_that_are_not_finite_stay_alone():
    x = bf16(5, 2560, seed=1)
    clean, rc = bw.rmsnorm(x, return_stats=True)
    x[1, 7], x[3, 9] = float("inf"), float("nan")
    y, rstd = bw.rmsnorm(x, return_stats=True)
    keep = [0, 2, 4]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(rstd[keep], rc[keep])
    assert torch.isnan(y[1, 7]) and torch.isnan(y[3]).all()


def back64(dy, x, w, rstd, dres):
    dy, x, rstd = dy.double(), x.double(), rstd.double()[:, None]
    w = torch.ones(x.shape[1], device=x.device).double() if w is None else w.double()
    z, g = x * rstd, dy * w
    add = 0.0 if dres is None else dres.double()
    dx = rstd * (g - z * (g * z).mean(1, keepdim=True)) + add
    size = rstd * (g.abs() + z.abs() * (g * z).abs().mean(1, keepdim=True)) + (
        0.0 if dres is None else add.abs())
    return dx, (dy * z).sum(0), size, (dy * z).abs().sum(0)


def check_back(dy, x, x64, w, rstd, x_scale, dres, what):
    dx, dw = bw.rmsnorm_backward(dy, x, w, rstd, x_scale=x_scale, dresidual=dres)
    rx, rw, size, sw = back64(dy, x64, w, rstd, dres)
    # 64 roundings of the sum, 10 of z, g and the products, the addition, then bf16
    close(dx, rx, BF * rx.abs() + (1 + BF) * 76 * U * size + TINY, what + " dx")
    # a column's path: rows of a lane, teams, blocks of a thread, 64 sums; z's three roundings
    M = dy.shape[0]
    close(dw, rw, (M / 64 + 96) * U * sw + TINY, what + " dw")
    dx2, none = bw.rmsnorm_backward(dy, x, w, rstd, x_scale=x_scale, dresidual=dres, need_sums=False)
    assert none is None and torch.equal(dx2, dx)
    again = bw.rmsnorm_backward(dy, x, w, rstd, x_scale=x_scale, dresidual=dres)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("M,K", [(1, 4), (1, 2560), (3, 60), (33, 252), (7, 1028), (17, 2564), (40, 4096),
                                 (9, 8196), (5, 16384), (3, 16388), (2100, 512), (600, 2048), (1100, 8192),
                                 (70, 20000), (1100, 4100), (7, 6140), (5, 6148)])
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("res", [False, True])
def test_backward(M, K, ckpt, res):
    x = bf16(M, K, seed=K, scale=2.0)
    dy = bf16(M, K, seed=K + 1, scale=1e-3, hot=False)
    dres = bf16(M, K, seed=K + 2, scale=1e-3, hot=False) if res else None
    w = f32(K, seed=1, scale=0.2, shift=1.0) if M % 2 else None
    _, rstd = bw.rmsnorm(x, w, return_stats=True)
    if ckpt:
        q, a = bw.quant_act_pow2(x)
        check_back(dy, q, q.double() / a.double()[:, None], w, rstd, a, dres, f"{M}x{K} checkpoint")
        q, a = bw.quant_act(x)
        check_back(dy, q, q.double() / a.double()[:, None], w, rstd, a, dres, f"{M}x{K} absmax codes")
    else:
        check_back(dy, x, x, w, rstd, None, dres, f"{M}x{K}")


@pytest.mark.parametrize("K", [256, 508, 2560, 4100, 8192, 20000])
def test_one_block_and_several(K):
    # column sums of a single block, and of several that a second launch joins
    for M in (2, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65):
        dy, x = bf16(M, K, seed=M, scale=1e-3, hot=False), bf16(M, K, seed=K)
        _, rstd = bw.rmsnorm(x, return_stats=True)
        check_back(dy, x, x, None, rstd, None, None, f"{M}x{K}")


def test_backward_is_the_gradient():
    # against automatic differentiation of the definition, and against differences
    M, K = 3, 24
    x, res = bf16(M, K, seed=1, hot=False), bf16(M, K, seed=2, hot=False)
    w = f32(K, seed=3, scale=0.2, shift=1.0)
    dy, ds = bf16(M, K, seed=4, hot=False), bf16(M, K, seed=5, hot=False)
    _, s, rstd = bw.rmsnorm(x, w, residual=res, return_stats=True)
    dx, dw = bw.rmsnorm_backward(dy, s, w, rstd, dresidual=ds)

    def loss(s64, w64):
        y = s64 * (s64.square().mean(1, keepdim=True) + EPS) ** -0.5 * w64
        return (y * dy.double()).sum() + (s64 * ds.double()).sum()
    s64, w64 = s.double().requires_grad_(), w.double().requires_grad_()
    gs, gw = torch.autograd.grad(loss(s64, w64), (s64, w64))
    size = 40.0  # sums of 24 products of values below 4 and 5
    close(dx, gs, BF * gs.abs() + 128 * U * size, "dx")
    close(dw, gw, 128 * U * size, "dw")
    h = 1e-5
    for m, k in ((0, 0), (1, 11), (2, 23)):
        e = torch.zeros_like(s64)
        e[m, k] = h
        with torch.no_grad():
            d = (loss(s64 + e, w64) - loss(s64 - e, w64)) / (2 * h)
        # differences of doubles: 2^-53 * size / h and the third derivative's h^2
        assert abs(d.item() - dx[m, k].item()) <= BF * abs(d.item()) + 1e-5


def test_empty_norms():
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert bw.rmsnorm(e, w).shape == (0, 64)
    dx, dw = bw.rmsnorm_backward(e, e, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


# ------------------------------------------------------------------- norm and clipping

def grads_of(shapes, seed=0, scale=1e-2):
    out = []
    for i, (shape, dt) in enumerate(shapes):
        out.append(f32(*shape, seed=seed + i, scale=scale).to(dt))
    return out


def norm64(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()


def check_norm(got, grads):
    ref = norm64(grads)
    assert got.shape == () and got.dtype == torch.float32
    # fp64 sums, rounded once
    assert abs(got.double() - ref) <= 1.001 * U * ref


def check_clipped(out, grads, max_norm, norm):
    c = min(1.0, max_norm / (norm.double().item() + 1e-6))
    for o, g in zip(out, grads):
        ref = g.double() * c
        # c: an addition, a quotient and the norm's own; the product; fp32 below 2^-126 in steps of 2^-149
        tol = 5 * U * ref.abs() + 2.0 ** -149
        if g.dtype == torch.bfloat16:
            tol = BF * ref.abs() + (1 + BF) * tol + 2.0 ** -133
        close(o, ref, tol, "clipped")


F, B = torch.float32, torch.bfloat16
LISTS = [
    [((1,), F)], [((3,), B)], [((7, 9), F), ((5,), B), ((0,), F), ((1, 1), B)],
    [((640, 2560), F), ((2560,), F), ((641, 260), B), ((129,), B)],
    [((8192 * 4,), F)], [((8192 * 2,), B), ((8192 * 4 + 1,), F)],
    [((17 + i,), (F, B)[i % 2]) for i in range(300)],
    [((4096, 4100), F), ((4096, 1111), B)],
    [((33_000_001,), B)],
]


@pytest.mark.parametrize("n", range(len(LISTS)))
def test_norm_and_clip(n):
    grads = grads_of(LISTS[n], seed=n)
    keep = [g.clone() for g in grads]
    norm = bw.grad_norm(grads)
    check_norm(norm, grads)
    assert torch.equal(bw.grad_norm(grads), norm)
    half = norm.item() / 2
    out = [torch.full_like(g, 9.0) for g in grads]
    got = bw.clip_grads(grads, half, out=out)
    assert torch.equal(got, norm) and all(torch.equal(g, k) for g, k in zip(grads, keep))
    check_clipped(out, keep, half, norm)
    given = [torch.empty_like(g) for g in grads]
    assert bw.clip_grads(grads, half, norm=norm, out=given) is norm
    assert all(torch.equal(p, q) for p, q in zip(given, out))
    # nothing to clip: copies into out, nothing in place
    bw.clip_grads(grads, 4 * half, out=given)
    assert all(torch.equal(p, q) for p, q in zip(given, keep))
    assert torch.equal(bw.clip_grads(grads, 4 * half), norm)
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    assert torch.equal(bw.clip_grads(grads, half), norm)  # in place
    assert all(torch.equal(p, q) for p, q in zip(grads, out))
    bw.clip_grads(grads, 0.0)
    assert not any(g.any() for g in grads)


@pytest.mark.parametrize("dt", [F, B])
def test_tensors_at_any_value(dt):
    # views that start and end anywhere, and outputs that lie differently: the neighbours stay
    flat, other = f32(5000, seed=1).to(dt), f32(5000, seed=2).to(dt)
    for start, n, at in ((0, 1, 0), (1, 2, 1), (3, 5, 2), (5, 31, 13), (2, 4096, 2), (7, 4001, 8), (9, 15, 1)):
        buf, to = flat.clone(), other.clone()
        g = buf[start:start + n]
        check_norm(bw.grad_norm([g]), [g])
        norm = norm64([g]).item()
        o = to[at:at + n]
        got = bw.clip_grads([g], norm / 3, out=[o])
        check_clipped([o], [g], norm / 3, got)
        assert torch.equal(to[:at], other[:at]) and torch.equal(to[at + n:], other[at + n:])
        bw.clip_grads([g], norm / 3)
        assert torch.equal(g, o)
        assert torch.equal(buf[:start], flat[:start]) and torch.equal(buf[start + n:], flat[start + n:])


def test_large_small_and_not_finite():
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((10,), 1e-30, device="cuda")]
    check_norm(bw.grad_norm(big), big)       # 1e61 does not fit fp32, its root does
    small = [torch.full((1 << 20,), 1e-25, device="cuda")]
    check_norm(bw.grad_norm(small), small)   # 1e-50 vanishes in fp32
    g = [torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=B)]
    g[0][3] = float("inf")
    norm = bw.clip_grads(g, 1.0)
    assert torch.isinf(norm) and torch.isnan(g[0][3]) and not g[1].any() and not g[0][:3].any()
    g[1][5] = float("nan")
    norm = bw.clip_grads(g, 1.0)
    assert torch.isnan(norm) and all(torch.isnan(t).all() for t in g)
    assert bw.grad_norm([]).item() == 0.0
    assert bw.clip_grads([torch.empty(0, device="cuda")], 1.0).item() == 0.0


def test_norm_past_32_bits():
    # more than 2^32 bytes and 2^31 values; zeros add nothing, so the ends are what is summed
    g = torch.zeros(2 ** 31 + 77, dtype=B, device="cuda")
    g[0], g[2 ** 31 - 1], g[-1] = 3.0, 4.0, 12.0
    assert bw.grad_norm([g]).item() == 13.0
    bw.clip_grads([g], 6.5)
    assert [g[0].item(), g[2 ** 31 - 1].item(), g[-1].item()] == [1.5, 2.0, 6.0]


def test_clip_in_graph_replays_and_streams():
    grads = grads_of(LISTS[3], seed=3)
    src = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    want = bw.clip_grads(grads, 0.25, out=out).clone()
    ref = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bw.clip_grads(grads, 0.25, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = bw.clip_grads(grads, 0.25)
    for rep in range(3):
        for g, s in zip(grads, src):
            g.copy_(s)
        graph.replay()
        bw.grad_norm(src)  # eager work in between
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(g, r) for g, r in zip(grads, ref)), rep


def test_refusals():
    x = bf16(4, 256, seed=1)
    w = torch.ones(256, device="cuda")
    with pytest.raises(TypeError):
        bw.rmsnorm(x.float())
    with pytest.raises(ValueError):
        bw.rmsnorm(x, residual=x[:2])
    with pytest.raises(ValueError):
        bw.rmsnorm(x, sum_out=x.clone())
    with pytest.raises(ValueError):
        bw.rmsnorm(x[:, ::2])
    with pytest.raises(bw.BitnetError):
        bw.rmsnorm(x, eps=0.0)
    many, few = bf16(400, 256, seed=2), torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(bw.BitnetError):
        bw.rmsnorm_backward(many, many, w, torch.ones(400, device="cuda"), workspace=few)
    bw.rmsnorm_backward(x, x, w, torch.ones(4, device="cuda"), workspace=few)  # a single block needs none
    with pytest.raises(ValueError):
        bw.rmsnorm(x, torch.ones(256, device="cuda", requires_grad=True))
    g = torch.ones(64, device="cuda")
    with pytest.raises(bw.BitnetError):
        bw.clip_grads([g, g], 1.0)                    # the same memory twice
    with pytest.raises(bw.BitnetError):
        bw.clip_grads([g[:40], g[32:]], 1.0)
    with pytest.raises(bw.BitnetError):
        bw.clip_grads([g[:32], g[32:]], 1.0, out=[g[16:48], torch.empty(32, device="cuda")])
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(bw.BitnetError):
            bw.clip_grads([g], bad)
    with pytest.raises(TypeError):
        bw.grad_norm([g.double()])
    with pytest.raises(TypeError):
        bw.grad_norm([g, None])
    with pytest.raises(ValueError):
        bw.grad_norm([g, torch.ones(3)])
    with pytest.raises(ValueError):
        bw.grad_norm([g[::2]])
    with pytest.raises(ValueError):
        bw.clip_grads([g], 1.0, out=[])
    with pytest.raises(TypeError):
        bw.clip_grads([g], 1.0, out=[torch.empty(64, dtype=B, device="cuda")])
    assert torch.equal(g, torch.ones(64, device="cuda"))
