"""The training entry points' boundary, on the CPU: bad arguments are refused on the host
before any HIP call, empty problems are accepted, and the Python binding refuses CPU
tensors."""
import ctypes

import pytest
import torch

import ternary_weight_linear_token_amd as bw

OK, INVALID, UNALIGNED, WORKSPACE, HIP, DEVICE = 0, 1, 2, 3, 4, 5
# fake, 16-byte-aligned, never-dereferenced addresses
A, B, C, D, E, F, G, H = (0x1000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def L():
    return bw.lib()


def i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)



@pytest.mark.parametrize("name", ["bitnet_quant_act_pow2", "bitnet_dequant_act"])
def test_checkpoint_validation(L, name):
    call = getattr(L, name)
    f = (lambda x, M, K, q, a: call(x, M, K, q, a, None)) if name.endswith("pow2") else (
        lambda x, M, K, q, a: call(q, a, M, K, x, None))
    assert f(None, 1, 8, B, C) == INVALID
    assert f(A, 1, 8, None, C) == INVALID
    assert f(A, 1, 8, B, None) == INVALID
    assert f(A, -1, 8, B, C) == INVALID
    assert f(A, 1, 0, B, C) == INVALID
    assert f(A, 1, 6, B, C) == UNALIGNED
    assert f(A + 8, 1, 8, B, C) == UNALIGNED
    assert f(A, 1, (1 << 20) + 4, B, C) == INVALID
    assert f(None, 0, 8, None, None) == OK


def test_layernorm_validation(L):
    def f(x=A, w=B, b=C, eps=1e-5, M=4, K=256, y=D, xq=E, a=F, scale=0, mean=G, rstd=H):
        return L.bitnet_layernorm(x, w, b, eps, M, K, y, xq, a, scale, mean, rstd, None)
    assert f(x=None) == INVALID
    assert f(y=None, xq=None, a=None) == INVALID      # nothing to write
    assert f(a=None) == INVALID and f(xq=None) == INVALID  # codes and scales go together
    assert f(scale=2) == INVALID and f(scale=-1) == INVALID
    for eps in (0.0, -1e-5, 1e-39, float("inf"), float("nan")):
        assert f(eps=eps) == INVALID
    assert f(K=255) == UNALIGNED and f(K=0) == INVALID and f(K=(1 << 20) + 4) == INVALID
    assert f(M=-1) == INVALID and f(M=1 << 31) == INVALID
    for name in ("x", "w", "b", "y", "xq", "a", "mean", "rstd"):
        assert f(**{name: A + 4}) == UNALIGNED, name
    assert f(M=0, x=None) == OK


def test_layernorm_backward_validation(L):
    ws = L.bitnet_layernorm_backward_workspace_size(8, 256)
    assert ws > 0 and ws % 2048 == 0  # whole (2, K) fp32 partials
    assert L.bitnet_layernorm_backward_workspace_size(8, 255) == 0
    assert L.bitnet_layernorm_backward_workspace_size(-1, 256) == 0

    def f(dy=A, x=B, xs=None, w=C, mean=D, rstd=E, M=8, K=256, dx=F, dw=G, db=H, ws_ptr=A, n=ws):
        return L.bitnet_layernorm_backward(dy, x, xs, w, mean, rstd, M, K, dx, dw, db, ws_ptr, n, None)
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert f(**{name: None}) == INVALID, name
    for name in ("dy", "x", "xs", "w", "mean", "rstd", "dx", "dw", "db", "ws_ptr"):
        assert f(**{name: A + 8}) == UNALIGNED, name
    assert f(ws_ptr=None) == INVALID                     # bytes but no buffer
    assert f(n=ws - 1) == WORKSPACE and f(ws_ptr=None, n=0) == WORKSPACE
    assert f(M=0, dw=None, db=None) == OK
    assert f(K=254) == UNALIGNED and f(M=-1) == INVALID


def test_swiglu_validation(L):
    def f(g=A, u=B, M=4, N=256, h=C, hq=D, hs=E, scale=0, gq=F, gs=G, uq=H, us=A):
        return L.bitnet_swiglu(g, u, M, N, h, hq, hs, scale, gq, gs, uq, us, None)
    assert f(g=None) == INVALID and f(u=None) == INVALID
    assert f(h=None, hq=None, hs=None) == INVALID
    assert f(hs=None) == INVALID and f(hq=None) == INVALID
    for name in ("gq", "gs", "uq", "us"):
        assert f(**{name: None}) == INVALID, name        # all four or none
    assert f(scale=3) == INVALID
    for name in ("g", "u", "h", "hq", "hs", "gq", "gs", "uq", "us"):
        assert f(**{name: A + 2}) == UNALIGNED, name
    assert f(N=250) == UNALIGNED and f(N=0) == INVALID and f(M=-1) == INVALID
    assert f(M=0, g=None) == OK

    def b(dh=A, g=B, gs=C, u=D, us=E, M=4, N=256, dg=F, du=G):
        return L.bitnet_swiglu_backward(dh, g, gs, u, us, M, N, dg, du, None)
    for name in ("dh", "g", "u", "dg", "du", "gs", "us"):
        assert b(**{name: None}) == INVALID, name
        assert b(**{name: A + 2}) == UNALIGNED, name
    assert b(N=6) == UNALIGNED and b(M=0) == OK


def test_grad_input_validation(L):
    def f(M=4, K=256, groups=2, dy=ptrs(A, B), p=ptrs(C, D), s=ptrs(E, F), N=i64s(16, 32), dx=G,
          ws=None, n=0):
        return L.bitnet_grad_input(M, K, groups, dy, p, s, N, dx, ws, n, None)
    assert f(groups=0) == INVALID and f(groups=5) == INVALID
    for name in ("dy", "p", "s", "N", "dx"):
        assert f(**{name: None}) == INVALID, name
    assert f(dy=ptrs(A, None)) == INVALID and f(p=ptrs(None, D)) == INVALID
    assert f(s=ptrs(E, None)) == INVALID
    assert f(dy=ptrs(A, B + 2)) == UNALIGNED and f(p=ptrs(C + 4, D)) == UNALIGNED
    assert f(dx=G + 8) == UNALIGNED and f(ws=A + 8, n=16) == UNALIGNED
    assert f(ws=None, n=16) == INVALID
    assert f(K=250) == UNALIGNED and f(K=0) == INVALID
    assert f(N=i64s(16, -1)) == INVALID and f(N=i64s(16, (1 << 20) + 1)) == INVALID
    assert f(M=-1) == INVALID and f(M=0, dx=None) == OK
    assert f(M=(1 << 30) + 1) == INVALID
    assert L.bitnet_grad_input_workspace_size(4, 250, 2, i64s(16, 32)) == 0
    assert L.bitnet_grad_input_workspace_size(4, 256, 0, i64s(16, 32)) == 0


def test_grad_weight_validation(L):
    def f(dy=A, xq=B, a=C, M=4, N=16, K=256, dw=D, dt=0, ws=None, n=0):
        return L.bitnet_grad_weight(dy, xq, a, M, N, K, dw, dt, ws, n, None)
    for name in ("dy", "xq", "a", "dw"):
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: A + 8}) == UNALIGNED, name
    assert f(dt=2) == INVALID and f(dt=-1) == INVALID
    assert f(ws=None, n=16) == INVALID and f(ws=A + 4, n=16) == UNALIGNED
    assert f(K=254) == UNALIGNED and f(N=(1 << 20) + 1) == INVALID and f(N=-1) == INVALID
    assert f(N=0, dw=None) == OK and f(M=(1 << 30) + 1) == INVALID
    assert L.bitnet_grad_weight_workspace_size(4, 16, 254) == 0
    assert L.bitnet_grad_weight_workspace_size(0, 16, 256) == 0


def test_grad_plans():
    seen = set()
    for M in (1, 4, 16, 64, 129, 333, 512, 2048, 8192):
        for N, K in ((641, 2564), (2560, 2560), (640, 2560), (6912, 2560), (2560, 6912),
                     (14336, 4096), (4096, 14336), (28672, 8192)):
            for weight in (False, True):
                bm, bn, g, slices = bw.grad_plan(M, K, [N], weight)
                seen.add((weight, bm, bn, g))
                ws = (bw.lib().bitnet_grad_weight_workspace_size(M, N, K) if weight else
                      bw.lib().bitnet_grad_input_workspace_size(M, K, 1, i64s(N)))
                rows = N if weight else M
                assert ws == (slices * rows * K * 4 if slices > 1 else 0)
                assert ws <= 64 << 20
    # every compiled configuration is one that some size takes
    assert {s[1:] for s in seen if s[0]} == {(256, 256, 1), (128, 128, 1)}
    assert {s[1:] for s in seen if not s[0]} == {(256, 256, 1), (256, 128, 2), (64, 128, 4), (32, 128, 4)}
    with pytest.raises(bw.BitnetError):
        bw.grad_plan(4, 256, [16, 16], weight=True)
    with pytest.raises(bw.BitnetError):
        bw.grad_plan(0, 256, [16])


def test_binding_refuses_what_the_library_cannot_take():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q = torch.zeros((4, 256), dtype=torch.int8)
    s = torch.ones(4)
    for call in (lambda: bw.quant_act_pow2(x), lambda: bw.dequant_act(q, s),
                 lambda: bw.layernorm(x), lambda: bw.layernorm_quant(x),
                 lambda: bw.layernorm_backward(x, x, None, s, s), lambda: bw.swiglu(x, x),
                 lambda: bw.swiglu_quant(x, x), lambda: bw.swiglu_backward(x, x, x),
                 lambda: bw.grad_input(x, q, s), lambda: bw.grad_weight(x, q, s)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError):
        bw.grad_input_grouped([], [], [])
    with pytest.raises(KeyError):
        bw.layernorm_quant(x, scale="amax")
