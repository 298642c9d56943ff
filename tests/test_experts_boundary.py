"""The boundary of the norm, clipping and mixture-of-experts entry points, on the CPU: bad
arguments are refused on the host before any HIP call, empty problems are accepted, and the
Python binding refuses CPU tensors."""
import ctypes
import subprocess

import pytest
import torch

import ternary_weight_linear_token_amd as bw

OK, INVALID, UNALIGNED, WORKSPACE, HIP, DEVICE = 0, 1, 2, 3, 4, 5
# fake, 16-byte-aligned, never-dereferenced addresses
A, B, C, D, E, F, G, H = (0x1000 * i for i in range(1, 9))
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    return bw.lib()


def i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def i32s(*v):
    return (ctypes.c_int32 * len(v))(*v)


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def test_rmsnorm_validation(L):
    def f(x=A, res=B, w=C, eps=1e-5, M=4, K=256, s=D, y=E, xq=F, a=G, scale=0, rstd=H):
        return L.bitnet_rmsnorm(x, res, w, eps, M, K, s, y, xq, a, scale, rstd, None)
    assert f(x=None) == INVALID
    assert f(y=None, xq=None, a=None) == INVALID           # nothing to write
    assert f(a=None) == INVALID and f(xq=None) == INVALID  # codes and scales go together
    assert f(s=None) == INVALID and f(res=None) == INVALID  # and the residual and its sum
    assert f(scale=2) == INVALID and f(scale=-1) == INVALID
    for eps in (0.0, -1e-5, 1e-39, float("inf"), float("nan")):
        assert f(eps=eps) == INVALID
    assert f(K=255) == UNALIGNED and f(K=0) == INVALID and f(K=(1 << 20) + 4) == INVALID
    assert f(M=-1) == INVALID and f(M=1 << 31) == INVALID
    for name in ("x", "res", "w", "s", "y", "xq", "a", "rstd"):
        assert f(**{name: A + 4}) == UNALIGNED, name
    assert f(M=0, x=None) == OK


def test_rmsnorm_backward_validation(L):
    ws = L.bitnet_rmsnorm_backward_workspace_size(800, 256)
    assert ws > 0 and ws % 1024 == 0  # whole rows of fp32 partials
    assert L.bitnet_rmsnorm_backward_workspace_size(8, 256) == 0  # a single block
    assert L.bitnet_rmsnorm_backward_workspace_size(8, 255) == 0
    assert L.bitnet_rmsnorm_backward_workspace_size(0, 256) == 0

    def f(dy=A, x=B, xs=None, w=C, rstd=D, dres=E, M=800, K=256, dx=F, dw=G, ws_ptr=H, n=ws):
        return L.bitnet_rmsnorm_backward(dy, x, xs, w, rstd, dres, M, K, dx, dw, ws_ptr, n, None)
    for name in ("dy", "x", "rstd", "dx"):
        assert f(**{name: None}) == INVALID, name
    for name in ("dy", "x", "xs", "w", "rstd", "dres", "dx", "dw", "ws_ptr"):
        assert f(**{name: A + 8}) == UNALIGNED, name
    assert f(ws_ptr=None) == INVALID
    assert f(n=ws - 1) == WORKSPACE and f(ws_ptr=None, n=0) == WORKSPACE
    assert f(M=0, dw=None) == OK
    assert f(K=254) == UNALIGNED and f(M=-1) == INVALID


def test_grad_norm_validation(L):
    ws = L.bitnet_grad_norm_workspace_size(2)
    assert ws > 0 and ws == L.bitnet_grad_norm_workspace_size(0)
    assert L.bitnet_grad_norm_workspace_size(1000) > ws
    assert L.bitnet_grad_norm_workspace_size(-1) == 0 and L.bitnet_grad_norm_workspace_size(1 << 31) == 0

    def f(count=2, g=ptrs(A, B), n=i64s(64, 3), dt=i32s(0, 1), norm=C, w=D, b=ws):
        return L.bitnet_grad_norm(count, g, n, dt, norm, w, b, None)
    assert f(count=-1) == INVALID and f(count=1 << 31) == INVALID
    for name in ("g", "n", "dt", "norm", "w"):
        assert f(**{name: None}) == INVALID, name
    assert f(g=ptrs(A, None)) == INVALID
    assert f(n=i64s(64, -1)) == INVALID and f(n=i64s(64, 1 << 61)) == INVALID
    assert f(dt=i32s(0, 2)) == INVALID and f(dt=i32s(-1, 1)) == INVALID
    assert f(g=ptrs(A + 2, B)) == UNALIGNED and f(g=ptrs(A, B + 1)) == UNALIGNED
    assert f(norm=C + 2) == UNALIGNED and f(w=D + 8) == UNALIGNED
    assert f(b=ws - 1) == WORKSPACE and f(w=None, b=0) == WORKSPACE


def test_clip_validation(L):
    ws = L.bitnet_grad_norm_workspace_size(3)
    g = ptrs(A, B, None)

    def f(count=3, g=g, out=g, n=i64s(64, 3, 0), dt=i32s(0, 1, 0), m=1.0, ni=None, no=C, w=D, b=ws):
        return L.bitnet_clip_grads(count, g, out, n, dt, m, ni, no, w, b, None)
    for name in ("g", "n", "dt", "out", "w"):
        assert f(**{name: None}) == INVALID, name
    for m in (-1.0, float("nan"), float("inf")):
        assert f(m=m) == INVALID
    assert f(out=ptrs(A, None, None)) == INVALID
    assert f(out=ptrs(A + 2, B, None)) == UNALIGNED and f(out=ptrs(A, B + 1, None)) == UNALIGNED
    assert f(ni=E + 2) == UNALIGNED and f(no=C + 1) == UNALIGNED
    assert f(b=ws - 16) == WORKSPACE
    # outputs over one another, over another's input, half over their own
    assert f(g=ptrs(A, A + 256, A + 256), out=ptrs(E, E + 4, None), n=i64s(64, 64, 0), dt=i32s(0, 0, 0)) == INVALID
    assert f(g=ptrs(A, A + 252, None), out=ptrs(A, A + 252, None), n=i64s(64, 64, 0)) == INVALID
    assert f(g=ptrs(A, B, None), out=ptrs(B + 4, E, None), n=i64s(64, 64, 0)) == INVALID
    assert f(g=ptrs(A, B, None), out=ptrs(A + 128, B, None), n=i64s(64, 64, 0)) == INVALID
    assert f(g=ptrs(A, A, None), out=ptrs(A, A, None), n=i64s(8, 8, 0), dt=i32s(0, 0, 0)) == INVALID


def test_overlaps_are_found_by_the_sorted_spans(L):
    # against every pair, on random spans; a call that passes the check fails later, without a device
    import random
    rng = random.Random(1)
    ws = L.bitnet_grad_norm_workspace_size(6)
    seen = set()
    for _ in range(300):
        n = [rng.randint(0, 40) for _ in range(6)]
        g = [0x10000 + 4 * rng.randint(0, 400) for _ in n]
        o = [x if rng.random() < 0.5 else 0x10000 + 4 * rng.randint(0, 2000) for x in g]
        spans = [(x, x + 4 * m) for x, m in zip(o, n)]
        ins = [(x, x + 4 * m) for x, m in zip(g, n)]
        cut = lambda p, q: p[0] < q[1] and q[0] < p[1]
        bad = False
        for i in range(6):
            for j in range(6):
                if n[i] and n[j]:
                    bad |= i < j and cut(spans[i], spans[j])
                    bad |= cut(spans[i], ins[j]) and not (i == j and g[i] == o[i])
        seen.add(bad)
        if bad:  # (calls that pass would reach the device, where there is one)
            st = L.bitnet_clip_grads(6, ptrs(*g), ptrs(*o), i64s(*n), i32s(*[0] * 6), 1.0, None, A, B, ws, None)
            assert st == INVALID, (n, g, o)
        elif not torch.cuda.is_available():
            st = L.bitnet_clip_grads(6, ptrs(*g), ptrs(*o), i64s(*n), i32s(*[0] * 6), 1.0, None, A, B, ws, None)
            assert st in (HIP, DEVICE), (n, g, o)
    assert seen == {False, True}


@pytest.mark.parametrize("count", [255, 256, 257, 600, 3000])
def test_overlaps_in_long_lists(L, count):
    # spans side by side in any order, in place or not; then one of them reaches over another's first value
    import random
    rng = random.Random(count)
    places = list(range(2 * count))
    rng.shuffle(places)
    ws = L.bitnet_grad_norm_workspace_size(count)
    n = [rng.randint(1, 16) for _ in range(count)]
    g = [0x100000 + 64 * places[2 * i] for i in range(count)]
    o = [p if rng.random() < 0.5 else 0x100000 + 64 * places[2 * i + 1] for i, p in enumerate(g)]

    def f(g, o, n):
        return L.bitnet_clip_grads(count, ptrs(*g), ptrs(*o), i64s(*n), i32s(*[0] * count), 1.0, None, A, B, ws, None)
    if not torch.cuda.is_available():  # (a call that passes would reach the device)
        assert f(g, o, n) in (HIP, DEVICE)
    at = {p: i for i, p in enumerate(o)}
    tried = 0
    for i in rng.sample(range(count), min(count, 40)):
        j = at.get(o[i] + 64)  # the output in the next place
        if j is None:
            continue
        tried += 1
        longer = list(n)
        longer[i] = 17
        assert f(g, o, longer) == INVALID, (i, j)
        # the same reach from an input over that output is an overlap too, unless the output lies elsewhere
        if g[i] != o[i] and g[j] != o[j]:
            moved = list(o)
            moved[i] = 0x100000 + 64 * (2 * count + 5)
            assert f(g[:i] + [o[i]] + g[i + 1:], moved, longer) == INVALID, (i, j)
            if not torch.cuda.is_available():
                free = list(o)
                free[i], free[j] = 0x100000 + 64 * (2 * count + 5), 0x100000 + 64 * (2 * count + 9)
                assert f(g[:i] + [o[i]] + g[i + 1:], free, longer) in (HIP, DEVICE), (i, j)
    assert tried > 0


def test_the_library_allocates_nothing_on_the_host(L):
    names = subprocess.run(["nm", "-D", "--undefined-only", bw.library_path()], capture_output=True, text=True,
                           check=True).stdout.split()
    assert not [n for n in names if n.startswith(("_Znw", "_Zna", "malloc", "calloc", "realloc", "aligned_alloc"))]


def test_expert_order_validation(L):
    assert L.bitnet_expert_order_workspace_size(64, 8) == 0
    big = L.bitnet_expert_order_workspace_size(1 << 20, 64)
    assert big > 0 and big % (65 * 4) == 0
    for P, n in ((-1, 8), (BIG + 1, 8), (64, 0), (64, 1025)):
        assert L.bitnet_expert_order_workspace_size(P, n) == 0

    def f(ids=A, wide=0, T=4, J=2, n=8, rows=B, off=C, slots=D, w=None, b=0):
        return L.bitnet_expert_order(ids, wide, T, J, n, rows, off, slots, w, b, None)
    for name in ("ids", "rows", "off", "slots"):
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: A + 8}) == UNALIGNED, name
    assert f(wide=2) == INVALID and f(T=-1) == INVALID and f(T=BIG + 1) == INVALID
    assert f(J=0) == INVALID and f(J=1025) == INVALID and f(T=BIG, J=2) == INVALID
    assert f(n=0) == INVALID and f(n=1025) == INVALID
    assert f(T=0, ids=None, rows=None, slots=None, off=None) == INVALID  # offsets are written all the same
    assert f(T=1 << 19, n=64) == WORKSPACE and f(T=1 << 19, n=64, w=E, b=big - 4) == WORKSPACE
    assert f(w=None, b=16) == INVALID and f(w=E + 4, b=16) == UNALIGNED


def test_gemm_experts_validation(L):
    def f(xq=A, a=B, T=6, rows=None, off=C, P=6, n=4, K=256, groups=2, p=ptrs(D, E), s=ptrs(F, G),
          N=i64s(16, 32), out=ptrs(H, A), dt=0):
        return L.bitnet_gemm_experts(xq, a, T, rows, off, P, n, K, groups, p, s, N, out, dt, None)
    assert f(groups=0) == INVALID and f(groups=5) == INVALID and f(dt=3) == INVALID
    for name in ("xq", "a", "off", "p", "s", "N", "out"):
        assert f(**{name: None}) == INVALID, name
    for name in ("xq", "a", "off"):
        assert f(**{name: A + 8}) == UNALIGNED, name
    assert f(rows=A + 4) == UNALIGNED
    assert f(p=ptrs(D, None)) == INVALID and f(s=ptrs(None, G)) == INVALID and f(out=ptrs(H, None)) == INVALID
    assert f(p=ptrs(D, E + 4)) == UNALIGNED and f(out=ptrs(H + 8, A)) == UNALIGNED
    assert f(n=0) == INVALID and f(n=1025) == INVALID
    assert f(T=5) == INVALID and f(P=7) == INVALID            # without rows, one token a row
    assert f(T=-1, rows=A) == INVALID
    assert f(T=1 << 23, rows=A) == INVALID                     # 2^31 bytes of codes
    assert f(K=254) == UNALIGNED and f(K=0) == INVALID and f(P=-1, T=-1) == INVALID
    assert f(P=BIG + 1, T=BIG + 1) == INVALID
    assert f(N=i64s(16, -1)) == INVALID and f(N=i64s(16, (1 << 20) + 1)) == INVALID
    assert f(P=0, T=0, xq=None, a=None, off=None) == OK
    assert f(N=i64s(0, 0), off=None) == OK


def test_experts_gradient_validation(L):
    def f(off=A, P=6, n=4, K=256, groups=2, dy=ptrs(B, C), p=ptrs(D, E), s=ptrs(F, G), N=i64s(16, 32), dx=H):
        return L.bitnet_grad_input_experts(off, P, n, K, groups, dy, p, s, N, dx, None)
    assert f(groups=0) == INVALID and f(groups=5) == INVALID
    for name in ("off", "dy", "p", "s", "N", "dx"):
        assert f(**{name: None}) == INVALID, name
    assert f(off=A + 4) == UNALIGNED and f(dx=H + 8) == UNALIGNED
    assert f(dy=ptrs(B, None)) == INVALID and f(dy=ptrs(B, C + 2)) == UNALIGNED
    assert f(n=0) == INVALID and f(n=1025) == INVALID and f(K=250) == UNALIGNED
    assert f(N=i64s(16, (1 << 20) + 1)) == INVALID and f(P=BIG + 1) == INVALID and f(P=-1) == INVALID
    assert f(P=0, off=None, dx=None) == OK

    ws = L.bitnet_grad_weight_experts_workspace_size(6, 256)
    assert ws >= 6 * 256 + 24
    assert L.bitnet_grad_weight_experts_workspace_size(6, 254) == 0
    assert L.bitnet_grad_weight_experts_workspace_size(0, 256) == 0
    assert L.bitnet_grad_weight_experts_workspace_size(BIG + 1, 256) == 0

    def g(dy=A, xq=B, a=C, T=5, rows=D, off=E, P=6, n=4, N=16, K=256, dw=F, dt=0, w=G, b=ws):
        return L.bitnet_grad_weight_experts(dy, xq, a, T, rows, off, P, n, N, K, dw, dt, w, b, None)
    for name in ("dy", "xq", "a", "off", "dw"):
        assert g(**{name: None}) == INVALID, name
        assert g(**{name: A + 8}) == UNALIGNED, name
    assert g(rows=A + 8) == UNALIGNED and g(w=G + 4) == UNALIGNED
    assert g(rows=None) == INVALID                             # five tokens, six rows
    assert g(dt=2) == INVALID and g(n=0) == INVALID and g(n=1025) == INVALID
    assert g(b=ws - 1) == WORKSPACE and g(w=None, b=0) == WORKSPACE and g(w=None) == INVALID
    assert g(K=254) == UNALIGNED and g(N=(1 << 20) + 1) == INVALID and g(N=-1) == INVALID
    assert g(T=1 << 23) == INVALID
    assert g(N=0, dw=None) == OK


def test_combine_validation(L):
    def f(y=A, slots=B, w=C, T=4, J=2, P=8, Dm=64, out=D):
        return L.bitnet_combine_experts(y, slots, w, T, J, P, Dm, out, None)

    def g(dout=A, y=B, slots=C, w=D, T=4, J=2, P=8, Dm=64, dy=E, dw=F):
        return L.bitnet_combine_experts_backward(dout, y, slots, w, T, J, P, Dm, dy, dw, None)
    for call, names in ((f, ("y", "slots", "out")), (g, ("dout", "y", "slots", "dy"))):
        for name in names:
            assert call(**{name: None}) == INVALID, name
            assert call(**{name: A + 8}) == UNALIGNED, name
        assert call(w=C + 4) == UNALIGNED
        assert call(J=0) == INVALID and call(J=1025) == INVALID
        assert call(T=-1) == INVALID and call(T=BIG + 1) == INVALID
        assert call(P=-1) == INVALID and call(P=BIG + 1) == INVALID
        assert call(Dm=62) == UNALIGNED and call(Dm=0) == INVALID and call(Dm=(1 << 20) + 4) == INVALID
        assert call(T=0, slots=None) == OK
    assert g(dw=F + 4) == UNALIGNED


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q = torch.zeros((4, 256), dtype=torch.int8)
    s = torch.ones(4)
    off = torch.zeros(3, dtype=torch.int32)
    p = torch.zeros((2, 16, 64), dtype=torch.uint8)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: bw.rmsnorm(x), lambda: bw.rmsnorm_quant(x), lambda: bw.rmsnorm_backward(x, x, None, s),
                 lambda: bw.grad_norm([x]), lambda: bw.clip_grads([x], 1.0), lambda: bw.expert_order(ids, 2),
                 lambda: bw.gemm_experts(q, s, off, p, torch.ones((2, 16))),
                 lambda: bw.grad_input_experts(x, off, p, torch.ones((2, 16))),
                 lambda: bw.grad_weight_experts(x, q, s, off), lambda: bw.combine_experts(x, ids),
                 lambda: bw.combine_experts_backward(x, x, ids)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(KeyError):
        bw.rmsnorm_quant(x, scale="amax")
