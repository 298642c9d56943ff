"""The products grouped by expert, the order of the tokens and the sum of their rows on the GPU
against plain forms: integers exactly, the rest against 64 bits with counted roundings (u = 2^-24
for fp32, 2^-8 for bf16, relative to the value)."""
import numpy as np
import pytest
import torch

import ternary_weight_linear_token_amd as bw
from test_gpu_train import (BF, TINY, U, bf16, check_grad_input, check_grad_weight, close, f32, gen, pow2_of,
                            ternary, weights64)

pytestmark = pytest.mark.gpu


def experts(E, N, K, seed=0):
    """Packed weights (E, N, K / 4) and scales (E, N)."""
    p, s = ternary(E * N, K, seed=seed)
    return p.view(E, N, K // 4), s.view(E, N)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def spread(P, E, seed, kind):
    """Counts of P rows over E experts."""
    if kind == "one":  # all of them to one expert in the middle
        c = np.zeros(E, dtype=np.int64)
        c[E // 2] = P
        return c
    p = np.ones(E) / E if kind == "even" else np.random.RandomState(seed).dirichlet(np.full(E, 0.4))
    return np.random.RandomState(seed + 1).multinomial(P, p)


# ------------------------------------------------------------------------------- order

def order64(ids, E):
    flat = ids.reshape(-1).cpu().numpy().astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    by = np.argsort(key, kind="stable")
    slots = np.empty_like(by)
    slots[by] = np.arange(by.size)
    live = key[by] < E
    rows = np.where(live, by // ids.shape[1], -1)
    slots = np.where(key < E, slots, -1).reshape(ids.shape)
    offsets = np.searchsorted(key[by], np.arange(E + 1))
    return rows, offsets, slots


ORDERS = [(1, 1, 1), (1, 2, 8), (3, 1, 2), (32, 8, 64), (63, 1, 5), (65, 3, 7), (500, 8, 1024), (1000, 4, 128),
          (4096, 2, 8), (8191, 2, 63), (8193, 2, 8), (20000, 1, 1), (30000, 3, 255), (100000, 8, 1024),
          (300001, 7, 64)]


@pytest.mark.parametrize("T,J,E", ORDERS)
@pytest.mark.parametrize("dt", [torch.int32, torch.int64])
def test_order(T, J, E, dt):
    g = gen(T + J + E)
    # some experts twice, some never, some choices dropped
    ids = torch.randint(-1, E + 1, (T, J), generator=g)
    if T % 2:
        ids = torch.randint(0, max(1, E // 3), (T, J), generator=g)
    got = bw.expert_order(ids.to(dt).cuda(), E)
    for name, p, q in zip(("rows", "offsets", "slots"), got, order64(ids, E)):
        assert p.dtype == torch.int32 and np.array_equal(p.cpu().numpy(), q), name


def test_order_of_strange_ids():
    big = torch.tensor([[2 ** 33, 1], [-2 ** 40, 0], [1, 2 ** 31]], dtype=torch.int64)
    for name, p, q in zip("ros", bw.expert_order(big.cuda(), 2), order64(big, 2)):
        assert np.array_equal(p.cpu().numpy(), q), name
    none = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    rows, offsets, slots = bw.expert_order(none, 3)
    assert (rows == -1).all() and (slots == -1).all() and not offsets.any()
    rows, offsets, slots = bw.expert_order(none[:0], 3)
    assert rows.numel() == 0 and slots.shape == (0, 2) and not offsets.any()


# ----------------------------------------------------------------------------- forward

def check_forward(xq, a, counts, packed, s, rows, what, dts=("i32", "f32", "bf16"), tail=0):
    E, N, K4 = packed.shape
    off = offsets_of(counts)
    P = int(sum(counts)) + tail
    for dt in dts:
        code = {"i32": torch.int32, "f32": torch.float32, "bf16": torch.bfloat16}[dt]
        out = torch.full((P, N), 77, dtype=code, device="cuda")
        got = bw.gemm_experts(xq, a, off, packed, s, dt, rows=rows, out=out)
        assert got is out
        assert (out[P - tail:] == 77).all(), f"{what}: rows behind the last"
        at = 0
        for e, c in enumerate(counts):
            if c == 0:
                continue
            pick = rows[at:at + c].long() if rows is not None else torch.arange(at, at + c, device="cuda")
            here = (pick >= 0) & (pick < xq.shape[0])
            x = xq[pick.clamp(0, xq.shape[0] - 1)].double() * here[:, None]
            acc = x @ (bw.unpack_weights(packed[e].clone(), 4 * K4).double().t().contiguous())
            o = out[at:at + c]
            if dt == "i32":
                assert torch.equal(o.double(), acc), f"{what} expert {e}"
            else:
                inv = torch.where(here, a[pick.clamp(0, xq.shape[0] - 1)].double(), 1.0)
                ref = acc * s[e].double() / inv[:, None]
                # the reciprocal and two products
                close(o, ref, (3.1 * U if dt == "f32" else BF + 3.1 * U) * ref.abs(), f"{what} {dt} {e}")
            at += c


SHAPES = [(1, 2, 16, 16), (2, 8, 33, 64), (5, 3, 640, 2560), (16, 64, 40, 256), (40, 4, 130, 260),
          (100, 16, 641, 2564), (256, 64, 640, 2560), (300, 3, 257, 1028), (700, 8, 300, 4096), (999, 5, 512, 132),
          (1500, 2, 256, 272), (2100, 8, 2560, 640), (600, 1, 256, 1024), (129, 200, 17, 20), (64, 1024, 8, 80), (1500, 64, 1100, 272), (1500, 64, 1100, 276)]


@pytest.mark.parametrize("P,E,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
def test_product_of_sorted_rows(P, E, N, K, kind):
    counts = spread(P, E, P + E, kind)
    xq, a = bw.quant_act(bf16(P + 3, K, seed=P))
    packed, s = experts(E, N, K, seed=N)
    # xq holds rows behind the last expert's, which are not written
    check_forward(xq, a, counts, packed, s, None, f"{P} {E} {N} {K} {kind}", tail=3)


@pytest.mark.parametrize("P,E,N,K", SHAPES)
def test_product_with_gather(P, E, N, K):
    counts = spread(P, E, P * E, "skewed")
    T = max(1, P // 2)
    xq, a = bw.quant_act(bf16(T, K, seed=P))
    packed, s = experts(E, N, K, seed=N)
    rows = torch.randint(0, T, (P + 2,), generator=gen(P), dtype=torch.int32)
    if P > 30:
        rows[7], rows[11], rows[P - 3] = -1, T, 2 ** 31 - 1  # no such token: zeros
    check_forward(xq, a, counts, packed, s, rows.cuda(), f"{P} {E} {N} {K}", tail=2)


@pytest.mark.parametrize("P,E,K", [(6, 4, 2560), (200, 4, 1028), (900, 4, 512)])
def test_grouped_equals_single(P, E, K):
    off = offsets_of(spread(P, E, 5, "skewed"))
    xq, a = bw.quant_act(bf16(P, K, seed=1))
    w = [experts(E, n, K, seed=n) for n in (300, 64, 17)]
    rows = torch.randperm(P, generator=gen(2)).to(torch.int32).cuda()
    for dt in ("i32", "f32", "bf16"):
        outs = bw.gemm_experts_grouped(xq, a, off, [p for p, _ in w], [s for _, s in w], dt, rows=rows)
        for (p, s), o in zip(w, outs):
            assert torch.equal(bw.gemm_experts(xq, a, off, p, s, dt, rows=rows), o)
            sorted_xq, sorted_a = xq[rows.long()].contiguous(), a[rows.long()].contiguous()
            assert torch.equal(bw.gemm_experts(sorted_xq, sorted_a, off, p, s, dt), o)


@pytest.mark.parametrize("c", [3, 40, 150, 300])
def test_rows_equal_the_dense_product(c):
    # bit for bit what the tiled product of one matrix gives
    E, N, K = 3, 200, 1024
    packed, s = experts(E, N, K, seed=1)
    xq, a = bw.quant_act(bf16(E * c, K, seed=c))
    for dt in ("f32", "bf16"):
        out = bw.gemm_experts(xq, a, offsets_of([c] * E), packed, s, dt)
        for e in range(E):
            r = slice(e * c, (e + 1) * c)
            want = bw.gemm(xq[r].clone(), a[r].clone(), packed[e].clone(), s[e].clone(), dt,
                           algo="tiled")
            assert torch.equal(out[r], want), (dt, e)


def test_offsets_that_make_no_sense():
    # rows outside 0 .. P and experts that run backwards: no access out of bounds, the others right
    P, E, N, K = 40, 5, 64, 256
    packed, s = experts(E, N, K, seed=1)
    xq, a = bw.quant_act(bf16(P, K, seed=2))
    dy = bf16(P, N, seed=3, hot=False)
    off = torch.tensor([-5, 10, 4, 30, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full((P, N), 5, dtype=torch.int32, device="cuda")
    bw.gemm_experts(xq, a, off, packed, s, "i32", out=out)
    dx = bw.grad_input_experts(dy, off, packed, s)
    dw = bw.grad_weight_experts(dy, xq, a, off)
    # expert 0: rows 0 .. 9; 1: none; 2: 4 .. 29 (over 0's); 3: 30 .. 39; 4: none
    for e, lo, hi in ((2, 10, 30), (3, 30, 40)):
        w = bw.unpack_weights(packed[e].clone(), K).double().t().contiguous()
        assert torch.equal(out[lo:hi].double(), xq[lo:hi].double() @ w)
    check_grad_input([dy[30:]], [packed[3].clone()], [s[3].clone()], K, dx[30:], "dx")
    check_grad_weight(dy[4:30].contiguous(), xq[4:30], a[4:30], "f32", dw[2], "dw")
    assert not dw[1].any() and not dw[4].any()


def test_a_long_table_of_tokens():
    # codes close to 2^31 bytes: the last tokens are found
    K, T = 4096, 524287
    packed, s = experts(2, 64, K, seed=1)
    xq = torch.zeros((T, K), dtype=torch.int8, device="cuda")
    a = torch.ones(T, device="cuda")
    tail, ta = bw.quant_act(bf16(4, K, seed=1))
    xq[-4:], a[-4:] = tail, ta
    rows = torch.tensor([T - 1, 0, T - 3, T - 4, T - 2], dtype=torch.int32, device="cuda")
    check_forward(xq, a, [2, 3], packed, s, rows, "long table", dts=("i32", "f32"))
    with pytest.raises(bw.BitnetError):  # one more token and 31 bits do not reach
        bw.gemm_experts(torch.zeros((T + 1, K), dtype=torch.int8, device="cuda"), torch.ones(T + 1, device="cuda"),
                        offsets_of([2, 3]), packed, s, rows=rows)


def test_outputs_past_32_bits():
    # more than 2^31 outputs, sorted rows whose codes pass 2^31 bytes as well
    P, E, N, K = 1_100_003, 3, 2048, 2048
    packed, s = experts(E, N, K, seed=1)
    xq = torch.zeros((P, K), dtype=torch.int8, device="cuda")
    a = torch.ones(P, device="cuda")
    tail, ta = bw.quant_act(bf16(5, K, seed=1))
    xq[-5:], a[-5:] = tail, ta
    off = offsets_of([500_000, 100_003, 500_000])
    out = bw.gemm_experts(xq, a, off, packed, s, "bf16")
    ref = (tail.double() @ weights64(packed[2].clone(), s[2], K).t().contiguous()) / ta.double()[:, None]
    close(out[-5:], ref, (BF + 3.1 * U) * ref.abs(), "last rows")
    assert not out[:-5].any()
    del xq
    dx = bw.grad_input_experts(out, off, packed, s)
    check_grad_input([out[-5:]], [packed[2].clone()], [s[2].clone()], K, dx[-5:], "last dx")
    assert not dx[:-5].any()


def test_more_tiles_than_a_launch():
    # 1472 row tiles of 16 times 16384 column tiles of 64 are more blocks than one launch takes
    E, N, K, c = 1024, 1 << 20, 4, 8
    packed = torch.randint(0, 3, (E, N, 4), device="cuda", dtype=torch.uint8)
    packed = (packed[..., 0] | packed[..., 1] << 2 | packed[..., 2] << 4 | packed[..., 3] << 6)[..., None].contiguous()
    s = torch.rand((E, N), device="cuda") + 0.5
    xq, a = bw.quant_act(bf16(E * c, K, seed=1))
    out = bw.gemm_experts(xq, a, offsets_of([c] * E), packed, s, "bf16")
    for e in (0, 511, 1023):
        r = slice(e * c, (e + 1) * c)
        ref = xq[r].double() @ weights64(packed[e].clone(), s[e], K).t().contiguous() / a[r].double()[:, None]
        close(out[r], ref, (BF + 3.1 * U) * ref.abs(), f"expert {e}")


# --------------------------------------------------------------------------- gradients

GRADS = [(1, 2, 1, 4), (3, 2, 17, 20), (5, 3, 640, 2560), (40, 4, 63, 252), (100, 16, 641, 2564), (300, 3, 257, 1028),
         (700, 8, 300, 516), (999, 5, 130, 260), (1200, 2, 256, 256), (4100, 4, 33, 64), (258, 64, 64, 640),
         (2100, 2, 2560, 512), (90, 200, 6, 20), (513, 4, 128, 4112), (1500, 64, 40, 2064), (1500, 64, 33, 2052)]


@pytest.mark.parametrize("P,E,N,K", GRADS)
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
def test_input_gradient(P, E, N, K, kind):
    counts = spread(P, E, P + E, kind)
    off = offsets_of(counts)
    dy = bf16(P + 2, N, seed=N, scale=1e-3, hot=False)
    dy[P:] = float("nan")  # rows of no expert
    packed, s = experts(E, N, K, seed=N)
    out = torch.full((P + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
    got = bw.grad_input_experts(dy, off, packed, s, out=out)
    assert got is out and (out[P:] == 5.0).all()
    at = 0
    for e, c in enumerate(counts):
        if c:
            check_grad_input([dy[at:at + c]], [packed[e].clone()], [s[e].clone()], K, out[at:at + c], f"{kind} expert {e}")
        at += c
    again = bw.grad_input_experts(dy, off, packed, s)
    assert torch.equal(again[:P], out[:P])


@pytest.mark.parametrize("P,E,Ns,K", [(10, 3, (640, 128), 512), (200, 4, (33, 0, 65), 252), (900, 4, (256, 256), 1024),
                                      (77, 5, (17, 18, 19, 20), 100)])
def test_input_gradient_of_several(P, E, Ns, K):
    counts = spread(P, E, 3, "skewed")
    off = offsets_of(counts)
    dys = [bf16(P, n, seed=n + i, scale=1e-3, hot=False) for i, n in enumerate(Ns)]
    w = [experts(E, n, K, seed=n + i) if n else (torch.empty((E, 0, K // 4), dtype=torch.uint8, device="cuda"),
                                                 torch.empty((E, 0), device="cuda")) for i, n in enumerate(Ns)]
    got = bw.grad_input_experts_grouped(dys, off, [p for p, _ in w], [s for _, s in w])
    at = 0
    for e, c in enumerate(counts):
        if c:
            check_grad_input([d[at:at + c] for d, n in zip(dys, Ns) if n], [p[e].clone() for (p, _), n in zip(w, Ns) if n],
                             [s[e].clone() for (_, s), n in zip(w, Ns) if n], K, got[at:at + c], f"expert {e}")
        at += c


@pytest.mark.parametrize("P,E,N,K", GRADS)
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_weight_gradient(P, E, N, K, kind, dt):
    counts = spread(P, E, P + E, kind)
    off = offsets_of(counts)
    dy = bf16(P + 2, N, seed=N, scale=1e-3, hot=False)
    dy[P:] = float("nan")
    xq, a = bw.quant_act_pow2(bf16(P + 2, K, seed=K))
    out = torch.full((E, N, K), 5.0, device="cuda").to(torch.float32 if dt == "f32" else torch.bfloat16)
    got = bw.grad_weight_experts(dy, xq, a, off, dt, out=out)
    assert got is out
    at = 0
    for e, c in enumerate(counts):
        if c:
            check_grad_weight(dy[at:at + c], xq[at:at + c], a[at:at + c], dt, out[e], f"{kind} expert {e}")
        else:
            assert not out[e].any()
        at += c
    # the same through the tokens of the rows
    T = P + 2
    perm = torch.randperm(T, generator=gen(1)).cuda()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T, device="cuda")
    again = bw.grad_weight_experts(dy, xq[perm].contiguous(), a[perm].contiguous(), off, dt,
                                   rows=inv.to(torch.int32))
    assert torch.equal(again, out)


def test_input_gradient_of_no_columns():
    # products without outputs have a zero gradient, in either tile, and rows of no expert stay
    for P, K in ((7, 64), (7, 20), (5000, 4096)):
        off = offsets_of([P, 0])
        none = (torch.empty((2, 0, K // 4), dtype=torch.uint8, device="cuda"), torch.empty((2, 0), device="cuda"))
        out = torch.full((P + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
        bw.grad_input_experts(torch.empty((P + 2, 0), dtype=torch.bfloat16, device="cuda"), off, *none, out=out)
        assert not out[:P].any() and (out[P:] == 5.0).all()


# sizes that reach the tiles of many rows and columns, and of long sums (those above are below their
# thresholds)
@pytest.mark.parametrize("P,E,N,K", [(500, 4, 16400, 2064), (4200, 2, 2100, 64), (700, 70, 1100, 1024)])
@pytest.mark.parametrize("kind", ["even", "skewed"])
def test_large_products(P, E, N, K, kind):
    test_product_of_sorted_rows(P, E, N, K, kind)


@pytest.mark.parametrize("P,E,N,K", [(600, 9, 1024, 2180), (600, 9, 1023, 2176), (1100, 3, 300, 260), (1100, 3, 301, 256),
                                     (40, 3, 1100, 260), (40, 3, 1104, 272), (1500, 64, 33, 1540),
                                     (1700, 4, 1280, 4100), (1100, 3, 1281, 1028), (1400, 20, 1023, 3856)])
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
def test_large_gradients(P, E, N, K, kind):
    test_input_gradient(P, E, N, K, kind)
    for dt in ("f32", "bf16"):
        test_weight_gradient(P, E, N, K, kind, dt)


def test_neighbours_stay_apart():
    # an expert's rows border on another's: values there that are not finite do not enter
    for N, K in ((33, 64), (32, 64), (641, 132)):
        E, counts = 3, [5, 7, 6]
        off = offsets_of(counts)
        packed, s = experts(E, N, K, seed=N)
        dy = bf16(18, N, seed=3, hot=False)
        xq, a = bw.quant_act_pow2(bf16(18, K, seed=4))
        dx, dw = bw.grad_input_experts(dy, off, packed, s), bw.grad_weight_experts(dy, xq, a, off)
        bad = dy.clone()
        bad[4], bad[12] = float("nan"), float("inf")
        dx2, dw2 = bw.grad_input_experts(bad, off, packed, s), bw.grad_weight_experts(bad, xq, a, off)
        keep = [i for i in range(18) if i not in (4, 12)]
        assert torch.equal(dx2[keep], dx[keep]) and torch.equal(dw2[1], dw[1])
        bad = dy.clone()
        bad[5:12] = float("nan")
        dw2 = bw.grad_weight_experts(bad, xq, a, off)
        assert torch.equal(dw2[0], dw[0]) and torch.equal(dw2[2], dw[2])
        assert torch.isnan(dw2[1]).all()


def test_empty_products():
    packed, s = experts(3, 16, 64, seed=1)
    off = offsets_of([0, 0, 0])
    q = torch.empty((0, 64), dtype=torch.int8, device="cuda")
    a = torch.empty(0, device="cuda")
    dy = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert bw.gemm_experts(q, a, off, packed, s).shape == (0, 16)
    assert bw.grad_input_experts(dy, off, packed, s).shape == (0, 64)
    assert not bw.grad_weight_experts(dy, q, a, off).any()
    # tokens, but every choice dropped
    xq, sa = bw.quant_act(bf16(4, 64, seed=1))
    rows = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((8, 16), 3.0, device="cuda")
    bw.gemm_experts(xq, sa, off, packed, s, rows=rows, out=out)
    assert (out == 3.0).all()
    assert not bw.grad_weight_experts(bf16(8, 16, seed=1), xq, sa, off, rows=rows).any()


# ----------------------------------------------------------------------------- combine

@pytest.mark.parametrize("T,J,D", [(1, 1, 4), (1, 8, 2560), (32, 8, 2560), (7, 3, 252), (65, 2, 1028), (5, 13, 4100),
                                   (1000, 2, 4096), (3, 64, 8192), (9, 5, 20)])
def test_combine(T, J, D):
    E = max(4, J)
    ids = torch.randint(-1, E, (T, J), generator=gen(T + J), dtype=torch.int32)
    if T > 2:
        ids[1] = -1   # a token none of whose choices is kept
    rows, offsets, slots = bw.expert_order(ids.cuda(), E)
    P = T * J
    y, w = bf16(P, D, seed=D, hot=False), f32(T, J, seed=J).abs()
    dout = bf16(T, D, seed=D + 1, hot=False)
    live = slots >= 0
    at = slots.clamp(min=0).long()
    y64 = torch.where(live[..., None], y[at].double(), 0.0)
    for weights in (w, None):
        c = torch.where(live, weights.double() if weights is not None else 1.0, 0.0)
        terms = y64 * c[..., None]
        ref = terms.sum(1)
        out = bw.combine_experts(y, slots, weights)
        close(out, ref, BF * ref.abs() + (1 + BF) * J * U * terms.abs().sum(1) + TINY, "sum")
        if T > 2:
            assert not out[1].any()
        dy = torch.full((P, D), 3.0, dtype=torch.bfloat16, device="cuda")
        got, dw = bw.combine_experts_backward(dout, y, slots, weights, out=dy)
        assert got is dy
        want = torch.full_like(dy, 3.0)  # rows of no choice stay
        grad = dout[:, None, :].expand(T, J, D).float()
        grad = (grad * weights[..., None] if weights is not None else grad).to(torch.bfloat16)
        want[slots[live].long()] = grad[live]
        assert torch.equal(dy, want)
        if weights is None:
            assert dw is None
        else:
            prod = y64 * dout[:, None, :].double()
            # a lane's terms, six lane steps, the product
            tol = (D / 64 + 16) * U * prod.abs().sum(2) + TINY
            close(dw, torch.where(live, prod.sum(2), 0.0), tol, "dweights")
            assert not dw[~live].any()


def test_combine_ignores_slots_outside():
    y = bf16(6, 64, seed=1)
    slots = torch.tensor([[0, 6], [2 ** 31 - 1, -7], [5, -1]], dtype=torch.int32, device="cuda")
    out = bw.combine_experts(y, slots)
    assert torch.equal(out[0], y[0]) and not out[1].any() and torch.equal(out[2], y[5])
    dy = torch.zeros_like(y)
    _, dw = bw.combine_experts_backward(out, y, slots, torch.ones((3, 2), device="cuda"), out=dy)
    assert torch.equal(dy[0], out[0]) and torch.equal(dy[5], out[2]) and not dy[1:5].any()
    assert dw[1].abs().max() == 0 and dw[0, 1] == 0 and dw[2, 1] == 0


# ------------------------------------------------------------------- the set as it is used

def moe_step(x, res, dy, gamma, ids, weights, gate, up, down, max_norm=0.5):
    """One training step through the residual's addition, norm, the experts' MLP and the sum, and
    back, with the gradients clipped."""
    E = gate[0].shape[0]
    xq, xa, s, rstd = bw.rmsnorm_quant(x, gamma, residual=res, scale="pow2", return_stats=True)
    rows, off, slots = bw.expert_order(ids, E)
    g, u = bw.gemm_experts_grouped(xq, xa, off, [gate[0], up[0]], [gate[1], up[1]], "bf16", rows=rows)
    hq, ha, ck = bw.swiglu_quant(g, u, scale="pow2", checkpoint=True)
    z = bw.gemm_experts(hq, ha, off, *down, "bf16")
    y = bw.combine_experts(z, slots, weights)
    dz, dweights = bw.combine_experts_backward(dy, z, slots, weights)
    dh = bw.grad_input_experts(dz, off, *down)
    dw_down = bw.grad_weight_experts(dz, hq, ha, off)
    dg, du = bw.swiglu_backward(dh, *ck)
    dw_gate = bw.grad_weight_experts(dg, xq, xa, off, rows=rows)
    dw_up = bw.grad_weight_experts(du, xq, xa, off, rows=rows)
    dpairs = bw.grad_input_experts_grouped([dg, du], off, [gate[0], up[0]], [gate[1], up[1]])
    dxn = bw.combine_experts(dpairs, slots)
    dx, dgamma = bw.rmsnorm_backward(dxn, s, gamma, rstd, dresidual=dy)
    grads = [dw_gate, dw_up, dw_down, dgamma]
    norm = bw.clip_grads(grads, max_norm)
    return [y, s, dx, dweights, norm] + grads


def moe_inputs(T=96, E=6, J=2, H=512, F=1028, seed=0):
    x, res = bf16(T, H, seed=seed, hot=False), bf16(T, H, seed=seed + 1, hot=False)
    dy = bf16(T, H, seed=seed + 2, scale=1e-2, hot=False)
    gamma = f32(H, seed=3, scale=0.1, shift=1.0)
    w, ids = torch.softmax(f32(T, E, seed=seed + 4), 1).topk(J, 1)
    return (x, res, dy, gamma, ids, (w / w.sum(1, keepdim=True)).contiguous(), experts(E, F, H, seed=5),
            experts(E, F, H, seed=6), experts(E, H, F, seed=7))


def test_moe_training_step():
    args = moe_inputs()
    x, res, dy, gamma, ids, weights, gate, up, down = args
    got = moe_step(*args)
    E, F, H = gate[0].shape[0], gate[0].shape[1], x.shape[1]

    class Round(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            a = pow2_of(t.abs().amax(1))[:, None]
            return torch.round(t * a) / a

        @staticmethod
        def backward(ctx, d):
            return d

    leaf = lambda t: t.detach().double().requires_grad_()
    s64, g64, w64 = leaf(got[1]), leaf(gamma), leaf(weights)
    dense = lambda w, k: leaf(torch.stack([weights64(w[0][e].clone(), w[1][e], k) for e in range(E)]))
    wg, wu, wd = dense(gate, H), dense(up, H), dense(down, F)
    xn = Round.apply(s64 * (s64.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * g64)
    y = torch.zeros_like(s64)
    for e in range(E):
        t, j = torch.where(ids == e)
        g, u = xn[t] @ wg[e].t(), xn[t] @ wu[e].t()
        h = Round.apply(g * torch.sigmoid(g) * u)
        y = y.index_add(0, t, w64[t, j][:, None] * (h @ wd[e].t()))
    (y + s64).backward(dy.double())
    grads = [wg.grad, wu.grad, wd.grad, g64.grad]
    norm = torch.stack([g.square().sum() for g in grads]).sum().sqrt()
    c = min(1.0, 0.5 / norm.item())
    refs = [y.detach(), s64.detach(), s64.grad, w64.grad, norm] + [g * c for g in grads]
    # bf16 activations between the stages and 8-bit g and u in the backward: 1/254 of a row's
    # maximum (some four standard deviations) per checkpointed value, twice, and codes that fall
    # to the other side; 5% in the 2-norm covers three such terms
    for k, (p, q) in enumerate(zip(got, refs)):
        rel = ((p.double() - q).norm() / q.norm()).item()
        assert rel <= 0.05, f"output {k}: {rel:.3g}"
    assert torch.equal(got[1], (x.float() + res.float()).to(torch.bfloat16))


def test_moe_steps_in_graphs():
    # two captured steps of different sizes, replayed in turn with eager work between
    steps = []
    for T, J, seed in ((96, 2, 0), (33, 3, 50)):
        args = moe_inputs(T=T, J=J, seed=seed)
        want = [t.clone() for t in moe_step(*args)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            moe_step(*args)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = moe_step(*args)
        steps.append((args, want, graph, outs))
    for rep in range(3):
        for args, want, graph, outs in steps:
            for t in outs:
                t.zero_()
            graph.replay()
            eager = moe_step(*args)
            torch.cuda.synchronize()
            for k, (p, q, r) in enumerate(zip(outs, want, eager)):
                assert torch.equal(p, q), f"replay {rep} output {k}"
                assert torch.equal(r, q), f"eager {rep} output {k}"
        # other tokens for the experts, in the captured buffers
        args, want, graph, outs = steps[0]
        args[4].copy_(args[4].flip(0).clone())
        steps[0] = (args, [t.clone() for t in moe_step(*args)], graph, outs)


def test_two_streams_at_once():
    args = [moe_inputs(seed=s) for s in (0, 9)]
    want = [[t.clone() for t in moe_step(*a)] for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for s, a in zip(streams, args):
        with torch.cuda.stream(s):
            got.append([moe_step(*a) for _ in range(3)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for run in g:
            assert all(torch.equal(p, q) for p, q in zip(run, w))


def test_moe_decode_step_of_a_padded_batch():
    # padding tokens have no expert: the others come out as they do alone
    x, res, _, gamma, ids, weights, gate, up, down = moe_inputs(T=8, E=16, J=4, H=2560, F=640)
    ids = ids.to(torch.int32)
    ids[5:] = -1

    def mlp(x, res, ids, weights):
        xq, xa, s = bw.rmsnorm_quant(x, gamma, residual=res)
        rows, off, slots = bw.expert_order(ids, 16)
        g, u = bw.gemm_experts_grouped(xq, xa, off, [gate[0], up[0]], [gate[1], up[1]], "bf16", rows=rows)
        hq, ha = bw.swiglu_quant(g, u)
        return bw.combine_experts(bw.gemm_experts(hq, ha, off, *down, "bf16"), slots, weights), s
    y, s = mlp(x, res, ids, weights)
    assert not y[5:].any()
    for n in (1, 5):
        cut = [t[:n].contiguous() for t in (x, res, ids, weights)]
        y2, s2 = mlp(*cut)
        assert torch.equal(y2, y[:n]) and torch.equal(s2, s[:n])


def test_refusals():
    E, N, K = 4, 16, 256
    packed, s = experts(E, N, K, seed=1)
    x = bf16(6, K, seed=1)
    xq, a = bw.quant_act(x)
    off = offsets_of([2, 2, 1, 1])
    dy = bf16(6, N, seed=2)
    with pytest.raises(ValueError):
        bw.gemm_experts(xq, a, off[:-1], packed, s)
    with pytest.raises(TypeError):
        bw.gemm_experts(xq, a, off.long(), packed, s)
    with pytest.raises(ValueError):
        bw.gemm_experts(xq[:, :128].contiguous(), a, off, packed, s)
    with pytest.raises(ValueError):
        bw.gemm_experts(xq, a, off, packed[0], s[0])
    with pytest.raises(ValueError):
        bw.gemm_experts_grouped(xq, a, off, [], [])
    with pytest.raises(bw.BitnetError):
        bw.gemm_experts_grouped(xq, a, off, [packed] * 5, [s] * 5)
    with pytest.raises(ValueError):
        bw.grad_input_experts(dy[:, :8].contiguous(), off, packed, s)
    with pytest.raises(ValueError):
        bw.grad_input_experts_grouped([dy], off, [packed, packed], [s, s])
    with pytest.raises(ValueError):
        bw.grad_weight_experts(dy, xq, a, off, "i32")
    with pytest.raises(bw.BitnetError):  # five rows of codes for six of dy
        bw.grad_weight_experts(dy, xq[:5], a[:5], off)
    with pytest.raises(bw.BitnetError):
        bw.grad_weight_experts(dy, xq, a, off, rows=torch.zeros(6, dtype=torch.int32, device="cuda"),
                               workspace=False)
    with pytest.raises(TypeError):
        bw.expert_order(torch.zeros((3, 2), device="cuda"), 4)
    for E in (0, 1025, -1):
        with pytest.raises(bw.BitnetError):
            bw.expert_order(torch.zeros((3, 2), dtype=torch.int32, device="cuda"), E)
    slots = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        bw.combine_experts(x, slots, torch.ones((2, 2), device="cuda"))
    with pytest.raises(bw.BitnetError):
        bw.combine_experts(bf16(6, 6, seed=1), slots)
    with pytest.raises(TypeError):
        bw.combine_experts(x, slots.long())
    with pytest.raises(ValueError):
        bw.combine_experts_backward(x, x, slots)      # six tokens of dout, three of slots
