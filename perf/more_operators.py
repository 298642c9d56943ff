"""A mixture-of-experts layer of BitLinear products: what is timed, its plain form and its exact values.

Operators: root-mean-square norm with the residual's addition and int8 codes (forward and
backward), the ternary product grouped by expert with ragged sizes (forward, both gradients),
the order of tokens by expert with the weighted sum of their outputs (and its backward), and
the gradients' global norm with clipping.

Activations and their gradients are bf16; norm weights, statistics, scales and router weights
fp32.  T tokens choose J of E experts each; the P = T J pairs, sorted by expert, are the rows
of the products: row p belongs to expert e for offsets[e] <= p < offsets[e + 1] and to the
token rows[p]; slots[t, j] is the row of token t's j-th choice.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the norm of a decode step: one token, the residual added, codes for the projections
        dict(name="rms_token", op="rms", m=1, k=2560, scale="absmax"),
        # training forward at 8B width: new residual stream, codes, statistics
        dict(name="rms_quant_8b", op="rms", m=2048, k=4096, scale="pow2"),
        # a long training batch of ragged sizes, the norm's input kept in 8 bits
        dict(name="rms_back_ragged", op="rms_back", m=8191, k=4100, ckpt=True),
        # the vectors and small matrices of a few layers: latency only
        dict(name="clip_small", op="clip", layers=4, n=641, k=260, out="bf16"),
        # every gradient of 2B-shaped layers: bandwidth
        dict(name="clip_2b", op="clip", layers=4, n=6912, k=2560, out="f32"),
        # a decode step's token through gate and up of two of eight 8B-wide experts
        dict(name="experts_token", op="experts", t=1, j=2, e=8, n=14336, k=4096, groups=2),
        # a decode batch over many small experts: a few ragged rows for each
        dict(name="experts_decode", op="experts", t=32, j=8, e=64, n=640, k=2560, groups=2),
        # a prompt through the gate and up of 8B-wide experts: the largest product
        dict(name="experts_prefill_8b", op="experts", t=2048, j=2, e=8, n=14336, k=4096, groups=2),
        # ragged in every size: odd rows, columns off the tile, some experts nearly idle
        dict(name="experts_back_ragged", op="experts_back", t=129, j=2, e=16, n=641, k=2564, out="bf16"),
        # training step of 2B-wide experts, the latent weights' gradients in fp32
        dict(name="experts_back_2b", op="experts_back", t=2048, j=2, e=8, n=6912, k=2560, out="f32"),
        # order and sum of a decode batch over many experts: latency
        dict(name="route_decode", op="route", t=32, j=8, e=64, d=2560),
        # the same for a long batch with its backward
        dict(name="route_8b", op="route", t=8192, j=2, e=8, d=4096),
    ]


def _size(rng, lo, hi, mult=1):
    """A multiple of `mult` spread over the logarithm of lo .. hi."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["rms", "rms_back", "clip", "experts", "experts", "experts_back", "route"])
    if op in ("rms", "rms_back"):
        c = dict(op=op, m=_size(rng, 1, 8192), k=_size(rng, 256, 8192, 4))
        while c["m"] * c["k"] > 8192 * 4096:
            c["m"] = max(1, c["m"] // 2)
        if op == "rms":
            c["scale"] = rng.choice(["absmax", "pow2"])
        else:
            c["ckpt"] = rng.random() < 0.5
        return c
    if op == "clip":
        c = dict(op=op, layers=rng.randint(1, 8), n=_size(rng, 64, 6912), k=_size(rng, 64, 4096, 4),
                 out=rng.choice(["f32", "bf16"]))
        while c["layers"] * c["n"] * c["k"] > 4 * 6912 * 2560:
            c["n"] = max(64, c["n"] // 2)
        return c
    c = dict(op=op, e=_size(rng, 2, 128), t=_size(rng, 1, 4096))
    c["j"] = rng.randint(1, min(8, c["e"]))
    if op == "route":
        c["d"] = _size(rng, 256, 8192, 4)
        while c["t"] * c["j"] * c["d"] > 8192 * 2 * 4096:
            c["t"] = max(1, c["t"] // 2)
        return c
    c.update(n=_size(rng, 320, 14336), k=_size(rng, 320, 14336, 4))
    while c["e"] * c["n"] * c["k"] > 8 * 6912 * 2560:
        c["n"], c["k"] = max(320, c["n"] // 2), max(320, c["k"] // 8 * 4)
        if c["n"] == c["k"] == 320:
            break
    while c["t"] * c["j"] * c["n"] * c["k"] > 4096 * 6912 * 2560:
        c["t"] = max(1, c["t"] // 2)
    if op == "experts":
        c["groups"] = rng.choice([1, 2])
    else:
        c["out"] = rng.choice(["f32", "bf16"])
    return c


# ----------------------------------------------------------------------------- inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _acts(m, k, gen):
    """bf16 N(0, 1) activations with 1% of the channels twenty times larger."""
    x = _randn((m, k), gen)
    hot = torch.rand((k,), generator=gen, device="cuda") < 0.01
    return torch.where(hot[None, :], 20.0 * x, x).to(torch.bfloat16)


def _grads(m, n, gen):
    """bf16 gradients: small, with a scale of their own per token."""
    s = 1e-3 * torch.exp(_randn((m, 1), gen))
    return (s * _randn((m, n), gen)).to(torch.bfloat16)


def _codes8(x, pow2=True):
    """int8 codes and scales of bf16 rows: the largest power of two that keeps |x a| <= 127, or
    127 / max |x|."""
    xf = x.to(torch.float32)
    amax = xf.abs().amax(1).clamp(min=1e-5)
    if pow2:
        mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1)
        a = torch.ldexp(torch.ones_like(amax), torch.where(mant <= 127.0 / 128.0, 7 - ex, 6 - ex))
    else:
        a = 127.0 / amax
    return torch.round(xf * a[:, None]).to(torch.int8), a


def _ternary(e, n, k, gen):
    """2-bit codes (e, n, k / 4) and scales (e, n) of latent weights N(0, 0.02^2)."""
    packed, scale = [], []
    for _ in range(e):
        w = 0.02 * _randn((n, k), gen)
        s = w.abs().mean(1).clamp(min=1e-5)
        q = (torch.round(w / s[:, None]).clamp(-1, 1) + 1).to(torch.uint8).view(n, k // 4, 4)
        packed.append(q[..., 0] | (q[..., 1] << 2) | (q[..., 2] << 4) | (q[..., 3] << 6))
        scale.append(s)
    return torch.stack(packed), torch.stack(scale)


def _choices(t, j, e, gen):
    """A router's choices (t, j) of experts, some of them more popular, and their weights."""
    logits = _randn((t, e), gen) + 0.7 * _randn((1, e), gen)
    w, ids = torch.softmax(logits, 1).topk(j, 1)
    return ids.to(torch.int32), w / w.sum(1, keepdim=True)


def _order(ids, e):
    """Stable order of the pairs by expert: tokens of the rows, offsets, rows of the pairs."""
    flat = ids.reshape(-1).to(torch.int64)
    by = torch.argsort(flat, stable=True)
    ends = torch.searchsorted(flat[by], torch.arange(e + 1, device=flat.device))
    slots = torch.empty_like(by)
    slots[by] = torch.arange(by.numel(), device=by.device)
    i32 = torch.int32
    return (by // ids.shape[1]).to(i32), ends.to(i32), slots.to(i32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = dict(op=op)
    if op in ("rms", "rms_back"):
        m, k = case["m"], case["k"]
        x = _acts(m, k, gen)
        st.update(x=x, weight=1.0 + 0.1 * _randn((k,), gen))
        if op == "rms":
            st.update(res=(2.0 * _randn((m, k), gen)).to(torch.bfloat16), scale=case["scale"])
        else:
            st.update(rstd=torch.rsqrt(x.double().square().mean(1) + EPS).float(),
                      dy=_grads(m, k, gen), dres=_grads(m, k, gen), x_scale=None)
            if case["ckpt"]:
                st["x"], st["x_scale"] = _codes8(x)
    elif op == "clip":
        dt = torch.float32 if case["out"] == "f32" else torch.bfloat16
        n, k = case["n"], case["k"]
        grads = []
        for _ in range(case["layers"]):  # a matrix, its transposed shape's half, two norms' vectors
            for shape, kind in (((n, k), dt), ((k, (n + 1) // 2), dt), ((k,), torch.float32),
                                ((n,), torch.float32)):
                grads.append((1e-3 * _randn(shape, gen)).to(kind))
        st.update(grads=grads, out=[torch.empty_like(g) for g in grads], max_norm=0.5)
    elif op == "route":
        ids, w = _choices(case["t"], case["j"], case["e"], gen)
        p, d = ids.numel(), case["d"]
        st.update(ids=ids, weights=w, e=case["e"], y=_acts(p, d, gen), dout=_grads(case["t"], d, gen))
    else:
        e, n, k = case["e"], case["n"], case["k"]
        ids, _ = _choices(case["t"], case["j"], e, gen)
        rows, offsets, _ = _order(ids, e)
        xq, a = _codes8(_acts(case["t"], k, gen), pow2=op != "experts")
        st.update(xq=xq, a=a, rows=rows, offsets=offsets,
                  most=int((offsets[1:] - offsets[:-1]).max()))
        w = [_ternary(e, n, k, gen) for _ in range(case.get("groups", 1))]
        st.update(packed=[p for p, _ in w], s=[s for _, s in w])
        if op == "experts_back":
            st.update(dy=_grads(rows.numel(), n, gen),
                      out=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    return st


# ------------------------------------------------------------------------- plain forms

def _rms(x, res, weight, scale):
    s = (x.to(torch.float32) + res.to(torch.float32)).to(torch.bfloat16)
    sf = s.to(torch.float32)
    rstd = torch.rsqrt(sf.square().mean(1) + EPS)
    y = (sf * rstd[:, None] * weight).to(torch.bfloat16)
    c, a = _codes8(y, scale == "pow2")
    return (c.to(torch.float32) / a[:, None]).to(torch.bfloat16), s, rstd


def _rms_back(dy, x, x_scale, dres, weight, rstd):
    xf = x.to(torch.float32)
    if x_scale is not None:
        xf = xf / x_scale[:, None]
    z = xf * rstd[:, None]
    dyf = dy.to(torch.float32)
    g = dyf * weight
    dx = rstd[:, None] * (g - z * (g * z).mean(1, keepdim=True)) + dres.to(torch.float32)
    return dx.to(torch.bfloat16), (dyf * z).sum(0)


def _clip(grads, max_norm):
    squares = torch.stack([g.to(torch.float64).square().sum() for g in grads])
    norm = squares.sum().sqrt().to(torch.float32)
    c = (max_norm / (norm + 1e-6)).clamp(max=1.0)
    return [(g.to(torch.float32) * c).to(g.dtype) for g in grads], norm


def _weights(packed, s):
    """fp32 weights (..., n, k) of packed codes and scales."""
    w = torch.stack([packed & 3, (packed >> 2) & 3, (packed >> 4) & 3, packed >> 6], -1)
    return (w.flatten(-2).to(torch.float32) - 1.0) * s[..., None]


def _places(offsets, p):
    """Expert of every row and its place among the expert's rows."""
    at = torch.arange(p, device=offsets.device)
    e = torch.searchsorted(offsets[1:].contiguous(), at.to(torch.int32), right=True)
    return e, at - offsets[e]


def _padded(rows, e, place, experts, most):
    """Rows (p, k) as (experts, most, k), zeros behind an expert's last."""
    pad = torch.zeros((experts, most, rows.shape[1]), dtype=torch.float32, device=rows.device)
    pad[e, place] = rows
    return pad


def _experts(st):
    e, place = _places(st["offsets"], st["rows"].numel())
    rows = st["rows"].to(torch.int64)
    x = st["xq"][rows].to(torch.float32) / st["a"][rows][:, None]
    experts = st["packed"][0].shape[0]
    if rows.numel() < experts:  # a few rows: each with its expert's weights
        return [torch.bmm(_weights(p[e], s[e]), x[:, :, None])[:, :, 0].to(torch.bfloat16)
                for p, s in zip(st["packed"], st["s"])]
    x = _padded(x, e, place, experts, st["most"])
    return [torch.bmm(x, _weights(p, s).transpose(1, 2).contiguous())[e, place].to(torch.bfloat16)
            for p, s in zip(st["packed"], st["s"])]


def _experts_back(st):
    e, place = _places(st["offsets"], st["rows"].numel())
    rows = st["rows"].to(torch.int64)
    experts, most = st["packed"][0].shape[0], st["most"]
    dy = _padded(st["dy"].to(torch.float32), e, place, experts, most)
    dx = torch.bmm(dy, _weights(st["packed"][0], st["s"][0]))[e, place].to(torch.bfloat16)
    x = _padded(st["xq"][rows].to(torch.float32) / st["a"][rows][:, None], e, place, experts, most)
    return dx, torch.bmm(dy.transpose(1, 2).contiguous(), x).to(st["out"])


def _route(st):
    rows, offsets, slots = _order(st["ids"], st["e"])
    at = slots.to(torch.int64)
    y, w = st["y"][at].to(torch.float32), st["weights"]
    d = st["dout"].to(torch.float32)
    out = (y * w[:, :, None]).sum(1).to(torch.bfloat16)
    dw = (y * d[:, None, :]).sum(2)
    dy = torch.empty_like(st["y"])
    dy[at.reshape(-1)] = (w[:, :, None] * d[:, None, :]).to(torch.bfloat16).flatten(0, 1)
    return rows, offsets, slots, out, dy, dw


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    if op == "rms":
        return _rms(state["x"], state["res"], state["weight"], state["scale"])
    if op == "rms_back":
        return _rms_back(state["dy"], state["x"], state["x_scale"], state["dres"], state["weight"],
                         state["rstd"])
    if op == "clip":
        return _clip(state["grads"], state["max_norm"])
    if op == "route":
        return _route(state)
    return _experts(state) if op == "experts" else _experts_back(state)


def _run_own(op, st):
    import ternary_weight_linear_token_amd as bw
    if op == "rms":
        xq, a, s, rstd = bw.rmsnorm_quant(st["x"], st["weight"], eps=EPS, residual=st["res"],
                                          scale=st["scale"], return_stats=True)
        return bw.dequant_act(xq, a), s, rstd
    if op == "rms_back":
        return bw.rmsnorm_backward(st["dy"], st["x"], st["weight"], st["rstd"],
                                   x_scale=st["x_scale"], dresidual=st["dres"])
    if op == "clip":
        norm = bw.clip_grads(st["grads"], st["max_norm"], out=st["out"])
        return st["out"], norm
    if op == "route":
        rows, offsets, slots = bw.expert_order(st["ids"], st["e"])
        out = bw.combine_experts(st["y"], slots, st["weights"])
        dy, dw = bw.combine_experts_backward(st["dout"], st["y"], slots, st["weights"])
        return rows, offsets, slots, out, dy, dw
    if op == "experts":
        return bw.gemm_experts_grouped(st["xq"], st["a"], st["offsets"], st["packed"], st["s"], "bf16",
                                       rows=st["rows"])
    dx = bw.grad_input_experts(st["dy"], st["offsets"], st["packed"][0], st["s"][0])
    dw = bw.grad_weight_experts(st["dy"], st["xq"], st["a"], st["offsets"], out_dtype=st["out"],
                                rows=st["rows"])
    return dx, dw


# -------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "rms":  # x and the residual in; the sum, the codes' values and statistics out
        m, k = case["m"], case["k"]
        return dict(bytes=8 * m * k + 4 * k + 4 * m, flops=8 * m * k)
    if op == "rms_back":
        m, k = case["m"], case["k"]
        return dict(bytes=(7 if case["ckpt"] else 8) * m * k + 8 * m + 8 * k, flops=12 * m * k)
    if op == "clip":
        n, k = case["n"], case["k"]
        size = 4 if case["out"] == "f32" else 2
        values = n * k + k * ((n + 1) // 2)
        return dict(bytes=2 * case["layers"] * (size * values + 4 * (n + k)),
                    flops=3 * case["layers"] * (values + n + k))
    t, j, e = case["t"], case["j"], case["e"]
    p = t * j
    if op == "route":
        d = case["d"]
        return dict(bytes=4 * p * d + 4 * t * d + 20 * p + 4 * e, flops=5 * p * d)
    n, k, g = case["n"], case["k"], case.get("groups", 1)
    if op == "experts":
        return dict(bytes=t * k + 8 * p + g * (min(e, p) * n * (k // 4 + 4) + 2 * p * n),
                    flops=2 * g * p * n * k)
    return dict(bytes=2 * p * n + min(e, p) * n * (k // 4 + 4) + 2 * p * k + t * k + 8 * p
                + (4 if case["out"] == "f32" else 2) * e * n * k, flops=4 * p * n * k)


# ------------------------------------------------------------------------ exact values

def exact(case, seed):
    """The outputs in 64 bits, from the definitions.  A value that went through 8 bits of
    computed numbers has none: next to a border of the codes it is a step off or it is not."""
    st = prepare(case, seed)
    op = case["op"]
    d = {key: v.double() for key, v in st.items() if isinstance(v, torch.Tensor)}
    if op == "rms":
        s = d["x"] + d["res"]
        kept = s.to(torch.bfloat16).double()  # the stream that is normalized is the stored one
        return None, s, ((kept * kept).sum(1) / case["k"] + EPS) ** -0.5
    if op == "rms_back":
        k = case["k"]
        x = d["x"] if st["x_scale"] is None else d["x"] / d["x_scale"].unsqueeze(1)
        r = d["rstd"].unsqueeze(1)
        q = d["dy"] * d["weight"]
        dot = torch.einsum("mk,mk->m", q, x).unsqueeze(1)
        return q * r - x * r ** 3 * dot / k + d["dres"], torch.einsum("mk,mk,m->k", d["dy"], x, d["rstd"])
    if op == "clip":
        norm = math.sqrt(sum(float(torch.dot(g.double().flatten(), g.double().flatten()))
                             for g in st["grads"]))
        c = min(1.0, st["max_norm"] / (norm + 1e-6))
        return [g.double() * c for g in st["grads"]], torch.tensor(norm, dtype=torch.float64)
    if op == "route":
        rows = torch.empty(st["ids"].numel(), dtype=torch.int64)
        flat = st["ids"].flatten().tolist()
        ranked = sorted(range(len(flat)), key=lambda i: (flat[i], i))
        for place, i in enumerate(ranked):
            rows[i] = place
        at = rows.view(st["ids"].shape).to("cuda")
        y, w, do = d["y"], d["weights"], d["dout"]
        out, dy, dw = torch.zeros_like(do), torch.empty_like(y), torch.empty_like(w)
        for c in range(case["j"]):
            out += w[:, c, None] * y[at[:, c]]
            dy[at[:, c]] = w[:, c, None] * do
            dw[:, c] = torch.einsum("td,td->t", y[at[:, c]], do)
        return None, None, None, out, dy, dw
    n, k = case["n"], case["k"]
    ends = st["offsets"].tolist()
    rows = st["rows"].to(torch.int64)
    x = d["xq"][rows] / d["a"][rows].unsqueeze(1)

    def dense(g, e):  # expert e's weights of matrix g
        digits = st["packed"][g][e].to(torch.int64).unsqueeze(2) // torch.tensor(
            [1, 4, 16, 64], device="cuda") % 4
        return (digits.reshape(n, k) - 1).double() * st["s"][g][e].double().unsqueeze(1)
    if op == "experts":
        out = [torch.zeros((rows.numel(), n), dtype=torch.float64, device="cuda") for _ in st["packed"]]
        for e in range(case["e"]):
            if ends[e] < ends[e + 1]:
                for g in range(len(out)):
                    torch.mm(x[ends[e]:ends[e + 1]], dense(g, e).t(), out=out[g][ends[e]:ends[e + 1]])
        return out
    if case["e"] * n * k > 1 << 29:
        return None
    dx = torch.zeros((rows.numel(), k), dtype=torch.float64, device="cuda")
    dw = torch.zeros((case["e"], n, k), dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        if ends[e] < ends[e + 1]:
            dy = d["dy"][ends[e]:ends[e + 1]]
            dx[ends[e]:ends[e + 1]] = torch.mm(dy, dense(0, e))
            dw[e] = torch.mm(dy.t().contiguous(), x[ends[e]:ends[e + 1]])
    return dx, dw
