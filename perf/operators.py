"""The training side of a BitLinear layer: what is timed, its plain form and its exact values.

Operators: layer norm (forward, forward with the int8 codes fused, backward from bf16 inputs
or from their 8-bit checkpoint), SwiGLU with 8-bit checkpoints of its inputs (forward and
backward), the input gradient through packed ternary weights, and the weight gradient from
int8 activation codes.

Activations and their gradients are bf16; norm weights, statistics and scales fp32.  An
8-bit checkpoint holds int8 codes c and one power-of-two scale a per token: x ~ c / a.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the norm in front of a decode step's projections: one token, latency only
        dict(name="norm_token", op="norm", m=1, k=2560),
        # training forward of an 8B-wide block: norm, int8 codes and statistics in one go;
        # the codes come back as the values they stand for
        dict(name="norm_quant_8b", op="norm_quant", m=2048, k=4096),
        # a short ragged batch, a row length off every power of two
        dict(name="norm_back_ragged", op="norm_back", m=333, k=2564, ckpt=False),
        # a long training batch, the norm's input kept in 8 bits
        dict(name="norm_back_8b", op="norm_back", m=8192, k=4096, ckpt=True),
        # the MLP's gate, 2B width, a small micro-batch
        dict(name="swiglu_2b", op="swiglu", m=64, n=6912),
        # the same at 8B width and a full batch
        dict(name="swiglu_8b", op="swiglu", m=2048, n=14336),
        # a few tokens through the 2B output projection: the weights' bytes and latency count
        dict(name="grad_input_4", op="grad_input", m=4, n1=2560, n2=0, n3=0, k=2560),
        # q, k and v of a 2B layer share their input: the three gradients are one sum
        dict(name="grad_input_2b_qkv", op="grad_input", m=512, n1=2560, n2=640, n3=640, k=2560),
        # gate and up of an 8B layer, a full batch: the largest product
        dict(name="grad_input_8b", op="grad_input", m=2048, n1=14336, n2=14336, n3=0, k=4096),
        # ragged in every size: odd tokens, odd rows, columns off the tile
        dict(name="grad_weight_ragged", op="grad_weight", m=129, n=641, k=2564, out="bf16"),
        # a 2B gate projection, the latent weight's gradient in fp32
        dict(name="grad_weight_2b", op="grad_weight", m=512, n=6912, k=2560, out="f32"),
        # an 8B down projection, a full batch
        dict(name="grad_weight_8b", op="grad_weight", m=2048, n=4096, k=14336, out="bf16"),
    ]


def _size(rng, lo, hi, mult=1):
    """A multiple of `mult` spread over the logarithm of lo .. hi."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["norm", "norm_quant", "norm_back", "swiglu", "grad_input", "grad_weight"])
    if op in ("norm", "norm_quant", "norm_back"):
        c = dict(op=op, m=_size(rng, 1, 8192), k=_size(rng, 256, 8192, 4))
        while c["m"] * c["k"] > 8192 * 4096:
            c["m"] = max(1, c["m"] // 2)
        if op == "norm_back":
            c["ckpt"] = rng.random() < 0.5
        return c
    if op == "swiglu":
        c = dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 640, 28672, 4))
        while c["m"] * c["n"] > 2048 * 14336:
            c["m"] = max(1, c["m"] // 2)
        return c
    c = dict(op=op, m=_size(rng, 1, 4096), k=_size(rng, 640, 14336, 4))
    if op == "grad_input":
        groups = rng.choice([1, 1, 2, 3])
        ns = [_size(rng, 640, 14336) for _ in range(groups)] + [0, 0]
        c.update(n1=ns[0], n2=ns[1], n3=ns[2])
        total = sum(ns)
    else:
        c.update(n=_size(rng, 640, 14336), out=rng.choice(["f32", "bf16"]))
        total = c["n"]
    while total * c["k"] > 28672 * 4096:
        c["k"] = max(640, c["k"] // 8 * 4)
        if c["k"] == 640:
            break
    while c["m"] * total * c["k"] > 2048 * 4096 * 14336:
        c["m"] = max(1, c["m"] // 2)
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


def _codes8(x):
    """int8 codes and power-of-two scales of bf16 rows (the checkpoint of x)."""
    xf = x.to(torch.float32)
    amax = xf.abs().amax(1).clamp(min=1e-5)
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1)
    p = torch.where(mant <= 127.0 / 128.0, 7 - ex, 6 - ex)
    a = torch.ldexp(torch.ones_like(amax), p)
    return torch.round(xf * a[:, None]).to(torch.int8), a


def _ternary(n, k, gen):
    """2-bit codes (n, k / 4) and scales of latent weights N(0, 0.02^2)."""
    w = 0.02 * _randn((n, k), gen)
    s = w.abs().mean(1).clamp(min=1e-5)
    q = (torch.round(w / s[:, None]).clamp(-1, 1) + 1).to(torch.uint8).view(n, k // 4, 4)
    packed = q[..., 0] | (q[..., 1] << 2) | (q[..., 2] << 4) | (q[..., 3] << 6)
    return packed.contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, m = case["op"], case["m"]
    st = dict(op=op)
    if op in ("norm", "norm_quant", "norm_back"):
        k = case["k"]
        x = _acts(m, k, gen) + 0.25
        st.update(x=x, weight=1.0 + 0.1 * _randn((k,), gen), bias=0.1 * _randn((k,), gen))
        if op == "norm_back":
            xd = x.to(torch.float64)
            mean = xd.mean(1)
            var = (xd - mean[:, None]).square().mean(1)
            st.update(mean=mean.float(), rstd=torch.rsqrt(var + EPS).float(), dy=_grads(m, k, gen),
                      scale=None)
            if case["ckpt"]:
                st["x"], st["scale"] = _codes8(x)
    elif op == "swiglu":
        st.update(g=_randn((m, case["n"]), gen).mul_(2.0).to(torch.bfloat16),
                  u=_acts(m, case["n"], gen), dh=_grads(m, case["n"], gen))
    elif op == "grad_input":
        ns = [n for n in (case["n1"], case["n2"], case["n3"]) if n]
        w = [_ternary(n, case["k"], gen) for n in ns]
        st.update(dy=[_grads(m, n, gen) for n in ns], packed=[p for p, _ in w], s=[s for _, s in w])
    else:
        xq, a = _codes8(_acts(m, case["k"], gen))
        st.update(dy=_grads(m, case["n"], gen), xq=xq, a=a,
                  out=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    return st


# ------------------------------------------------------------------------- plain forms

def _norm(x, weight, bias):
    xf = x.to(torch.float32)
    mean = xf.mean(1)
    xc = xf - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + EPS)
    return (xc * rstd[:, None] * weight + bias).to(torch.bfloat16), mean, rstd


def _norm_back(dy, x, scale, weight, mean, rstd):
    xf = x.to(torch.float32)
    if scale is not None:
        xf = xf / scale[:, None]
    xh = (xf - mean[:, None]) * rstd[:, None]
    dyf = dy.to(torch.float32)
    g = dyf * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(torch.bfloat16), (dyf * xh).sum(0), dyf.sum(0)


def _swiglu(g, u, dh):
    gf, uf = g.to(torch.float32), u.to(torch.float32)
    h = (gf / (1.0 + torch.exp(-gf)) * uf).to(torch.bfloat16)
    (gq, ga), (uq, ua) = _codes8(g), _codes8(u)
    gf, uf = gq.to(torch.float32) / ga[:, None], uq.to(torch.float32) / ua[:, None]
    sig = 1.0 / (1.0 + torch.exp(-gf))
    d = dh.to(torch.float32)
    dg = d * uf * sig * (1.0 + gf * (1.0 - sig))
    return h, dg.to(torch.bfloat16), (d * gf * sig).to(torch.bfloat16)


def _grad_input(dy, packed, s):
    p, s = torch.cat(packed), torch.cat(s)
    w = torch.stack([p & 3, (p >> 2) & 3, (p >> 4) & 3, p >> 6], 2).view(p.shape[0], -1)
    w = (w.to(torch.float32) - 1.0) * s[:, None]
    return (torch.cat(dy, 1).to(torch.float32) @ w).to(torch.bfloat16)


def _grad_weight(dy, xq, a, out):
    x = xq.to(torch.float32) / a[:, None]
    return (dy.to(torch.float32).t() @ x).to(out)


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    if op == "norm":
        return _norm(state["x"], state["weight"], state["bias"])[0]
    if op == "norm_quant":
        y, mean, rstd = _norm(state["x"], state["weight"], state["bias"])
        c, a = _codes8(y)
        return (c.to(torch.float32) / a[:, None]).to(torch.bfloat16), mean, rstd
    if op == "norm_back":
        return _norm_back(state["dy"], state["x"], state["scale"], state["weight"], state["mean"],
                          state["rstd"])
    if op == "swiglu":
        return _swiglu(state["g"], state["u"], state["dh"])
    if op == "grad_input":
        return _grad_input(state["dy"], state["packed"], state["s"])
    return _grad_weight(state["dy"], state["xq"], state["a"], state["out"])


def _run_own(op, st):
    import ternary_weight_linear_token_amd as bw
    if op == "norm":
        return bw.layernorm(st["x"], st["weight"], st["bias"], eps=EPS)
    if op == "norm_quant":
        xq, a, mean, rstd = bw.layernorm_quant(st["x"], st["weight"], st["bias"], eps=EPS,
                                               scale="pow2", return_stats=True)
        return bw.dequant_act(xq, a), mean, rstd
    if op == "norm_back":
        return bw.layernorm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"],
                                     x_scale=st["scale"])
    if op == "swiglu":
        h, ckpt = bw.swiglu(st["g"], st["u"], checkpoint=True)
        return (h,) + tuple(bw.swiglu_backward(st["dh"], *ckpt))
    if op == "grad_input":
        return bw.grad_input_grouped(st["dy"], st["packed"], st["s"])
    return bw.grad_weight(st["dy"], st["xq"], st["a"], out_dtype=st["out"])


# -------------------------------------------------------------------------------- work

def work(case):
    op, m = case["op"], case["m"]
    if op == "norm":
        k = case["k"]
        return dict(bytes=4 * m * k + 8 * k, flops=8 * m * k)
    if op == "norm_quant":  # bf16 in, codes out; the values the codes stand for
        k = case["k"]
        return dict(bytes=4 * m * k + 8 * k + 8 * m, flops=10 * m * k)
    if op == "norm_back":
        k = case["k"]
        return dict(bytes=(5 if case["ckpt"] else 6) * m * k + 12 * m + 12 * k, flops=14 * m * k)
    if op == "swiglu":  # g, u, dh in; h, dg, du out (the codes stay between the two passes)
        return dict(bytes=12 * m * case["n"], flops=24 * m * case["n"])
    if op == "grad_input":
        n, k = case["n1"] + case["n2"] + case["n3"], case["k"]
        return dict(bytes=2 * m * n + n * k // 4 + 4 * n + 2 * m * k, flops=2 * m * n * k)
    n, k = case["n"], case["k"]
    return dict(bytes=2 * m * n + m * k + 4 * m + (4 if case["out"] == "f32" else 2) * n * k,
                flops=2 * m * n * k)


# ------------------------------------------------------------------------ exact values

def exact(case, seed):
    """The outputs in 64 bits, from the definitions.  A value that went through 8 bits of
    computed numbers has none: next to a border of the codes it is a step off or it is not."""
    st = prepare(case, seed)
    d = {key: v.double() for key, v in st.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op in ("norm", "norm_quant"):
        k = case["k"]
        mu = d["x"].sum(1) / k
        var = ((d["x"] - mu.unsqueeze(1)) ** 2).sum(1) / k
        r = (var + EPS) ** -0.5
        y = torch.addcmul(d["bias"], (d["x"] - mu.unsqueeze(1)) * r.unsqueeze(1), d["weight"])
        return y if op == "norm" else (None, mu, r)
    if op == "norm_back":
        k = case["k"]
        x = d["x"] / d["scale"].unsqueeze(1) if st["scale"] is not None else d["x"]
        z = (x - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
        q = d["dy"] * d["weight"]
        c1, c2 = q.sum(1, keepdim=True) / k, (q * z).sum(1, keepdim=True) / k
        dx = (q - (c1 + c2 * z)) * d["rstd"].unsqueeze(1)
        return dx, torch.einsum("mk,mk->k", d["dy"], z), d["dy"].sum(0)
    if op == "swiglu":
        def kept(t):  # the checkpoint: nearest multiple of 1/a, a = 2^floor(log2(127 / amax))
            p = torch.floor(torch.log2(127.0 / t.abs().amax(1, keepdim=True).clamp(min=1e-5)))
            return torch.round(t * 2.0 ** p) / 2.0 ** p
        h = d["g"] * torch.sigmoid(d["g"]) * d["u"]
        g, u = kept(d["g"]), kept(d["u"])
        f = torch.sigmoid(g)
        return h, d["dh"] * u * (f + g * f * torch.sigmoid(-g)), d["dh"] * (g * f)
    if op == "grad_input":
        total = None
        for dy, packed, s in zip(st["dy"], st["packed"], st["s"]):
            digits = packed.to(torch.int64).unsqueeze(2) // torch.tensor([1, 4, 16, 64], device="cuda") % 4
            w = (digits.reshape(packed.shape[0], -1) - 1).double() * s.double().unsqueeze(1)
            part = torch.mm(dy.double(), w)
            total = part if total is None else total + part
        return total
    return torch.mm((d["dy"] / d["a"].unsqueeze(1)).t().contiguous(), d["xq"])
