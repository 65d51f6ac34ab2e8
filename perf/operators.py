"""Cases of the block-scaled 8-bit floating-point (e4m3) linear path: quantization of
weights and activations, the residual RMS norm with an 8-bit output, the matrix product
and the mixture-of-experts layer for a few tokens.

Format: e4m3 codes (largest value 448) with one fp32 scale per 128 channels of a row
(activations) or per 128 x 128 block (weights); blocks start at channel and row 0 and the
last one may be shorter.  The plain forms below are the definitions, in fp32 with one
rounding at the end; ``exact`` is the same in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
EPS = 1e-6
HALVES = 2  # gate and up


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token entering a 7B layer
        dict(name="norm 1x4096", op="norm", M=1, K=4096, residual=True, keep=False),
        # a long prompt of odd length before an expert layer, whose router reads bf16
        dict(name="norm 8191x8192", op="norm", M=8191, K=8192, residual=True, keep=True),
        # input of a down projection while decoding 16 sequences
        dict(name="quant x 16x11008", op="quant_x", M=16, K=11008),
        # input of a down projection of a prompt, width of a 13B layer
        dict(name="quant x 4099x13824", op="quant_x", M=4099, K=13824),
        # one attention projection of a 7B layer
        dict(name="quant w 4096x4096", op="quant_w", B=1, N=4096, K=4096),
        # the gate and up projections of 8 experts, rows not a multiple of the block
        dict(name="quant w 16x2000x4096", op="quant_w", B=16, N=2000, K=4096),
        # fused q/k/v projection, one token
        dict(name="gemm 1x12288x4096", op="gemm", M=1, N=12288, K=4096),
        # down projection with the tokens of a small batch
        dict(name="gemm 33x4096x11008", op="gemm", M=33, N=4096, K=11008),
        # 13B up projection, a short prompt of odd length
        dict(name="gemm 511x13824x5120", op="gemm", M=511, N=13824, K=5120),
        # 70B up projection, a long prompt
        dict(name="gemm 2048x28672x8192", op="gemm", M=2048, N=28672, K=8192),
        # many small experts, one decoded token
        dict(name="moe 1 of 64x1024x4096", op="moe", T=1, E=64, top=8, H=4096, I=1024,
             renorm=True),
        # few large experts, a batch of 37 sequences
        dict(name="moe 37 of 8x14336x4096", op="moe", T=37, E=8, top=2, H=4096, I=14336,
             renorm=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    top = 2048 * 28672 * 8192
    while True:
        op = rng.choice(["norm", "quant_x", "quant_w", "gemm", "gemm", "moe", "moe"])
        if op == "norm":
            c = dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 256, 16384, 16),
                     residual=rng.random() < 0.7, keep=rng.random() < 0.5)
            if c["M"] * c["K"] <= 8191 * 8192:
                return c
        elif op == "quant_x":
            c = dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 256, 28672, 16))
            if c["M"] * c["K"] <= 4099 * 13824:
                return c
        elif op == "quant_w":
            c = dict(op=op, B=_log(rng, 1, 16), N=_log(rng, 100, 14336), K=_log(rng, 256, 14336, 16))
            if c["B"] * c["N"] * c["K"] <= 16 * 2000 * 4096:
                return c
        elif op == "gemm":
            c = dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 128, 28672), K=_log(rng, 256, 28672, 16))
            if c["M"] * c["N"] * c["K"] <= top and c["N"] * c["K"] <= 28672 * 8192:
                return c
        else:
            e = _log(rng, 4, 128)
            c = dict(op=op, T=_log(rng, 1, 128), E=e, top=rng.randint(1, min(8, e)),
                     H=_log(rng, 256, 8192, 16), I=_log(rng, 128, 14336, 16),
                     renorm=rng.random() < 0.5)
            if c["E"] * c["H"] * c["I"] <= 8 * 14336 * 4096:
                return c


def _active(c):
    """Experts that T tokens with `top` choices each are expected to reach."""
    return c["E"] * (1 - (1 - c["top"] / c["E"]) ** c["T"])


def work(c):
    op = c["op"]
    if op == "norm":
        mk = c["M"] * c["K"]
        moved = mk * (2 + 1 + (4 if c["residual"] else 0) + (2 if c["keep"] else 0))
        return dict(bytes=moved + 2 * c["K"] + 4 * c["M"] * _blocks(c["K"]), flops=6 * mk)
    if op == "quant_x":
        return dict(bytes=3 * c["M"] * c["K"] + 4 * c["M"] * _blocks(c["K"]),
                    flops=2 * c["M"] * c["K"])
    if op == "quant_w":
        n = c["B"] * c["N"] * c["K"]
        return dict(bytes=5 * n + 4 * c["B"] * _blocks(c["N"]) * _blocks(c["K"]), flops=2 * n)
    if op == "gemm":
        m, n, k = c["M"], c["N"], c["K"]
        return dict(bytes=m * k + n * k + 2 * m * n + 4 * (m + _blocks(n)) * _blocks(k),
                    flops=2 * m * n * k)
    t, h, i = c["T"], c["H"], c["I"]
    return dict(bytes=_active(c) * 3 * h * i + 2 * c["E"] * h + 4 * t * h,
                flops=2 * t * (c["E"] * h + c["top"] * 3 * h * i))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", dtype=dtype, generator=g)


def _activations(g, m, k):
    """Standard normal with 0.1 % of the channels 50 times larger."""
    x = _randn(g, m, k)
    loud = torch.rand(k, device="cuda", generator=g) < 0.001
    return (x * torch.where(loud, 50.0, 1.0)).to(torch.bfloat16)


def _stored_weights(g, *shape):
    """Codes and scales as a quantized checkpoint holds them: normal weights of deviation
    about 0.02, each block's largest near the end of the code range."""
    codes = _randn(g, *shape, dtype=torch.bfloat16).mul_(104.0).clamp_(-E4M3_MAX, E4M3_MAX)
    blocks = shape[:-2] + (_blocks(shape[-2]), _blocks(shape[-1]))
    scales = 0.02 / 104.0 * (0.8 + 0.45 * torch.rand(*blocks, device="cuda", generator=g))
    return codes.to(torch.float8_e4m3fn), scales


def prepare(c, seed):
    g = _gen(seed)
    op = c["op"]
    s = dict(op=op)
    if op == "norm":
        s["x"] = _activations(g, c["M"], c["K"])
        s["res"] = (_activations(g, c["M"], c["K"]) if c["residual"] else None)
        s["weight"] = (1 + 0.1 * _randn(g, c["K"])).to(torch.bfloat16)
        s["keep"] = c["keep"]
    elif op == "quant_x":
        s["x"] = _activations(g, c["M"], c["K"])
    elif op == "quant_w":
        shape = (c["N"], c["K"]) if c["B"] == 1 else (c["B"], c["N"], c["K"])
        s["w"] = _randn(g, *shape).mul_(0.02)
    elif op == "gemm":
        s["qx"], s["sx"] = _quantize_rows(_activations(g, c["M"], c["K"]).float())
        s["qw"], s["sw"] = _stored_weights(g, c["N"], c["K"])
    else:
        s["x"] = _activations(g, c["T"], c["H"])
        s["router"] = (_randn(g, c["E"], c["H"]) * c["H"] ** -0.5).to(torch.bfloat16)
        s["w13"], s["s13"] = _stored_weights(g, c["E"], HALVES, c["I"], c["H"])
        s["w2"], s["s2"] = _stored_weights(g, c["E"], c["H"], c["I"])
        s["top"], s["renorm"] = c["top"], c["renorm"]
    return s


# ------------------------------------------------------------------ plain forms

def _pad(x, dims):
    """x with zeros up to whole blocks in its last `dims` dimensions."""
    k = x.shape[-1]
    pad = [0, _blocks(k) * BLOCK - k]
    if dims == 2:
        n = x.shape[-2]
        pad += [0, _blocks(n) * BLOCK - n]
    return torch.nn.functional.pad(x, pad) if any(pad) else x


def _scales(largest):
    """largest / 448, correctly rounded (a division by a Python number would multiply by
    its rounded reciprocal), 1 for a block of zeros."""
    s = largest / torch.full_like(largest, E4M3_MAX)
    return torch.where(s == 0, 1.0, s)


def _quantize_rows(x):
    """Codes and scales of rows, one scale per 128 channels."""
    m, k = x.shape
    b = _pad(x, 1).view(m, _blocks(k), BLOCK)
    s = _scales(b.abs().amax(-1))
    q = (b / s[..., None]).view(m, -1)[:, :k]
    return q.to(torch.float8_e4m3fn), s


def _quantize_blocks(w):
    """Codes and scales of matrices, one scale per 128 x 128 block."""
    n, k = w.shape[-2:]
    b = _pad(w, 2).unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    s = _scales(b.abs().amax((-3, -1)))
    q = (b / s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def _values_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _values_blocks(q, s):
    n, k = q.shape[-2:]
    rows = s.repeat_interleave(BLOCK, -1)[..., :k]
    return q.float().mul_(rows.repeat_interleave(BLOCK, -2)[..., :n, :])


def _plain_norm(x, res, weight):
    r = x.float() if res is None else x.float() + res.float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * weight.float()
    return r, y


def _plain_route(x, router, top, renorm):
    logits = x.double() @ router.double().T
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids = order.indices[:, :top]
    chosen = order.values[:, :top]
    rest = chosen if renorm else logits
    w = torch.exp(chosen - order.values[:, :1]) / torch.exp(rest - order.values[:, :1]).sum(-1, True)
    return ids.to(torch.int32), w.float()


def _plain_moe(s):
    x, ids_w = s["x"], _plain_route(s["x"], s["router"], s["top"], s["renorm"])
    ids, weights = ids_w
    t, top = ids.shape
    experts = s["w13"].shape[0]
    rows = _values_rows(*_quantize_rows(x.float()))
    pair = ids.long().flatten()
    if t * top < experts:  # each choice's own expert gathered
        w13 = _values_blocks(s["w13"][pair], s["s13"][pair]).flatten(1, 2)
        gu = torch.bmm(w13, rows.repeat_interleave(top, 0)[:, :, None])[..., 0]
    else:                  # every expert on every token, the chosen ones kept
        w13 = _values_blocks(s["w13"], s["s13"]).flatten(1, 2)
        gu = torch.matmul(rows, w13.transpose(1, 2))
        gu = gu[pair, torch.arange(t, device=x.device).repeat_interleave(top)]
    del w13
    gate, up = gu.chunk(2, -1)
    h = _values_rows(*_quantize_rows(gate / (1 + torch.exp(-gate)) * up))
    if t * top < experts:
        w2 = _values_blocks(s["w2"][pair], s["s2"][pair])
        d = torch.bmm(w2, h[:, :, None])[..., 0]
    else:
        w2 = _values_blocks(s["w2"], s["s2"])
        spread = torch.zeros(experts, t, h.shape[1], device=x.device)
        spread[pair, torch.arange(t, device=x.device).repeat_interleave(top)] = h
        d = torch.bmm(spread, w2.transpose(1, 2))
        d = d[pair, torch.arange(t, device=x.device).repeat_interleave(top)]
    y = (d.view(t, top, -1) * weights[..., None]).sum(1)
    return y.to(torch.bfloat16), ids, weights


def _plain(s):
    op = s["op"]
    if op == "norm":
        r, y = _plain_norm(s["x"], s["res"], s["weight"])
        q, sc = _quantize_rows(y)
        return (q, sc, None if s["res"] is None else r.to(torch.bfloat16),
                y.to(torch.bfloat16) if s["keep"] else None)
    if op == "quant_x":
        return _quantize_rows(s["x"].float())
    if op == "quant_w":
        return _quantize_blocks(s["w"])
    if op == "gemm":
        x, w = _values_rows(s["qx"], s["sx"]), _values_blocks(s["qw"], s["sw"])
        return (x @ w.T).to(torch.bfloat16)
    return _plain_moe(s)


def _own(s):
    from weight_only_bit_gemm_b200 import w4

    op = s["op"]
    if op == "norm":
        return w4.fp8_add_rmsnorm(s["x"], s["weight"], residual=s["res"], eps=EPS,
                                  want_y=s["keep"])
    if op == "quant_x":
        return w4.fp8_quantize_activations(s["x"])
    if op == "quant_w":
        return w4.fp8_quantize_weights(s["w"])
    if op == "gemm":
        return w4.fp8_gemm(s["qx"], s["sx"], s["qw"], s["sw"])
    return w4.fp8_moe(s["x"], s["router"], s["w13"], s["s13"], s["w2"], s["s2"], s["top"],
                      renormalize=s["renorm"])


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------ 64-bit definitions

def _exact_rows(x):
    """Codes and scales of rows from the definition, block by block, in 64 bits; the scale
    takes its fp32 value, the one that is stored, before the codes are chosen with it."""
    q, s = torch.empty_like(x), []
    for k0 in range(0, x.shape[1], BLOCK):
        b = x[:, k0:k0 + BLOCK]
        a = (b.abs().amax(1, keepdim=True) / E4M3_MAX).float().double()
        a[a == 0] = 1
        q[:, k0:k0 + BLOCK] = (b / a).float().to(torch.float8_e4m3fn).double()
        s.append(a)
    return q, torch.cat(s, 1)


def _exact_values(q, s):
    v = q.double()
    for j in range(s.shape[-1]):
        for i in range(s.shape[-2]):
            v[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= s[i, j].double()
    return v


def _exact_row_values(q, s):
    v = q.double()
    for j in range(s.shape[-1]):
        v[:, j * BLOCK:(j + 1) * BLOCK] *= s[:, j:j + 1].double()
    return v


def _exact_moe(c, s):
    x = s["x"].double()
    p = x @ s["router"].double().T
    y = torch.zeros_like(x)
    rows = _exact_row_values(*_exact_rows(x))
    left, ids, weights = p.clone(), [], []
    for _ in range(c["top"]):
        best = left.amax(1, keepdim=True)
        first = (left == best).double().argmax(1, keepdim=True)
        ids.append(first)
        weights.append(best)
        left.scatter_(1, first, -math.inf)
    ids, weights = torch.cat(ids, 1), torch.cat(weights, 1)
    total = torch.logsumexp(weights if c["renorm"] else p, 1, keepdim=True)
    weights = torch.exp(weights - total)
    for e in torch.unique(ids).tolist():
        tok, slot = (ids == e).nonzero(as_tuple=True)
        gate = rows[tok] @ _exact_values(s["w13"][e, 0], s["s13"][e, 0]).T
        up = rows[tok] @ _exact_values(s["w13"][e, 1], s["s13"][e, 1]).T
        h = _exact_row_values(*_exact_rows(gate * torch.sigmoid(gate) * up))
        y[tok] += weights[tok, slot, None] * (h @ _exact_values(s["w2"][e], s["s2"][e]).T)
    return y, ids, weights


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        r = s["x"].double()
        if s["res"] is not None:
            r = r + s["res"].double()
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / c["K"] + EPS) * s["weight"].double()
        q, sc = _exact_rows(y)
        return q, sc, None if s["res"] is None else r, y if s["keep"] else None
    if op == "quant_x":
        return _exact_rows(s["x"].double())
    if op == "quant_w":
        w = s["w"].double().view(-1, c["N"], c["K"])
        nb, kb = _blocks(c["N"]), _blocks(c["K"])
        sc = torch.empty(w.shape[0], nb, kb, dtype=torch.float64, device="cuda")
        q = torch.empty_like(w)
        for i in range(nb):
            for j in range(kb):
                b = w[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                a = (b.abs().amax((1, 2)) / E4M3_MAX).float().double()
                a = torch.where(a == 0, torch.ones_like(a), a)
                sc[:, i, j] = a
                q[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = (
                    (b / a[:, None, None]).float().to(torch.float8_e4m3fn).double())
        return (q[0], sc[0]) if c["B"] == 1 else (q, sc)
    if op == "gemm":
        return _exact_row_values(s["qx"], s["sx"]) @ _exact_values(s["qw"], s["sw"]).T
    return _exact_moe(c, s)
