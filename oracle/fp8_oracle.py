"""Oracle of the block-scaled 8-bit floating-point (e4m3) path, TEST
INFRASTRUCTURE ONLY: codes and scales, the residual RMS norm, the matrix
product and the mixture-of-experts layer, in numpy.

R21 e4m3: bias 7, subnormals below 2^-6 in steps of 2^-9, largest value 448
    (the all-ones magnitude is NaN, no infinity); rounding to nearest, ties to
    the even code;
R22 scale = fp32(max|v| / 448) per 128 channels of a token (activations) or
    128 x 128 block (weights), 1 where that is 0; the code is that of
    fp32(v / scale); a block holding a non-finite value has the scale NaN;
R23 the product and everything after the codes is in fp64 here.
"""
from __future__ import annotations

import numpy as np

__all__ = [
    "e4m3_values", "e4m3_codes", "e4m3_decode", "fp8_quantize_rows", "fp8_quantize_blocks",
    "fp8_row_values", "fp8_block_values", "fp8_rmsnorm_ref", "fp8_gemm_ref", "fp8_gemm_tolerance",
    "moe_route_ref", "moe_ref",
]

B = 128


def e4m3_values() -> np.ndarray:
    """The 127 non-negative values, by code."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """uint8 codes of fp64 values: nearest, ties to the even code, at most 448."""
    t = e4m3_values()
    mid = (t[:-1] + t[1:]) / 2
    a = np.abs(v)
    below = np.searchsorted(mid, a, side="left")    # midpoints < a
    upto = np.searchsorted(mid, a, side="right")    # midpoints <= a
    code = np.where((below != upto) & (below % 2 == 1), upto, below).astype(np.uint8)
    code = np.where(np.isnan(v), np.uint8(0x7F), code)
    return code | (np.signbit(v).astype(np.uint8) << 7)


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    """fp64 values of uint8 codes."""
    t = np.append(e4m3_values(), np.nan)
    v = t[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def _scale(a: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        s = (a.astype(np.float32) / np.float32(448)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    return np.where(np.isfinite(a), s, np.float32(np.nan))


def fp8_quantize_rows(x: np.ndarray):
    """fp32 x [M, K] -> (codes uint8 [M, K], scales fp32 [M, KB])."""
    q, s = np.empty(x.shape, np.uint8), []
    for k in range(0, x.shape[1], B):
        b = x[:, k:k + B].astype(np.float32)
        sc = _scale(np.abs(b).max(axis=1))
        with np.errstate(invalid="ignore"):
            q[:, k:k + B] = e4m3_codes((b / sc[:, None]).astype(np.float32).astype(np.float64))
        s.append(sc)
    return q, np.stack(s, axis=1)


def fp8_quantize_blocks(w: np.ndarray):
    """fp32 w [N, K] -> (codes uint8 [N, K], scales fp32 [NB, KB])."""
    N, K = w.shape
    q = np.empty(w.shape, np.uint8)
    s = np.empty((-(-N // B), -(-K // B)), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * B:(i + 1) * B, j * B:(j + 1) * B]
            s[i, j] = _scale(np.abs(w[at]).max())
            with np.errstate(invalid="ignore"):
                q[at] = e4m3_codes((w[at] / s[i, j]).astype(np.float32).astype(np.float64))
    return q, s


def fp8_row_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return e4m3_decode(q) * np.repeat(s.astype(np.float64), B, axis=1)[:, :q.shape[1]]


def fp8_block_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    full = np.repeat(np.repeat(s.astype(np.float64), B, axis=0), B, axis=1)
    return e4m3_decode(q) * full[:q.shape[0], :q.shape[1]]


def fp8_rmsnorm_ref(x, residual, weight, eps):
    """fp64 (r, y) of fp32 x [M, K], residual (or None) and weight [K]."""
    r = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    y = r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * weight.astype(np.float64)
    return r, y


def fp8_gemm_ref(qx, sx, qw, sw):
    """fp64 (y, sum of the terms' magnitudes)."""
    x, w = fp8_row_values(qx, sx), fp8_block_values(qw, sw)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def fp8_gemm_tolerance(y, absum, K):
    """Half a bf16 step of the result (2^-8 relative), and for the fp32 sums
    over K terms: at most one fp32 step (2^-23, truncation allowed) of the
    terms' magnitude per addition inside a block of 128, one rounding (2^-24)
    per block for its scaled addition and two for the scale product and the
    scaling.  With few bits left between bf16 neighbours the bf16 step is
    taken of the largest value the fp32 result can have."""
    blocks = -(-K // B)
    acc = absum * (min(K, B) * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24)
    return 2.0 ** -8 * (np.abs(y) + acc) + acc + 2.0 ** -133


def moe_route_ref(logits: np.ndarray, top: int, renormalize: bool):
    """(ids, weights) of fp64 logits: largest first, ties to the lowest index."""
    key = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top]
    chosen = np.take_along_axis(logits, ids, axis=1)
    e = np.exp(chosen - chosen[:, :1])
    total = e.sum(1) if renormalize else np.exp(logits - chosen[:, :1]).sum(1)
    return ids, e / total[:, None]


def _flip(v: np.ndarray, s: np.ndarray, rel: float) -> np.ndarray:
    """How far the stored value of v may move when v has this relative error:
    0 where every value within it has the same code, else the distance of the
    two codes (v and s in fp64, s per element)."""
    lo, hi = np.abs(v) * (1 - rel), np.abs(v) * (1 + rel)
    return (e4m3_decode(e4m3_codes(hi / s)) - e4m3_decode(e4m3_codes(lo / s))) * s


def moe_ref(x, router, q13, s13, q2, s2, top, renormalize):
    """fp64 (y, bound on |y - y_ref|, ids, weights) of fp32 x [T, H], router
    [E, H] and the experts' codes and scales.  The bound has half a bf16 step;
    the fp32 sums of both products as in fp8_gemm_tolerance; for h, whose
    relative error follows from its gate and up sums, the codes that this
    error can move; and 2^-16 for the routing weights."""
    T, H = x.shape
    I = q2.shape[2]
    ids, wts = moe_route_ref(x.astype(np.float64) @ router.astype(np.float64).T, top, renormalize)
    xq, sx = fp8_quantize_rows(x)
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        tok, slot = np.nonzero(ids == e)
        g, ga = fp8_gemm_ref(xq[tok], sx[tok], q13[e, 0], s13[e, 0])
        u, ua = fp8_gemm_ref(xq[tok], sx[tok], q13[e, 1], s13[e, 1])
        unit = min(H, B) * 2.0 ** -23 + (-(-H // B) + 2) * 2.0 ** -24
        with np.errstate(over="ignore"):
            h = g / (1 + np.exp(-g)) * u
        # |d silu / dg| <= 1.1, |silu(g)| <= |g|; the exponential and the
        # division add a few fp32 roundings relative to h
        dh = 1.1 * ga * unit * np.abs(u) + np.abs(h / np.where(u == 0, 1, u)) * ua * unit \
            + 2.0 ** -20 * np.abs(h)
        hq, sh = fp8_quantize_rows(h.astype(np.float32))
        full = np.repeat(sh.astype(np.float64), B, axis=1)[:, :I]
        rel = np.where(h == 0, 0, dh / np.where(h == 0, 1, np.abs(h)))
        top_rel = np.zeros_like(sh, dtype=np.float64)     # the scale moves with its block's largest
        for j in range(sh.shape[1]):
            top_rel[:, j] = (dh[:, j * B:(j + 1) * B]).max(axis=1) / \
                np.maximum(np.abs(h[:, j * B:(j + 1) * B]).max(axis=1), 1e-300)
        scale_rel = np.repeat(top_rel, B, axis=1)[:, :I] + 2.0 ** -22
        move = _flip(h, full, np.minimum(rel + scale_rel, 1.0)) + \
            np.abs(fp8_row_values(hq, sh)) * scale_rel
        d, da = fp8_gemm_ref(hq, sh, q2[e], s2[e])
        w2 = np.abs(fp8_block_values(q2[e], s2[e]))
        acc = da * (min(I, B) * 2.0 ** -23 + (-(-I // B) + 2) * 2.0 ** -24)
        w = wts[tok, slot][:, None]
        y[tok] += w * d
        bound[tok] += w * (acc + move @ w2.T + 2.0 ** -16 * np.abs(d))
    return y, bound + 2.0 ** -8 * (np.abs(y) + bound) + 2.0 ** -133, ids, wts
