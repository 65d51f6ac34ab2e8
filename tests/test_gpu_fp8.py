"""GPU parity of the block-scaled e4m3 path, through the public calls, against
the oracle on the same seeded inputs.

Codes and scales of the quantizers: bit-exact.  The norm: scales within the
fp32 error of its mean, codes within half an e4m3 step.  The products within
the bounds that the oracle derives (fp32 sums, half a bf16 step)."""
import numpy as np
import pytest
import torch

import oracle as O
from weight_only_bit_gemm_b200 import synthetic as S

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def w4():
    from weight_only_bit_gemm_b200 import build
    build.build()
    from weight_only_bit_gemm_b200 import w4 as mod
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def x_dev(bits):
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def q_dev(codes):
    return dev(codes).view(F8)


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def f32(bits):
    return S.bf16_bits_to_f32(bits)


def ok(w4):
    assert w4.device_status() == w4.W4_OK


def same_scales(a, b):
    assert np.array_equal(a.view(np.uint32) if not np.isnan(b).any() else np.nan_to_num(a, nan=-1.0),
                          b.view(np.uint32) if not np.isnan(b).any() else np.nan_to_num(b, nan=-1.0))


def draw_x(M, K, seed):
    return S.draw_x(M, K, seed=seed, tag=80, N=1, outlier_frac=0.01, outlier_scale=50.0)


def draw_q(N, K, seed):
    return O.fp8_quantize_blocks(S.draw_w(N, K, 0.02, seed=seed, tag=81))


# ------------------------------------------------------------- quantizers

@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (300, 400), (129, 1040), (7, 4096)])
def test_weights_bit_exact(w4, N, K):
    W = S.draw_w(N, K, 0.02, seed=N, tag=82)
    W[N // 2, :] = 0.0
    W[: min(N, 128), : min(K, 128)] *= np.float32(1e-39)   # a subnormal block
    q, s = w4.fp8_quantize_weights(dev(W))
    ok(w4)
    qr, sr = O.fp8_quantize_blocks(W)
    assert np.array_equal(codes(q), qr)
    same_scales(s.cpu().numpy(), sr)


def test_weights_batch_and_zero_block(w4):
    W = np.stack([S.draw_w(130, 272, 0.02, seed=i, tag=83) for i in range(6)]).reshape(3, 2, 130, 272)
    W[1, 1] = 0.0
    q, s = w4.fp8_quantize_weights(dev(W))
    ok(w4)
    assert s.shape == (3, 2, 2, 3) and bool((s[1, 1] == 1).all())
    for i in range(3):
        for j in range(2):
            qr, sr = O.fp8_quantize_blocks(W[i, j])
            assert np.array_equal(codes(q[i, j]), qr)
            same_scales(s[i, j].cpu().numpy(), sr)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 144), (17, 1008), (128, 11008), (5, 28672)])
def test_activations_bit_exact(w4, M, K):
    xb = draw_x(M, K, M)
    xb[0, : min(K, 128)] = 0
    q, s = w4.fp8_quantize_activations(x_dev(xb))
    ok(w4)
    qr, sr = O.fp8_quantize_rows(f32(xb))
    assert np.array_equal(codes(q), qr)
    same_scales(s.cpu().numpy(), sr)


def test_every_bf16_value_quantizes_as_the_oracle(w4):
    # all finite bf16 values, 128 neighbours to a block, and shuffled
    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80][: 509 * 128]
    for xb in (bits, np.random.default_rng(3).permutation(bits)):
        xb = xb.reshape(-1, 128 * 1)
        q, s = w4.fp8_quantize_activations(x_dev(xb))
        ok(w4)
        qr, sr = O.fp8_quantize_rows(f32(xb))
        assert np.array_equal(codes(q), qr)
        same_scales(s.cpu().numpy(), sr)


@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
def test_non_finite_values_reach_the_output(w4, bad):
    xb = draw_x(3, 272, 9)
    xb[1, 140] = bad
    q, s = w4.fp8_quantize_activations(x_dev(xb))
    qr, sr = O.fp8_quantize_rows(f32(xb))
    same_scales(s.cpu().numpy(), sr)
    assert np.array_equal(codes(q)[[0, 2]], qr[[0, 2]])
    assert ((codes(q)[1, 128:256] & 0x7F) == 0x7F).all()
    qw, sw = draw_q(200, 272, 1)
    y = f64(w4.fp8_gemm(q, s, q_dev(qw), dev(sw)))
    ok(w4)
    assert np.isnan(y[1]).all() and np.isfinite(y[[0, 2]]).all()


# ------------------------------------------------------------------- norm

@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (5, 4112), (3, 8192), (33, 1040), (2, 16384),
                                 (3, 28672), (1, 65536)])
@pytest.mark.parametrize("res", [False, True])
def test_norm(w4, M, K, res):
    xb, rb = draw_x(M, K, M), draw_x(M, K, M + 50)
    wb = S.to_bf16_bits(1 + 0.1 * np.random.default_rng(K).standard_normal(K, dtype=np.float32))
    eps = 1e-5
    q, s, ro, y = w4.fp8_add_rmsnorm(x_dev(xb), x_dev(wb), x_dev(rb) if res else None, eps,
                                     want_y=True)
    ok(w4)
    r_ref, y_ref = O.fp8_rmsnorm_ref(f32(xb), f32(rb) if res else None, f32(wb), eps)
    # relative error of y: the rounding of r (2^-24, and 2^-24 |x| + |res| is
    # not more where they do not cancel: bounded absolutely below); the mean
    # of squares over chains of at most 64 + 37 additions, halved by the root;
    # rsqrtf (2 steps) and two products
    rel = (64 + 37) / 2 * 2.0 ** -24 + 8 * 2.0 ** -24
    y_err = rel * np.abs(y_ref) + 2.0 ** -24 * np.abs(y_ref)
    assert (np.abs(f64(y) - y_ref) <= 2.0 ** -8 * np.abs(y_ref) + y_err).all()
    if res:
        # the sum of two bf16 values rounds once in fp32, then to bf16
        assert (np.abs(f64(ro) - r_ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(r_ref)).all()
        assert torch.equal(ro, (x_dev(xb).float() + x_dev(rb).float()).to(torch.bfloat16))
    else:
        assert ro is None
    amax = np.stack([np.abs(y_ref[:, k:k + 128]).max(1) for k in range(0, K, 128)], 1)
    sv = f64(s)
    s_rel = rel + 2 * 2.0 ** -24
    assert (np.abs(sv - amax / 448) <= s_rel * amax / 448).all()
    full = np.repeat(sv, 128, axis=1)[:, :K]
    got = O.e4m3_decode(codes(q)) * full
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 of the scale below
    half = np.maximum(2.0 ** -4 * np.abs(y_ref), 2.0 ** -10 * full)
    assert (np.abs(got - y_ref) <= half * (1 + 2.0 ** -10) + y_err + 2 * s_rel * np.abs(y_ref)).all()


def test_norm_in_place_and_zero_row(w4):
    xb, rb = draw_x(4, 400, 1), draw_x(4, 400, 2)
    xb[2], rb[2] = 0, 0
    w = torch.ones(400, dtype=torch.bfloat16, device="cuda")
    res = x_dev(rb)
    q0, s0, r0, _ = w4.fp8_add_rmsnorm(x_dev(xb), w, res)
    q1, s1, r1, _ = w4.fp8_add_rmsnorm(x_dev(xb), w, res, residual_out=res)
    ok(w4)
    assert r1 is res and torch.equal(r0, r1) and torch.equal(s0, s1)
    assert np.array_equal(codes(q0), codes(q1))
    assert (codes(q0)[2] == 0).all() and bool((s0[2] == 1).all())


# ---------------------------------------------------------------- product

GEMM = [
    # (M, N, K)
    (1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 127, 144), (7, 1000, 1040), (8, 136, 4096),
    (16, 512, 11008), (17, 300, 2064), (31, 257, 2048), (32, 4104, 1024), (33, 4096, 2048),
    (64, 260, 8192), (65, 129, 256), (100, 640, 2048), (127, 384, 1024), (128, 1024, 4096),
    (129, 512, 2048), (200, 1000, 656), (256, 2304, 1024), (300, 20000, 512), (511, 768, 5120),
    (1000, 1000, 1008), (1025, 2050, 272),
    # more tokens: cut tails with odd rows and columns, 128- and 256-row tiles
    (257, 1001, 14336), (400, 6001, 4096), (700, 259, 9008), (300, 9473, 1040),
]


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm(w4, M, N, K):
    qx, sx = O.fp8_quantize_rows(f32(draw_x(M, K, M)))
    qw, sw = draw_q(N, K, M)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.fp8_gemm(q_dev(qx), dev(sx), q_dev(qw), dev(sw), out=y)
    ok(w4)
    ref, absum = O.fp8_gemm_ref(qx, sx, qw, sw)
    err = np.abs(f64(y) - ref)
    tol = O.fp8_gemm_tolerance(ref, absum, K)
    assert (err <= tol).all(), f"worst error / tolerance = {(err / tol).max()}"


@pytest.mark.parametrize("M,N,K", [(3, 48, 128), (40, 300, 1024), (64, 256, 4096), (256, 130, 512),
                                   (300, 1100, 2048)])
def test_gemm_exact_on_exact_inputs(w4, M, N, K):
    # codes that are whole numbers up to 14 and scales that are powers of two:
    # every sum is exact in fp32, so the result is the rounded exact one
    rng = np.random.default_rng(M)
    x, w = rng.integers(-14, 15, (M, K)).astype(np.float64), rng.integers(-14, 15, (N, K)).astype(np.float64)
    qx, qw = O.e4m3_codes(x), O.e4m3_codes(w)
    sx = 2.0 ** rng.integers(-2, 3, (M, -(-K // 128))).astype(np.float32)
    sw = 2.0 ** rng.integers(-2, 3, (-(-N // 128), -(-K // 128))).astype(np.float32)
    y = w4.fp8_gemm(q_dev(qx), dev(sx), q_dev(qw), dev(sw))
    ok(w4)
    ref, _ = O.fp8_gemm_ref(qx, sx, qw, sw)
    exact = S.to_bf16_bits(ref.astype(np.float32))
    assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), exact)


def test_gemm_repeats_bit_for_bit_and_leaves_the_workspace_clean(w4):
    # calls of different shapes in turn on one workspace, INT4 among them
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    W = S.draw_w(512, 4096, 0.02, seed=1, tag=84)
    q4, s4, z4 = (dev(a) for a in O.quantize_rtn(W, 128))
    Wq, sc, zr = w4.quantize_rtn(dev(W), 128)
    Wp = w4.prepack(Wq, sc, zr, 128)
    X = x_dev(draw_x(4, 4096, 1))
    y4 = w4.w4a16_gemm(X, Wp, 512, 4096, 128, workspace=ws)
    first = {}
    for turn in range(3):
        for M, N, K in [(1, 4096, 4096), (40, 300, 8192), (300, 2000, 1024), (16, 130, 272)]:
            qx, sx = w4.fp8_quantize_activations(x_dev(draw_x(M, K, M)))
            qw, sw = (q_dev(a) if a.dtype == np.uint8 else dev(a) for a in draw_q(N, K, M))
            y = w4.fp8_gemm(qx, sx, qw, sw, workspace=ws)
            if turn == 0:
                first[M] = y
            assert torch.equal(first[M], y)
        assert torch.equal(w4.w4a16_gemm(X, Wp, 512, 4096, 128, workspace=ws), y4)
        assert not bool(ws[: 65536 * 4].any())
    ok(w4)


# ---------------------------------------------------------------- experts

def draw_moe(T, E, H, I, seed):
    rng = np.random.default_rng([seed, T, E, H, I])
    xb = draw_x(T, H, seed)
    rb = S.to_bf16_bits(rng.standard_normal((E, H), dtype=np.float32) / np.float32(np.sqrt(H)))
    q13, s13, q2, s2 = [], [], [], []
    for e in range(E):
        g = [draw_q(I, H, seed + 2 * e + i) for i in range(2)]
        q13.append(np.stack([a[0] for a in g]))
        s13.append(np.stack([a[1] for a in g]))
        d = draw_q(H, I, seed + 100 + e)
        q2.append(d[0])
        s2.append(d[1])
    return xb, rb, np.stack(q13), np.stack(s13), np.stack(q2), np.stack(s2)


def run_moe(w4, data, top, renorm, **kw):
    xb, rb, q13, s13, q2, s2 = data
    return w4.fp8_moe(x_dev(xb), x_dev(rb), q_dev(q13), dev(s13), q_dev(q2), dev(s2), top,
                      renormalize=renorm, **kw)


MOE = [
    # (T, E, top, H, I, renormalize)
    (1, 1, 1, 16, 16, True), (1, 8, 2, 256, 128, True), (1, 16, 8, 1024, 256, True),
    (2, 4, 1, 400, 144, False), (3, 5, 5, 272, 400, True), (8, 8, 2, 512, 512, False),
    (17, 8, 3, 1040, 272, True), (33, 16, 4, 256, 640, True), (64, 4, 2, 768, 1040, False),
    (128, 8, 2, 512, 384, True), (128, 3, 3, 144, 2064, True), (5, 130, 16, 256, 128, True),
    (1, 512, 4, 128, 32, False),
]


@pytest.mark.parametrize("T,E,top,H,I,renorm", MOE)
def test_moe(w4, T, E, top, H, I, renorm):
    data = draw_moe(T, E, H, I, T)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    y, ids, wts = run_moe(w4, data, top, renorm, out=out)
    ok(w4)
    xb, rb, q13, s13, q2, s2 = data
    ref, bound, ids_ref, w_ref = O.moe_ref(f32(xb), f32(rb), q13, s13, q2, s2, top, renorm)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    # the logits' fp32 sums and the exponential: 2^-16 relative is far above both
    assert np.allclose(f64(wts), w_ref, rtol=2.0 ** -16, atol=0)
    err = np.abs(f64(y) - ref)
    assert (err <= bound).all(), f"worst error / bound = {(err / bound).max()}"


def test_moe_exact_on_exact_inputs(w4):
    # gates of at least 32 (1 + exp(-g) is 1 in fp32, so h = g u exactly),
    # whole-number weights, every scale a power of two: the expert outputs are
    # exact, and with one choice of renormalized weight 1 so is the result
    T, E, H, I = 9, 6, 272, 144
    rng = np.random.default_rng(5)
    x = np.zeros((T, H), np.float32)
    x[:, 0] = 448.0                                    # scale 1 in the first block
    x[:, 128] = 448.0
    x[:, 256] = 448.0
    pick = rng.integers(0, E, T)
    router = np.zeros((E, H), np.float32)
    x[np.arange(T), 1 + pick] = 32.0
    router[np.arange(E), 1 + np.arange(E)] = 1.0
    x[:, 20:27] = rng.integers(1, 9, (T, 7))
    w13 = np.zeros((E, 2, I, H))
    w13[:, 0, :, 20:27] = rng.integers(0, 2, (E, I, 7))
    w13[:, 0, :, 1:1 + E] = 1.0                        # +32 on every gate
    w13[:, 1, :, 20] = 1.0
    w2 = rng.integers(-3, 4, (E, H, I)).astype(np.float64)
    one = np.ones
    data = (S.to_bf16_bits(x), S.to_bf16_bits(router), O.e4m3_codes(w13),
            one((E, 2, 2, 3), np.float32), O.e4m3_codes(w2), one((E, 3, 2), np.float32))
    y, ids, wts = run_moe(w4, data, 1, True)
    ok(w4)
    assert np.array_equal(ids.cpu().numpy()[:, 0], pick) and bool((wts == 1).all())
    xq, sx = O.fp8_quantize_rows(x)
    assert (sx == 1).all()
    xv = O.fp8_row_values(xq, sx)
    ref = np.empty((T, H), np.float64)
    for t in range(T):
        g, u = w13[pick[t], 0] @ xv[t], w13[pick[t], 1] @ xv[t]
        assert g.min() >= 32
        hq, sh = O.fp8_quantize_rows((g * u).astype(np.float32)[None])
        d = 0.0
        for j in range(2):
            blk = np.s_[j * 128:(j + 1) * 128]
            part = w2[pick[t]][:, blk] @ O.e4m3_decode(hq[0, blk])
            d = (np.float32(part) * sh[0, j] + np.float32(d)).astype(np.float32)
        ref[t] = d
    got = f64(y)
    # the two blocks' scaled sums: one rounding each in fp32, then half a bf16 step
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(ref).max()).all()


def test_moe_ties_and_nan_router(w4):
    T, E, H, I = 4, 9, 128, 32
    xb, rb, *rest = draw_moe(T, E, H, I, 3)
    rb[:] = rb[0]                                      # equal logits: the lowest indices
    y, ids, wts = run_moe(w4, (xb, rb, *rest), 3, True)
    ok(w4)
    assert (ids.cpu().numpy() == np.array([0, 1, 2])).all()
    assert np.allclose(f64(wts), 1 / 3, rtol=2.0 ** -20)
    xb[1, 7] = 0x7FC0                                  # a NaN token: its row alone is lost
    y2, ids2, _ = run_moe(w4, (xb, rb, *rest), 3, True)
    ok(w4)
    assert (ids2.cpu().numpy()[1] == np.array([0, 1, 2])).all()
    keep = [0, 2, 3]
    assert torch.equal(y[keep], y2[keep]) and bool(y2[1].isnan().all())


def test_moe_one_expert_takes_every_token(w4):
    # all tokens on one expert (the largest group), the others untouched
    T, E, H, I = 128, 4, 256, 144
    xb, rb, *rest = draw_moe(T, E, H, I, 6)
    x = f32(xb)
    x[:, 0] = 64.0
    router = np.zeros((E, H), np.float32)
    router[2, 0] = 1.0
    data = (S.to_bf16_bits(x), S.to_bf16_bits(router), *rest)
    y, ids, _ = run_moe(w4, data, 1, True)
    ok(w4)
    assert (ids.cpu().numpy() == 2).all()
    ref, bound, _, _ = O.moe_ref(x, router, *rest, 1, True)
    assert (np.abs(f64(y) - ref) <= bound).all()


def test_moe_repeats_bit_for_bit(w4):
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(4):
        for T, E, top, H, I in [(1, 8, 2, 512, 256), (40, 8, 4, 400, 272), (3, 64, 6, 256, 128)]:
            if (T, E) not in first:
                first[T, E] = draw_moe(T, E, H, I, 8), []
            data, seen = first[T, E]
            seen.append(run_moe(w4, data, top, True, workspace=ws)[0])
            assert torch.equal(seen[0], seen[-1])
        assert not bool(ws[: 65536 * 4].any())
    ok(w4)


# ------------------------------------------------------------ as used together

def layer(w4, x, res, weight, router, w13, s13, w2, s2, qp, sp):
    """norm -> projection -> norm -> experts, the path of one decoder layer."""
    q, s, res, _ = w4.fp8_add_rmsnorm(x, weight, res)
    a = w4.fp8_gemm(q, s, qp, sp)
    _, _, res, y = w4.fp8_add_rmsnorm(a, weight, res, want_y=True)
    out, ids, wts = w4.fp8_moe(y, router, w13, s13, w2, s2, 2)
    return out, res, ids


def layer_inputs(T, H, I, E, seed):
    xb, rb, q13, s13, q2, s2 = draw_moe(T, E, H, I, seed)
    qp, sp = draw_q(H, H, seed + 7)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    return (x_dev(xb), x_dev(draw_x(T, H, seed + 1)), w, x_dev(rb), q_dev(q13), dev(s13), q_dev(q2),
            dev(s2), q_dev(qp), dev(sp))


@pytest.mark.parametrize("T", [1, 24])
def test_layer_matches_the_oracle_step_by_step(w4, T):
    H, I, E = 512, 272, 8
    args = layer_inputs(T, H, I, E, 11)
    x, res, weight, router, w13, s13, w2, s2, qp, sp = args
    q, s, res1, _ = w4.fp8_add_rmsnorm(x, weight, res)
    a = w4.fp8_gemm(q, s, qp, sp)
    ref, absum = O.fp8_gemm_ref(codes(q), s.cpu().numpy(), codes(qp), sp.cpu().numpy())
    assert (np.abs(f64(a) - ref) <= O.fp8_gemm_tolerance(ref, absum, H)).all()
    _, _, res2, y = w4.fp8_add_rmsnorm(a, weight, res1, want_y=True)
    out, ids, _ = w4.fp8_moe(y, router, w13, s13, w2, s2, 2)
    ok(w4)
    mref, bound, ids_ref, _ = O.moe_ref(f64(y).astype(np.float32), f64(router).astype(np.float32),
                                        codes(w13), s13.cpu().numpy(), codes(w2), s2.cpu().numpy(),
                                        2, True)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert (np.abs(f64(out) - mref) <= bound).all()
    got = layer(w4, *args)
    assert torch.equal(got[0], out) and torch.equal(got[1], res2)


def test_layer_captured_in_graphs(w4):
    # two graphs with the default workspaces, replayed at once on two streams,
    # with eager calls in between: each gives the eager result
    sets = [layer_inputs(T, 512, 272, 8, 20 + T) for T in (1, 24)]
    eager = [layer(w4, *a) for a in sets]
    graphs, outs = [], []
    for a in sets:
        layer(w4, *a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(w4, *a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for g, st, o in zip(graphs, streams, outs):
            with torch.cuda.stream(st):
                o[0].zero_()
                g.replay()
        again = layer(w4, *sets[1])
        assert torch.equal(again[0], eager[1][0])
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o[0], e[0]) and torch.equal(o[1], e[1])
    ok(w4)


def test_large_product_captured_and_eager(w4):
    # a product with partial sums: two graphs of it replayed at once beside
    # eager calls, and the eager default workspace stays clean
    M, N, K = 300, 600, 16384
    ins = []
    for seed in (1, 2):
        qx, sx = w4.fp8_quantize_activations(x_dev(draw_x(M, K, seed)))
        qw, sw = w4.fp8_quantize_weights(dev(S.draw_w(N, K, 0.02, seed=seed, tag=88)))
        ins.append((qx, sx, qw, sw))
    assert w4.lib.fp8_gemm_workspace_bytes(M, N, K) > 65536 * 4
    eager = [w4.fp8_gemm(*a) for a in ins]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w4.fp8_gemm(*a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        again = [w4.fp8_gemm(*a) for a in ins]
        torch.cuda.synchronize()
        for o, e, v in zip(outs, eager, again):
            assert torch.equal(o, e) and torch.equal(v, e)
    ok(w4)


def test_two_streams_at_once(w4):
    sets = [layer_inputs(T, 512, 272, 8, 30 + T) for T in (2, 33)]
    eager = [layer(w4, *a)[0] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(layer(w4, *sets[i])[0])
    torch.cuda.synchronize()
    ok(w4)
    for g, e in zip(got, eager):
        assert all(torch.equal(v, e) for v in g)


# ---------------------------------------------------------------- refusals

def test_wrong_tensors_refused(w4):
    q = torch.zeros(4, 256, device="cuda").to(F8)
    s = torch.ones(4, 2, device="cuda")
    qw, sw = torch.zeros(130, 256, device="cuda").to(F8), torch.ones(2, 2, device="cuda")
    assert w4.fp8_gemm(q, s, qw, sw).shape == (4, 130)
    for args in [(q, s.t().contiguous(), qw, sw), (q, s, qw, sw[:1]), (q, s, qw[:, :128], sw),
                 (q.view(torch.uint8), s, qw, sw), (q, s.half(), qw, sw),
                 (q, s, torch.zeros(256, 256, device="cuda").to(F8).t()[:130], sw)]:
        with pytest.raises(ValueError):
            w4.fp8_gemm(*args)
    with pytest.raises(ValueError):
        w4.fp8_gemm(q, s, qw, sw, out=torch.zeros(4, 131, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(4, 200, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(w4.W4Error):
        w4.fp8_quantize_activations(x)
    with pytest.raises(ValueError):
        w4.fp8_add_rmsnorm(x, x[0, :100])
    with pytest.raises(ValueError):
        w4.fp8_add_rmsnorm(x, x[0], residual_out=x)


def test_moe_refusals(w4):
    data = draw_moe(1, 4, 128, 32, 1)
    with pytest.raises(w4.W4Error) as e:
        run_moe(w4, data, 5, True)
    assert e.value.status == w4.W4_ERR_INVALID_ARG
    big = draw_moe(129, 1, 128, 32, 1)
    with pytest.raises(w4.W4Error) as e:
        run_moe(w4, big, 1, True)
    assert e.value.status == w4.W4_ERR_UNSUPPORTED
    ok(w4)


# ------------------------------------------------- offsets beyond 32 bits

def big_bf16(M, K, seed):
    """[M, K] on the GPU: one drawn block of rows repeated, so that any row's
    expectation is cheap."""
    base = draw_x(97, K, seed)
    x = x_dev(base)
    return x.repeat(-(-M // 97), 1)[:M].contiguous(), base


def test_more_than_2_31_activations(w4):
    M, K = 66001, 32800                                  # 2.16e9 values
    x, base = big_bf16(M, K, 91)
    q, s = w4.fp8_quantize_activations(x)
    ok(w4)
    rows = [0, 40000, M - 1]
    qr, sr = O.fp8_quantize_rows(f32(base[[r % 97 for r in rows]]))
    assert np.array_equal(codes(q[rows]), qr)
    same_scales(s[rows].cpu().numpy(), sr)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    qn, sn, ro, _ = w4.fp8_add_rmsnorm(x, w, x)
    ok(w4)
    # the same rows in a small call: the same bits
    q1, s1, r1, _ = w4.fp8_add_rmsnorm(x[rows].contiguous(), w, x[rows].contiguous())
    assert np.array_equal(codes(qn[rows]), codes(q1)) and torch.equal(sn[rows], s1)
    assert torch.equal(ro[rows], r1)


def test_more_than_2_31_weights(w4):
    B, N, K = 3, 22001, 32784                            # 2.16e9 values
    W = torch.empty(B, N, K, device="cuda").normal_(std=0.02)
    q, s = w4.fp8_quantize_weights(W)
    ok(w4)
    part = W[2, 21888:, 32640:].cpu().numpy()            # the last blocks of the last matrix
    qr, sr = O.fp8_quantize_blocks(part)
    assert np.array_equal(codes(q[2, 21888:, 32640:].contiguous()), qr)
    same_scales(s[2, -1:, -2:].cpu().numpy(), sr)


def test_more_than_2_31_outputs(w4):
    M, N, K = 66001, 32808, 144                          # 2.17e9 outputs
    x, base = big_bf16(M, K, 92)
    qx, sx = w4.fp8_quantize_activations(x)
    qw, sw = draw_q(N, K, 93)
    y = w4.fp8_gemm(qx, sx, q_dev(qw), dev(sw))
    ok(w4)
    rows = [0, 40000, M - 1]
    ref, absum = O.fp8_gemm_ref(codes(qx[rows]), sx[rows].cpu().numpy(), qw, sw)
    assert (np.abs(f64(y[rows]) - ref) <= O.fp8_gemm_tolerance(ref, absum, K)).all()


def test_back_to_back_calls_on_reused_memory(w4):
    # every call starts while the one before it runs, and the allocator hands the
    # same memory to the next turn's codes and scales: no turn may see another's
    sets = [layer_inputs(T, 512, 272, 8, 40 + T) for T in (3, 3 + 32, 3 + 64)]
    alone = []
    for a in sets:
        alone.append(layer(w4, *a)[:2])
        torch.cuda.synchronize()
    big = []
    for seed in (1, 2):
        x = x_dev(draw_x(160, 1040, seed))
        qw, sw = w4.fp8_quantize_weights(dev(S.draw_w(700, 1040, 0.02, seed=seed, tag=89)))
        torch.cuda.synchronize()
        y = w4.fp8_gemm(*w4.fp8_quantize_activations(x), qw, sw)
        torch.cuda.synchronize()
        big.append((x, qw, sw, y))
    got = []
    for turn in range(60):
        got.append([layer(w4, *a)[:2] for a in sets])
        for x, qw, sw, y in big:
            got[-1].append((w4.fp8_gemm(*w4.fp8_quantize_activations(x), qw, sw),))
    torch.cuda.synchronize()
    ok(w4)
    for turn in got:
        for g, e in zip(turn[:3], alone):
            assert torch.equal(g[0], e[0]) and torch.equal(g[1], e[1])
        for g, b in zip(turn[3:], big):
            assert torch.equal(g[0], b[3])
