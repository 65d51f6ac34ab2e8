"""Ways of calling the block-scaled e4m3 path that a program may take: host
threads that share a stream, tensors rewritten on the stream between calls,
sizes and values at the ends of their ranges.  Results are compared with the
same calls made alone, or with the oracle."""
import threading

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_fp8 import codes, dev, draw_moe, draw_x, ok, q_dev, same_scales, x_dev
from weight_only_bit_gemm_b200 import synthetic as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from weight_only_bit_gemm_b200 import build
    build.build()
    from weight_only_bit_gemm_b200 import w4 as mod
    return mod


# ------------------------------------------------------------ host threads

def in_threads(calls, turns):
    """The results of each call, made `turns` times by a thread of its own, all
    on the current stream."""
    start, stream = threading.Barrier(len(calls)), torch.cuda.current_stream()
    got = [[] for _ in calls]

    def work(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(turns):
                got[i].append(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == turns for g in got)
    return got


def moe_tensors(data):
    return tuple(conv(a) for conv, a in zip((x_dev, x_dev, q_dev, dev, q_dev, dev), data))


def test_first_calls_of_a_host_thread(w4):
    # a thread whose first call into CUDA is this library's: the tensor maps
    # are made by driver calls, which need the device's context on the thread
    qx, sx = w4.fp8_quantize_activations(x_dev(draw_x(200, 400, 1)))
    qw, sw = w4.fp8_quantize_weights(dev(S.draw_w(300, 400, 0.02, seed=1, tag=90)))
    moe = moe_tensors(draw_moe(2, 4, 256, 128, 62))
    Wp = w4.prepack(*w4.quantize_rtn(dev(S.draw_w(256, 512, 0.02, seed=2, tag=90)), 128), 128)
    X = x_dev(draw_x(300, 512, 2))
    q1, s1 = qx[:3].contiguous(), sx[:3].contiguous()
    y1, y200, y4 = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
                    for M, N in ((3, 300), (200, 300), (300, 256)))
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    calls = [lambda: w4.fp8_gemm(q1, s1, qw, sw, out=y1, workspace=ws).clone(),
             lambda: w4.fp8_gemm(qx, sx, qw, sw, out=y200, workspace=ws).clone(),
             lambda: w4.fp8_moe(*moe, 2, workspace=ws)[0],
             lambda: w4.w4a16_gemm(X, Wp, 256, 512, 128, out=y4, workspace=ws).clone()]
    for call in calls:
        alone = call()
        torch.cuda.synchronize()
        (got,), = in_threads([call], 1)
        assert torch.equal(got, alone)
    ok(w4)


@pytest.mark.parametrize("own_workspace", [False, True])
def test_two_host_threads_on_one_stream(w4, own_workspace):
    # one stream and one workspace for both threads: the two kernels of an
    # expert layer stay together, whatever the other thread's calls, of another
    # shape, leave in the workspace between them
    shapes = [(3, 8, 2, 512, 272), (40, 16, 4, 400, 144)]
    kw = dict(workspace=torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")) if own_workspace else {}
    calls = []
    for T, E, top, H, I in shapes:
        a = moe_tensors(draw_moe(T, E, H, I, 60 + T))
        calls.append(lambda a=a, top=top: w4.fp8_moe(*a, top, **kw))
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    got = in_threads(calls, 300)
    ok(w4)
    for g, e in zip(got, alone):
        for r in g:
            assert all(torch.equal(x, y) for x, y in zip(r, e))


# ------------------------------------------------- after a wait that gave up

@pytest.mark.parametrize("wait", ["selftest_wait_timeout", "fp8_selftest_wait_timeout"])
def test_calls_after_a_timeout(w4, wait):
    # a wait has run out (the short one of a self-test): whatever the default
    # workspaces' counters hold then, the next calls do not start from it
    args = moe_tensors(draw_moe(5, 6, 400, 144, 63))
    alone = w4.fp8_moe(*args, 2)
    ok(w4)
    here = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream)
    w4._FP8_WS[here].fill_(1)
    getattr(w4, wait)()
    assert w4.device_status() == w4.W4_ERR_TIMEOUT
    assert here not in w4._FP8_WS       # (else the next line must not run)
    again = w4.fp8_moe(*args, 2)
    ok(w4)
    assert all(torch.equal(a, b) for a, b in zip(again, alone))


# ------------------------------------------------------- the longest rows

K_MAX = 2 ** 31 - 16                    # the largest K an int can name


def tiled(dtype, M, K, seed):
    """[M, K] of drawn values that repeat every 65536."""
    x = torch.empty(M, K, dtype=dtype, device="cuda")
    base = x_dev(draw_x(1, 65536, seed)).to(dtype).view(-1)
    flat = x.view(-1)
    n = flat.numel() // 65536
    flat[: n * 65536].view(n, 65536).copy_(base)
    flat[n * 65536:].copy_(base[: flat.numel() - n * 65536])
    return x


LAST = K_MAX // 128 * 128               # where a row's last, shorter block starts


@pytest.mark.parametrize("at", [0, 2 ** 30, LAST - 128, LAST])
def test_activation_rows_of_the_largest_length(w4, at, rows):
    x, q, s = rows
    qr, sr = O.fp8_quantize_rows(x[:, at:at + 128].float().cpu().numpy())
    assert np.array_equal(codes(q[:, at:at + 128].contiguous()), qr)
    same_scales(s[:, at // 128:at // 128 + 1].cpu().numpy(), sr)


@pytest.fixture(scope="module")
def rows(w4):
    x = tiled(torch.bfloat16, 2, K_MAX, 64)
    q, s = w4.fp8_quantize_activations(x)
    ok(w4)
    assert s.shape == (2, 2 ** 24)
    return x, q, s


@pytest.mark.parametrize("at", [0, 2 ** 30, LAST - 128, LAST])
def test_weight_rows_of_the_largest_length(w4, at, weight_rows):
    W, q, s = weight_rows
    qr, sr = O.fp8_quantize_blocks(W[:, at:at + 128].cpu().numpy())
    assert np.array_equal(codes(q[:, at:at + 128].contiguous()), qr)
    same_scales(s[:, at // 128:at // 128 + 1].cpu().numpy(), sr)


@pytest.fixture(scope="module")
def weight_rows(w4):
    W = tiled(torch.float32, 2, K_MAX, 65)
    q, s = w4.fp8_quantize_weights(W)
    ok(w4)
    assert s.shape == (1, 2 ** 24)
    return W, q, s


# --------------------------------------- operands written on the stream before

def ahead_of_the_gpu():
    """A few milliseconds of work on the stream, so that the calls made next are
    queued and follow each other on the GPU without a gap."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(8):
        a @ a


def between(w4, how, small):
    """What runs between the writer of an operand and the product."""
    if how == "norm":                    # starts while the kernel ahead of it runs
        w4.fp8_add_rmsnorm(*small)
    elif how == "torch":
        small[0].clone()


@pytest.mark.parametrize("how", ["nothing", "norm", "torch"])
@pytest.mark.parametrize("writer", ["quantizer", "copy"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_weights_written_on_the_stream(w4, M, writer, how):
    # the product's weights are the codes of a kernel that may still run when
    # the product's blocks are already on the SMs; in memory that held the turn
    # before's codes
    N, K = 16, 2048
    X = [x_dev(draw_x(N, K, 70 + i)) for i in range(2)]
    Q = [w4.fp8_quantize_activations(x)[0] for x in X]
    qx, sx = w4.fp8_quantize_activations(x_dev(draw_x(M, K, 72)))
    sw = torch.full((1, K // 128), 2.0 ** -6, device="cuda")
    small = (x_dev(draw_x(2, 256, 73)), torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    alone = []
    for q in Q:
        torch.cuda.synchronize()
        alone.append(w4.fp8_gemm(qx, sx, q, sw))
    torch.cuda.synchronize()
    assert not torch.equal(*alone)
    held, scales, got = torch.empty_like(Q[0]), torch.empty(N, K // 128, device="cuda"), []
    ahead_of_the_gpu()
    for turn in range(100):
        i = turn & 1
        if writer == "quantizer":
            w4._check(w4.lib.fp8_quantize_activations(X[i].data_ptr(), N, K, held.data_ptr(),
                                                      scales.data_ptr(), w4._raw_stream(0)), "quantize")
        else:
            held.copy_(Q[i])
        between(w4, how, small)
        got.append(w4.fp8_gemm(qx, sx, held, sw))
    torch.cuda.synchronize()
    ok(w4)
    bad = [t for t, y in enumerate(got) if not torch.equal(y, alone[t & 1])]
    assert not bad, f"{len(bad)} of {len(got)} turns saw other weights"


@pytest.mark.parametrize("M", [3, 200])
def test_weight_scales_written_on_the_stream(w4, M):
    # an SM may still hold the lines of the product before, which read the same
    # memory's older scales while this product's blocks were already resident
    K, NB = 512, 296                    # two blocks on every SM
    N = NB * 128
    X = [x_dev(draw_x(NB, K, 80 + i)) for i in range(2)]
    qx, sx = w4.fp8_quantize_activations(x_dev(draw_x(M, K, 82)))
    qw, _ = w4.fp8_quantize_weights(dev(S.draw_w(N, K, 0.02, seed=4, tag=91)))
    S2 = [w4.fp8_quantize_activations(x)[1] for x in X]
    alone = [w4.fp8_gemm(qx, sx, qw, s) for s in S2]
    torch.cuda.synchronize()
    assert not torch.equal(*alone)
    q, s, got = torch.empty(NB, K, dtype=torch.uint8, device="cuda"), torch.empty_like(S2[0]), []
    ahead_of_the_gpu()
    for turn in range(400):
        w4._check(w4.lib.fp8_quantize_activations(X[turn & 1].data_ptr(), NB, K, q.data_ptr(), s.data_ptr(),
                                                  w4._raw_stream(0)), "quantize")
        got.append(w4.fp8_gemm(qx, sx, qw, s))
    torch.cuda.synchronize()
    ok(w4)
    assert [t for t, y in enumerate(got) if not torch.equal(y, alone[t & 1])] == []


@pytest.mark.parametrize("call", ["norm", "norm of many rows", "moe"])
def test_vectors_written_on_the_stream(w4, call):
    # the norm's weight and the router, written by a product on the stream
    K, E = 4096, 8
    qx, sx = zip(*(w4.fp8_quantize_activations(x_dev(draw_x(E, K, 84 + i))) for i in range(2)))
    qw, sw = w4.fp8_quantize_weights(dev(S.draw_w(K, K, 0.02, seed=3, tag=91)))
    x = x_dev(draw_x(700 if "many" in call else 2, K, 86))
    moe = moe_tensors(draw_moe(2, E, K, 128, 87))
    vec = [w4.fp8_gemm(a, b, qw, sw) for a, b in zip(qx, sx)]

    def use(v):
        if call == "moe":
            return w4.fp8_moe(x, v, *moe[2:], 2)[2]
        return w4.fp8_add_rmsnorm(x, v[0], want_y=True)[3]

    alone = [use(v) for v in vec]
    torch.cuda.synchronize()
    assert not torch.equal(*alone)
    held, got = torch.empty_like(vec[0]), []
    ahead_of_the_gpu()
    for turn in range(200):
        i = turn & 1
        w4.fp8_gemm(qx[i], sx[i], qw, sw, out=held)
        got.append(use(held))
    torch.cuda.synchronize()
    ok(w4)
    assert [t for t, y in enumerate(got) if not torch.equal(y, alone[t & 1])] == []


# ------------------------------------------------------- the smallest blocks

def test_weight_blocks_with_subnormal_scales(w4):
    # one block per largest value, in units of 2^-149
    units = [1, 223, 224, 225, 300, 448, 600, 671, 672, 1000, 5000, 10 ** 6, 2 ** 23, 2 ** 25]
    rng = np.random.default_rng(11)
    W = np.concatenate([np.rint(rng.uniform(-u, u, (16, 128))) * 2.0 ** -149 for u in units], axis=1)
    W = W.astype(np.float32)
    for i, u in enumerate(units):
        W[i % 16, 128 * i + 5] = -u * 2.0 ** -149
        W[(i + 3) % 16, 128 * i + 77] = u * 2.0 ** -149
    q, s = w4.fp8_quantize_weights(dev(W))
    ok(w4)
    qr, sr = O.fp8_quantize_blocks(W)
    assert np.array_equal(codes(q), qr)
    same_scales(s.cpu().numpy(), sr)
