"""The block-scaled e4m3 entry points in the bounds-checked build: no kernel
index outside its buffer on ragged cases, and results bit-identical to the
normal build's."""
import numpy as np
import pytest
import torch

from weight_only_bit_gemm_b200 import synthetic as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    from weight_only_bit_gemm_b200 import build
    build.build()
    build.build(checked=True)
    from weight_only_bit_gemm_b200 import w4
    return w4, w4.checked_library()


def both(libs, fn):
    w4, chk = libs
    a = fn()
    assert w4.device_status() == w4.W4_OK
    with w4.using(chk):
        b = fn()
        assert w4.device_status() == w4.W4_OK
    for x, y in zip(a, b):
        if x is not None:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    return a


def x_dev(M, K, seed):
    bits = S.draw_x(M, K, seed=seed, tag=85, N=1, outlier_frac=0.01, outlier_scale=50.0)
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(1, 77, 336), (17, 300, 1040), (40, 200, 4096), (100, 257, 2064),
                                   (128, 640, 1024), (129, 300, 2064), (300, 5000, 656),
                                   (520, 2304, 16384)])
def test_checked_linear_path(libs, M, N, K):
    w4, _ = libs
    W = torch.from_numpy(S.draw_w(N, K, 0.02, seed=M, tag=86)).cuda()
    X, R = x_dev(M, K, M), x_dev(M, K, M + 1)
    weight = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    qw, sw = both(libs, lambda: w4.fp8_quantize_weights(W))
    both(libs, lambda: w4.fp8_quantize_activations(X))
    q, s, _, _ = both(libs, lambda: w4.fp8_add_rmsnorm(X, weight, R, want_y=True))
    both(libs, lambda: (w4.fp8_gemm(q, s, qw, sw),))


@pytest.mark.parametrize("T,E,top,H,I", [(1, 8, 2, 400, 272), (5, 40, 6, 256, 144),
                                         (33, 6, 2, 528, 400), (70, 9, 3, 256, 128),
                                         (128, 4, 4, 144, 1040)])
def test_checked_experts(libs, T, E, top, H, I):
    w4, _ = libs
    rng = np.random.default_rng([T, E, 87])
    dev = lambda *shape: torch.from_numpy(  # noqa: E731
        rng.standard_normal(shape, dtype=np.float32) * np.float32(0.02)).cuda()
    w13, s13 = w4.fp8_quantize_weights(dev(E, 2, I, H))
    w2, s2 = w4.fp8_quantize_weights(dev(E, H, I))
    router = dev(E, H).to(torch.bfloat16)
    X = x_dev(T, H, T)
    both(libs, lambda: w4.fp8_moe(X, router, w13, s13, w2, s2, top))
