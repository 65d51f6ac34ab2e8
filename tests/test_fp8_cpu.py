"""Host-side checks of the block-scaled e4m3 entry points (no GPU needed): the
oracle's e4m3 rounding against torch's, and bad arguments refused before any
launch (the pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

from weight_only_bit_gemm_b200 import build

build.build()
from weight_only_bit_gemm_b200 import w4  # noqa: E402

import oracle as O  # noqa: E402

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 1)
WS = 1 << 40


def test_oracle_e4m3_is_torchs():
    t = O.e4m3_values()
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), t)
    mid = (t[:-1] + t[1:]) / 2
    v = np.concatenate([t, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    v = np.concatenate([v, -v])
    ref = torch.from_numpy(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_codes(v), ref)
    assert np.array_equal(O.e4m3_decode(O.e4m3_codes(t)), t)


def test_oracle_scales():
    x = np.zeros((3, 160), np.float32)
    x[0, 5], x[1, 150], x[2, 0] = 448.0, np.inf, -3.5
    q, s = O.fp8_quantize_rows(x)
    assert s[0].tolist() == [1.0, 1.0] and q[0, 5] == 0x7E
    assert s[1, 0] == 1.0 and np.isnan(s[1, 1]) and (q[1, 128:] & 0x7F == 0x7F).all()
    assert s[2, 0] == np.float32(3.5) / np.float32(448) and q[2, 0] == 0xFE


INVALID = {
    "weights null": lambda L: L.fp8_quantize_weights(None, 1, 4, 128, P, P, None),
    "weights K % 16": lambda L: L.fp8_quantize_weights(P, 1, 4, 120, P, P, None),
    "weights B 0": lambda L: L.fp8_quantize_weights(P, 0, 4, 128, P, P, None),
    "weights alignment": lambda L: L.fp8_quantize_weights(ODD, 1, 4, 128, P, P, None),
    "activations null": lambda L: L.fp8_quantize_activations(P, 1, 128, P, None, None),
    "activations M 0": lambda L: L.fp8_quantize_activations(P, 0, 128, P, P, None),
    "activations K": lambda L: L.fp8_quantize_activations(P, 1, 8, P, P, None),
    "activations alignment": lambda L: L.fp8_quantize_activations(P, 1, 128, ODD, P, None),
    "norm null": lambda L: L.fp8_add_rmsnorm(P, P, None, 1e-6, 1, 128, P, P, P, P, None),
    "norm eps": lambda L: L.fp8_add_rmsnorm(P, P, P, -1.0, 1, 128, P, P, P, P, None),
    "norm eps NaN": lambda L: L.fp8_add_rmsnorm(P, P, P, float("nan"), 1, 128, P, P, P, P, None),
    "norm residual alignment": lambda L: L.fp8_add_rmsnorm(P, ODD, P, 1e-6, 1, 128, P, P, P, P, None),
    "gemm null": lambda L: L.fp8_gemm(P, P, P, None, 1, 4, 128, P, P, WS, None),
    "gemm no workspace": lambda L: L.fp8_gemm(P, P, P, P, 1, 4, 128, P, None, WS, None),
    "gemm small workspace": lambda L: L.fp8_gemm(P, P, P, P, 1, 4, 128, P, P, 256, None),
    "gemm K % 16": lambda L: L.fp8_gemm(P, P, P, P, 1, 4, 100, P, P, WS, None),
    "gemm M 0": lambda L: L.fp8_gemm(P, P, P, P, 0, 4, 128, P, P, WS, None),
    "gemm alignment": lambda L: L.fp8_gemm(P, P, ODD, P, 1, 4, 128, P, P, WS, None),
    "gemm Y alignment": lambda L: L.fp8_gemm(P, P, P, P, 1, 4, 128, BYTE, P, WS, None),
    "moe null": lambda L: L.fp8_moe(P, P, P, P, P, None, 1, 8, 2, 128, 128, 1, P, P, P, P, WS, None),
    "moe top > E": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 9, 128, 128, 1, P, P, P, P, WS, None),
    "moe top 0": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 0, 128, 128, 1, P, P, P, P, WS, None),
    "moe H": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 2, 120, 128, 1, P, P, P, P, WS, None),
    "moe I": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 2, 128, 136, 1, P, P, P, P, WS, None),
    "moe small workspace": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 2, 128, 128, 1, P, P, P, P,
                                               4096, None),
    "moe alignment": lambda L: L.fp8_moe(P, ODD, P, P, P, P, 1, 8, 2, 128, 128, 1, P, P, P, P, WS,
                                         None),
}


@pytest.mark.parametrize("name", INVALID)
def test_invalid_arguments_refused(name):
    assert INVALID[name](w4.lib) == w4.W4_ERR_INVALID_ARG


UNSUPPORTED = {
    "norm K": lambda L: L.fp8_add_rmsnorm(P, P, P, 1e-6, 1, 65536 + 16, P, P, P, P, None),
    "moe T": lambda L: L.fp8_moe(P, P, P, P, P, P, 129, 8, 2, 128, 128, 1, P, P, P, P, WS, None),
    "moe E": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 513, 2, 128, 128, 1, P, P, P, P, WS, None),
    "moe top": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 64, 17, 128, 128, 1, P, P, P, P, WS, None),
    "moe H": lambda L: L.fp8_moe(P, P, P, P, P, P, 1, 8, 2, 1 << 20, 128, 1, P, P, P, P, WS, None),
    "gemm M": lambda L: L.fp8_gemm(P, P, P, P, 1 << 25, 4, 128, P, P, WS, None),
    "gemm K": lambda L: L.fp8_gemm(P, P, P, P, 1, 4, 1 << 21, P, P, WS, None),
    "gemm N K": lambda L: L.fp8_gemm(P, P, P, P, 1, 1 << 21, 1 << 19, P, P, WS, None),
    "gemm M N": lambda L: L.fp8_gemm(P, P, P, P, 1 << 20, 1 << 19, 128, P, P, WS, None),
    "weights blocks": lambda L: L.fp8_quantize_weights(P, 1 << 20, 1 << 18, 4096, P, P, None),
}


@pytest.mark.parametrize("name", UNSUPPORTED)
def test_unsupported_shapes_refused(name):
    assert UNSUPPORTED[name](w4.lib) == w4.W4_ERR_UNSUPPORTED


def test_workspace_sizes():
    L = w4.lib
    assert L.fp8_gemm_workspace_bytes(1, 4096, 4096) >= 65536 * 4
    assert L.fp8_gemm_workspace_bytes(0, 4096, 4096) == 0
    assert L.fp8_gemm_workspace_bytes(1, 4096, 100) == 0
    assert L.fp8_gemm_workspace_bytes(1, 4096, 1 << 21) == 0
    assert L.fp8_moe_workspace_bytes(1, 8, 2, 4096, 1024) > 65536 * 4
    assert L.fp8_moe_workspace_bytes(129, 8, 2, 4096, 1024) == 0
    assert L.fp8_moe_workspace_bytes(1, 8, 9, 4096, 1024) == 0


@pytest.mark.parametrize("call", [
    lambda t: w4.fp8_quantize_activations(t),
    lambda t: w4.fp8_quantize_weights(t.float()),
    lambda t: w4.fp8_add_rmsnorm(t, t[0]),
    lambda t: w4.fp8_gemm(t, t, t, t),
    lambda t: w4.fp8_moe(t, t, t, t, t, t, 2),
])
def test_host_tensors_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(16, 16, dtype=torch.bfloat16))


# ------------------------------------- the matrix product's split of the work

def plan(M, N, K, sms=148):
    """The library's split above 128 tokens (148 SMs is its count without a device)."""
    best = None
    for nt, block, read in ((256, 0.56, 3.0), (128, 0.36, 2.0)):
        p = dict(KB=-(-K // 128), workers=sms // 2, runs=0)
        p["rounds"], p["tail"] = divmod(-(-M // 256) * -(-N // nt), p["workers"])
        units = p["tail"] * p["KB"]
        cost = p["KB"] * block + 1.5 if p["tail"] else 0.0
        for runs in range(p["tail"] + 1, p["workers"] + 1):
            if p["tail"] == 0 or runs > units:
                break
            c = units / runs * block + 10 + read * (1 + runs / p["tail"])
            if c < cost:
                cost, p["runs"] = c, runs
        cost += p["rounds"] * (p["KB"] * block + 1.5)
        p["partial"] = 2 * p["runs"] * 2 * 128 * nt
        if best is None or cost < best:
            best, chosen = cost, p
    return chosen


SHAPES = [(M, N, K) for M in (129, 256, 511, 2048, 8192)
          for N, K in ((1, 16), (4096, 4096), (4096, 11008), (12288, 4096), (13824, 5120),
                       (28672, 8192), (129, 28672), (20000, 512))]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_split_covers_every_block_once(M, N, K):
    p = plan(M, N, K)
    L = w4.lib
    assert L.fp8_gemm_workspace_bytes(128, N, K) == 65536 * 4
    assert L.fp8_gemm_workspace_bytes(M, N, K) == 65536 * 4 + -(-p["partial"] * 4 // 256) * 256
    if not p["runs"]:
        return
    KB, U, G = p["KB"], p["tail"] * p["KB"], p["runs"]
    assert p["tail"] <= G <= p["workers"]
    start = [U * c // G for c in range(G + 1)]
    pieces = {}                                   # tail tile -> [(run, k0, k1, slot)]
    for c in range(G):
        assert start[c] < start[c + 1]
        u = start[c]
        while u < start[c + 1]:
            t, k0 = divmod(u, KB)
            k1 = min(KB, k0 + start[c + 1] - u)
            pieces.setdefault(t, []).append((c, k0, k1, 2 * c + (start[c] < t * KB)))
            u += k1 - k0
    slots = [s for v in pieces.values() for _, k0, k1, s in v if (k0, k1) != (0, KB)]
    assert len(set(slots)) == len(slots) and max(slots, default=0) < 2 * G
    run_of = lambda v: ((v + 1) * G - 1) // U  # noqa: E731
    for t in range(p["tail"]):
        v = pieces[t]
        assert v[0][1] == 0 and v[-1][2] == KB
        assert all(a[2] == b[1] for a, b in zip(v, v[1:]))
        # the reducer's walk: runs first..last, the first one's slot by where
        # it starts, the others' first slots
        first, last = run_of(t * KB), run_of(t * KB + KB - 1)
        assert [a[0] for a in v] == list(range(first, last + 1))
        assert [a[3] for a in v[1:]] == [2 * c for c in range(first + 1, last + 1)]
