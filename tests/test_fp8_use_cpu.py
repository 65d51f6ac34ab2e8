"""The Python calls of the block-scaled e4m3 path around the library (no GPU
needed: the library's entry points are stood in for, tensors are on the host)."""
import gc
import types
import weakref

import numpy as np
import pytest
import torch

from weight_only_bit_gemm_b200 import build

build.build()
from weight_only_bit_gemm_b200 import w4  # noqa: E402

import oracle as O  # noqa: E402

F8 = torch.float8_e4m3fn
STREAM = 7


@pytest.fixture
def host(monkeypatch):
    """w4 with host tensors taken for a device's (index -1), a fake library and
    no workspaces yet."""
    monkeypatch.setattr(w4, "_fp8_first", lambda t, dtype, dim, name: -1)
    monkeypatch.setattr(w4, "_raw_stream", lambda dev: STREAM)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(w4, "_FP8_WS", {})
    fake = types.SimpleNamespace(fp8_gemm_workspace_bytes=lambda *a: 1 << 21,
                                 fp8_moe_workspace_bytes=lambda *a: 1 << 21)
    monkeypatch.setattr(w4, "lib", fake)
    return fake


def gemm():
    return w4.fp8_gemm(torch.zeros(4, 128).to(F8), torch.ones(4, 1), torch.zeros(8, 128).to(F8),
                       torch.ones(1, 1))


def moe():
    return w4.fp8_moe(torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(2, 128, dtype=torch.bfloat16),
                      torch.zeros(2, 2, 128, 128).to(F8), torch.ones(2, 2, 1, 1),
                      torch.zeros(2, 128, 128).to(F8), torch.ones(2, 1, 1), 1)


@pytest.mark.parametrize("call,entry", [(gemm, "fp8_gemm"), (moe, "fp8_moe")])
def test_workspace_outlives_its_replacement_by_another_thread(host, call, entry):
    # while a call is on its way into the library, another thread's call needs a
    # larger workspace of the same stream: the first one's must not be freed
    # before its kernels are launched
    seen = []

    def launch(*args):
        (key, buf), = w4._FP8_WS.items()
        seen.append(weakref.ref(buf))
        w4._FP8_WS[key] = torch.zeros(8, dtype=torch.uint8)
        del buf
        gc.collect()
        assert seen[0]() is not None, "the workspace was freed before the launch"
        return w4.W4_OK

    setattr(host, entry, launch)
    call()
    assert len(seen) == 1
    gc.collect()
    assert seen[0]() is None            # nothing keeps it afterwards


@pytest.mark.parametrize("status", ["W4_ERR_TIMEOUT", "W4_ERR_BOUNDS", "W4_OK", "W4_ERR_DEVICE_INPUT"])
def test_default_workspaces_given_up_after_a_call_that_did_not_run_through(host, monkeypatch, status):
    # their counters may be nonzero, and no caller can reach them
    monkeypatch.setattr(w4, "_stream", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    host.w4_device_status = lambda stream: getattr(w4, status)
    w4._FP8_WS.update({(0, 5): torch.ones(8), (0, 6): torch.ones(8), (1, 5): torch.ones(8)})
    assert w4.device_status() == getattr(w4, status)
    lost = status in ("W4_ERR_TIMEOUT", "W4_ERR_BOUNDS")
    assert sorted(w4._FP8_WS) == ([(1, 5)] if lost else [(0, 5), (0, 6), (1, 5)])


@pytest.mark.parametrize("units", [224, 225, 300, 600, 671, 672, 1000])
def test_oracle_saturates_where_the_scale_is_subnormal(units):
    # the largest value in units of 2^-149: its scale is rounded to a whole
    # number of them, and a quotient past 448 has the code of 448
    w = np.zeros((2, 16), np.float32)
    w[0, :3] = np.array([units, -units, units // 2]) * 2.0 ** -149
    q, s = O.fp8_quantize_blocks(w)
    scale = int(np.rint(units / 448))
    assert s[0, 0] == (np.float32(scale * 2.0 ** -149) if scale else np.float32(1))
    top = O.e4m3_codes(np.array([min(units / scale, 448.0) if scale else 0.0]))[0]
    assert q[0, 0] == top and q[0, 1] == (top | 0x80)
    if units in (600, 671):
        assert top == 0x7E
