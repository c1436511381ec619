"""The launch plans of the decoder block's products, from sizes and types alone
(host code): the ones that were measured faster with the weights in memory."""
import ctypes

import pytest

from lora_adapter_pool_amd import _lib

LINEAR, GATED = 0, 1
BF16 = _lib.LORA_BF16


class Plan(ctypes.Structure):
    _fields_ = [("shape", ctypes.c_int32), ("whole", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("ws_bytes", ctypes.c_int64), ("us", ctypes.c_float)]


def plan(form, T, K, N, dtype=BF16, out=BF16, size=2):
    f = getattr(_lib.lib(), "_ZN4lora9gemm_planEiiNS_4FormElll")
    f.restype = Plan
    f.argtypes = [ctypes.c_int32] * 3 + [ctypes.c_int64] * 3
    return f(dtype, out, form, T, N, K * size)


# tile shapes: 1 is 64 x 64, 2 is 128 x 128, 3 is 256 x 256
@pytest.mark.parametrize("form,T,K,N,shape,parts", [
    (LINEAR, 64, 4096, 4096, 1, 4),      # 13.6 us, in 8 parts 15.8
    (LINEAR, 192, 4096, 6144, 2, 2),     # 30.4 us, 64 x 64 in one part 35.5
    (LINEAR, 256, 4096, 6144, 2, 2),     # 31.8 us, 35.5
    (GATED, 64, 8192, 1024, 1, 8),       # 16.3 us, in 16 parts 21.8
    (GATED, 256, 4096, 4096, 2, 2),      # 34.4 us, 64 x 64 in one part 38.9
    (GATED, 300, 4096, 6144, 3, 2)])     # 57.2 us, 69.5
def test_decode_batches_take_the_plan_that_is_faster_from_memory(form, T, K, N, shape, parts):
    p = plan(form, T, K, N)
    assert (p.shape, p.splits) == (shape, parts)
