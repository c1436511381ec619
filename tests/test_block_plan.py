"""The launch plans of the decoder block's products, from sizes and types alone
(host code): the ones that were measured faster with the weights in memory; and
the workspaces that they ask for."""
import ctypes

import pytest

import lora_adapter_pool_amd as L
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


SIZES = sorted({*range(1, 300, 7), 32, 33, 64, 65, 128, 129, 256, 257, 511, 512, 513, 777, 1024,
                2000, 2048, 4096, 8192, 8960, 1 << 17})


def grows(size, label):
    """`size` of every T in SIZES; it never shrinks, so that the largest T's
    workspace serves them all."""
    got = [size(T) for T in SIZES]
    for k in range(1, len(got)):
        assert got[k - 1] <= got[k] <= (64 << 20) + 256, (label, SIZES[k - 1:k + 1], got[k - 1:k + 1])
    return got


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,od", TYPES)
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(dtype, od):
    """What the queries return does not shrink with T, and no plan takes more."""
    code = {"f32": _lib.LORA_F32, "bf16": BF16, "e4m3": _lib.LORA_E4M3}
    es = {"f32": 4, "bf16": 2, "e4m3": 1}[dtype]
    for K, O in ((64, 32), (256, 256), (4096, 4096), (4096, 6144), (14336, 4096), (4096, 14336),
                 (2048, 2048), (528, 2064), (16, 9408)):
        d = L.make_linear_desc(dtype, od, K, O)
        g = L.make_gated_desc(dtype, od, K, O)
        for form, f, desc in ((LINEAR, L.lora_linear_workspace_bytes, d),
                              (GATED, L.lora_gated_ffn_workspace_bytes, g)):
            got = grows(lambda T: f(desc, T), (dtype, od, K, O, form))
            for T, n in zip(SIZES, got):
                assert plan(form, T, K, O, code[dtype], code[od], es).ws_bytes <= n, (T, K, O, form)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_gradients_workspace_serves_smaller_batches_and_either_gradient(dtype):
    size = L.lora_gated_ffn_backward_workspace_bytes
    for K, I in ((64, 32), (520, 264), (2048, 2048), (4096, 4096), (144, 968), (4096, 14336),
                 (1024, 2816)):
        d = L.make_gated_desc(dtype, dtype, K, I)
        both = grows(lambda T: size(d, T), (dtype, K, I))
        for k, alone in enumerate((grows(lambda T: size(d, T, True, False), (dtype, K, I, "dx")),
                                   grows(lambda T: size(d, T, False, True), (dtype, K, I, "dw")))):
            assert all(a <= b for a, b in zip(alone, both)), (K, I, k)
