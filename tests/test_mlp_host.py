"""LoraMlp's checks of weights, pools and rows, on the CPU (nothing is launched)."""
import gc
import weakref

import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib


def weights(H=64, I=72, dtype=torch.bfloat16):
    return [torch.ones(H, dtype=dtype), torch.zeros(2 * I, H, dtype=dtype),
            torch.zeros(H, I, dtype=dtype)]


def refused(status, *a, **k):
    with pytest.raises(L.LoraError) as e:
        L.LoraMlp(*a, **k)
    assert e.value.status == status


def test_weight_refusals():
    n, gu, d = weights()
    L.LoraMlp(n, gu, d)
    refused(_lib.LORA_E_DTYPE, n.float(), gu, d)
    refused(_lib.LORA_E_DTYPE, n, gu.float(), d)
    refused(_lib.LORA_E_DTYPE, n.half(), gu.half(), d.half())
    refused(_lib.LORA_E_SHAPE, n, gu[:-1].clone(), d)
    refused(_lib.LORA_E_SHAPE, n[:-8].clone(), gu, d)
    refused(_lib.LORA_E_SHAPE, n, gu.t().contiguous().t(), d)
    g8 = gu.to(torch.float8_e4m3fn)
    refused(_lib.LORA_E_DTYPE, n, g8, d)                                    # no scales
    refused(_lib.LORA_E_DTYPE, n, gu, d, gate_up_scale=torch.ones(144))     # scales of nothing
    refused(_lib.LORA_E_SHAPE, n, g8, d, gate_up_scale=torch.ones(143))
    n4, g4, d4 = weights(dtype=torch.float32)
    refused(_lib.LORA_E_DTYPE, n4, g8, d4, gate_up_scale=torch.ones(144))   # fp32 activations


def test_pool_refusals():
    n, gu, d = weights()
    fits = L.LoraPool("bf16", 2, 8, 64, [72, 72], device="cpu")
    L.LoraMlp(n, gu, d, gate_up=fits)
    refused(_lib.LORA_E_SHAPE, n, gu, d, gate_up=L.LoraPool("bf16", 2, 8, 64, [144], device="cpu"))
    refused(_lib.LORA_E_SHAPE, n, gu, d, down=fits)
    refused(_lib.LORA_E_SHAPE, n, gu, d, gate_up=L.LoraPool("f32", 2, 8, 64, [72, 72], device="cpu"))


def test_row_refusals():
    n, gu, d = weights()
    m = L.LoraMlp(n, gu, d)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for a, b, status in ((x.float(), x, _lib.LORA_E_DTYPE), (x[:, :56], x, _lib.LORA_E_SHAPE),
                         (x, x[:3], _lib.LORA_E_SHAPE), (x[0], x, _lib.LORA_E_SHAPE),
                         (x.t().contiguous().t(), x, _lib.LORA_E_SHAPE)):
        with pytest.raises(L.LoraError) as e:
            m.forward(a, b)
        assert e.value.status == status
    with pytest.raises(L.LoraError) as e:
        m.forward(x, x)                                                     # not on a GPU
    assert e.value.status == _lib.LORA_E_ARG
    with pytest.raises(L.LoraError):
        m.gate_up_backward(torch.zeros(4, 72, dtype=torch.bfloat16))        # nothing kept


def test_an_outgrown_workspace_lives_as_long_as_the_block():
    """A captured graph holds its address: the memory must not go to another
    tensor when a later call needs more."""
    m = L.LoraMlp(*weights())
    sizes = (0, 300, 100, 301, 5000, 4000, 70000)
    held = [weakref.ref(m._workspace(n)) for n in sizes]
    assert all(m._workspace(n).numel() >= n for n in sizes)
    gc.collect()
    assert all(r() is not None for r in held)
    assert held[1]() is held[2]() and held[4]() is held[5]()       # grown only where needed
    kept = {id(r()): r().numel() for r in held}
    assert sum(kept.values()) <= 2 * m._workspace(0).numel()       # and not without end
