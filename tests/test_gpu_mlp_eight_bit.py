"""LoraMlp with gate/up weights in 8 bits and no adapters in the batch: the norm
writes its 8-bit output alone (nobody reads the other), with the same result."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import gen, normal, rows8
from gpu_helpers import say
from lora_adapter_pool_amd import mlp as mlp_module

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 70])
def test_norm_output_that_nobody_reads(T, monkeypatch):
    say(f"[gpu] test_norm_output_that_nobody_reads {T}")
    H, I = 272, 528
    g = gen(T)
    w8, scale = rows8(torch.randn((2 * I, H), generator=g, device="cuda") * H ** -0.5)
    w = normal(g, (H,), "bf16"), w8, normal(g, (H, I), "bf16", I ** -0.5)
    pool = L.LoraPool("bf16", 2, 8, H, [I, I])
    x, r = normal(g, (T, H), "bf16"), normal(g, (T, H), "bf16")
    written, norm = [], L.lora_add_rms_norm

    def spy(desc, *a, **k):
        written.append(a[4] is not None)
        norm(desc, *a, **k)

    monkeypatch.setattr(mlp_module.L, "lora_add_rms_norm", spy)
    plain = L.LoraMlp(*w, gate_up_scale=scale).forward(x, r)
    pooled = L.LoraMlp(*w, gate_up_scale=scale, gate_up=pool)
    without = pooled.forward(x, r, keep=True)
    none = pooled.forward(x, r, np.full(T, -1, np.int32))
    assert written == [False, False, True]
    assert torch.equal(plain, without) and torch.equal(plain, none)
    with pytest.raises(L.LoraError) as e:
        pooled.forward(x, r, keep=True)
        pooled.gate_up_backward(torch.zeros((T, I), dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == L._lib.LORA_E_DTYPE
