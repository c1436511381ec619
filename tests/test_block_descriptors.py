"""Descriptors of the decoder-block operators: what they refuse, as LoraError."""
import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib


def refused(status, f, *a, **k):
    with pytest.raises(L.LoraError) as e:
        f(*a, **k)
    assert e.value.status == status


@pytest.mark.parametrize("name", ["fp16", "int8", "", None, 2])
def test_unknown_types(name):
    refused(_lib.LORA_E_DTYPE, L.make_norm_desc, name, 64, 1e-5)
    for make in (L.make_linear_desc, L.make_gated_desc):
        refused(_lib.LORA_E_DTYPE, make, name, "bf16", 64, 64)
        refused(_lib.LORA_E_DTYPE, make, "bf16", name, 64, 64)


@pytest.mark.parametrize("act", ["swish", "SILU", None, 1])
def test_unknown_activations(act):
    for make in (L.make_linear_desc, L.make_gated_desc):
        refused(_lib.LORA_E_ARG, make, "bf16", "bf16", 64, 64, act)
    w = [torch.ones(64), torch.zeros(144, 64), torch.zeros(64, 72)]
    refused(_lib.LORA_E_ARG, L.LoraMlp, *w, act=act)


@pytest.mark.parametrize("n", [(1 << 32) + 64, 1 << 31, -(1 << 32) + 64, 64.5])
def test_sizes_that_a_field_does_not_hold(n):
    refused(_lib.LORA_E_SHAPE, L.make_norm_desc, "bf16", n, 1e-5)
    for make in (L.make_linear_desc, L.make_gated_desc):
        refused(_lib.LORA_E_SHAPE, make, "bf16", "bf16", n, 64)
        refused(_lib.LORA_E_SHAPE, make, "bf16", "bf16", 64, n)


def test_weights_of_the_wrong_rank():
    refused(_lib.LORA_E_SHAPE, L.LoraMlp, torch.ones(64), torch.zeros(144, 64), torch.zeros(64))


def test_known_names():
    for names, code in ((("f32", "fp32", "float32"), 0), (("bf16", "bfloat16"), 1),
                        (("e4m3", "float8_e4m3fn"), 2)):
        for name in names:
            assert L.make_linear_desc(name, "f32", 64, 17).dtype == code
    for k, act in enumerate(("none", "silu", "gelu", "gelu_tanh", "relu")):
        d = L.make_gated_desc("bf16", "f32", 64, 72, act)
        assert (d.act, d.in_features, d.inter_features, d.out_dtype) == (k, 64, 72, 0)
