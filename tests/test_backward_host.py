"""LoraPool.backward's and LoraMlp.backward's checks on the CPU (nothing is launched)."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib


def refused(status, f, *a, **k):
    with pytest.raises(L.LoraError) as e:
        f(*a, **k)
    assert e.value.status == status


def test_pool_refusals():
    pool = L.LoraPool("bf16", 2, 8, 64, [72], device="cpu")
    plan = pool.backward_plan([0, 1, -1])
    assert plan.T == 3 and plan.image.dtype == torch.int32
    x, dy = torch.zeros(3, 64).bfloat16(), torch.zeros(3, 72).bfloat16()
    refused(_lib.LORA_E_ARG, pool.backward, x, dy, plan)            # not on a GPU
    refused(_lib.LORA_E_ID, pool.backward_plan, [0, 2])
    refused(_lib.LORA_E_SHAPE, pool.backward_plan, np.zeros((2, 2), np.int32))


def test_another_pools_plan():
    a = L.make_desc("bf16", 8, 16, 256, [256])
    b = L.make_desc("bf16", 4, 16, 256, [256])
    plan, _ = L.lora_delta_backward_plan(a, [7, 0, 1])
    refused(_lib.LORA_E_ARG, L.lora_delta_backward, b, *[1 << 20] * 8, 3, plan, 1 << 20, False,
            1 << 20, 1 << 40, stream=0)


def test_mlp_refusals():
    w = [torch.ones(64).bfloat16(), torch.zeros(144, 64).bfloat16(), torch.zeros(64, 72).bfloat16()]
    refused(_lib.LORA_E_DTYPE, L.LoraMlp, *w, gate=torch.ones(64))
    refused(_lib.LORA_E_SHAPE, L.LoraMlp, *w, post_norm_weight=torch.ones(72).bfloat16())
    m = L.LoraMlp(*w)
    dy, wt = torch.zeros(4, 64).bfloat16(), torch.zeros(72, 64).bfloat16()
    refused(_lib.LORA_E_ARG, m.backward, dy, wt)                    # nothing kept
    m._saved, m._saved_rest = (dy, torch.zeros(4, 144).bfloat16()), (dy, dy, None, None)
    refused(_lib.LORA_E_SHAPE, m.backward, dy[:3], wt)
    refused(_lib.LORA_E_DTYPE, m.backward, dy.float(), wt)
    refused(_lib.LORA_E_SHAPE, m.backward, dy, wt.t())
    refused(_lib.LORA_E_DTYPE, m.backward, dy, wt.float())
    refused(_lib.LORA_E_ARG, m.backward, dy, wt, grads={"x": dy})
    refused(_lib.LORA_E_SHAPE, m.backward, dy, wt, grads={"gate": torch.zeros(64).bfloat16()})
    assert m._saved is not None


def test_forms_of_the_block():
    w = [torch.ones(64), torch.zeros(144, 64), torch.zeros(64, 72)]
    assert L.LoraMlp(*w).join_desc is None
    d = L.LoraMlp(*w, residual_scale=0.5).join_desc
    assert (d.gate, d.residual_scale, d.block_scale) == (0, 0.5, 1.0)
    d = L.LoraMlp(*w, gate=torch.ones(64), block_scale=2.0).join_desc
    assert (d.gate, d.residual_scale, d.block_scale) == (1, 1.0, 2.0)


def test_slots_of_a_list():
    pool = L.LoraPool("bf16", 2, 8, 64, [72], device="cpu")
    dA, dB = torch.zeros(pool.A_view().shape), torch.zeros(pool.B_view().shape)
    for slots in ([-1], [2], [0, 5]):
        refused(_lib.LORA_E_ID, pool.slot_grads, dA, dB, slots)
    refused(_lib.LORA_E_SHAPE, pool.slot_grads, dA[:1], dB, [0])
    refused(_lib.LORA_E_SHAPE, pool.slot_grads, dA, dB, [0], (dA, dB[:, :8]))
    refused(_lib.LORA_E_DTYPE, pool.slot_grads, dA.bfloat16(), dB, [0])
    refused(_lib.LORA_E_ARG, pool.slot_grads, dA, None, [0])
    refused(_lib.LORA_E_ARG, pool.slot_grads, dA, dB, [])


def test_a_block_refuses_before_it_adds():
    """Gradients and plans that do not fit are refused while nothing has been added to."""
    w = [torch.ones(64), torch.zeros(144, 64), torch.zeros(64, 72)]
    pools = [L.LoraPool("f32", 2, 8, 64, [72, 72], device="cpu"),
             L.LoraPool("f32", 2, 8, 72, [64], device="cpu")]
    m = L.LoraMlp(*w, gate_up=pools[0], down=pools[1], gate=torch.ones(64))
    dy, wt, ids = torch.zeros(4, 64), torch.zeros(72, 64), np.array([0, 1, -1, 0], np.int32)
    m._saved, m._saved_rest = (dy, torch.zeros(4, 144)), (dy, dy, dy, ids)
    pair = [torch.zeros(p.A_view().shape) for p in pools]
    for grads in ({"post_norm_weight": torch.zeros(64)},                  # the block has none
                  {"gate_up": (pair[0], None)}, {"down": (pair[0], pair[1])},
                  {"norm_weight": torch.zeros(72)}):
        with pytest.raises(L.LoraError):
            m.backward(dy, wt, grads=grads)
    for plans in ({"norm_weight": None}, {"down": pools[0].backward_plan(ids)},
                  {"down": pools[1].backward_plan(ids[:3])}):
        refused(_lib.LORA_E_ARG, m.backward, dy, wt, plans=plans)
    assert m._saved is not None and m._saved_rest is not None


def test_only_a_kept_pass_copies_its_ids():
    class Ids:
        def __array__(self, *a, **k):
            raise AssertionError("copied")

    m = L.LoraMlp(torch.ones(64), torch.zeros(144, 64), torch.zeros(64, 72))
    m._workspace = lambda need: torch.zeros(1)
    x = torch.zeros(3, 64)
    names = ("lora_add_rms_norm", "lora_gated_ffn", "lora_linear")
    with pytest.MonkeyPatch.context() as patch:
        for name in names:
            patch.setattr(_lib, name, lambda *a, **k: None)
        m._forward(x, x, Ids(), None, False)
        assert m._saved_rest is None
        m._forward(x, x, [0, 1, 0], None, True)
        assert m._saved_rest[3].tolist() == [0, 1, 0]
