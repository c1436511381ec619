"""lora_block_norm on the CPU: the 64-bit gradients that the GPU tests compare with
against differences of the 64-bit forward pass, and every refusal before a GPU call."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_norm_helpers import inputs, join64, join_grad64, norm64
from lora_adapter_pool_amd import _lib
from test_block_host import FAKE, status, variants


@pytest.mark.parametrize("gate", ["none", "channel", "element"])
@pytest.mark.parametrize("post", [False, True])
def test_formulas_against_differences(gate, post):
    s = {k: None if v is None else v.double() for k, v in
         inputs(5, 3, 16, "f32", gate, device="cpu").items()}
    alpha, beta, eps, h = 0.7, -0.4, 1e-3, 1e-6
    pw = s["post"] if post else None

    def value(y, residual, g, w, pre):
        t, _ = join64(y, residual, g, w, alpha, beta, eps)
        return (norm64(t, pre, eps) * s["dout"]).sum() + (t * s["dsum"]).sum()

    at = [s["y"], s["residual"], s["gate"], pw, s["pre"]]
    t, _ = join64(*at[:4], alpha, beta, eps)
    got = join_grad64(s["dout"], s["dsum"], s["y"], t, s["gate"], pw, s["pre"], alpha, beta, eps)
    for k, name in enumerate(("dy", "dresidual", "dgate", "dpost", "dpre")):
        if at[k] is None:
            assert name not in got
            continue
        num = torch.empty_like(at[k])
        for i in range(num.numel()):
            v = []
            for sign in (1, -1):
                moved = list(at)
                moved[k] = at[k].clone()
                moved[k].view(-1)[i] += sign * h
                v.append(value(*moved))
            num.view(-1)[i] = (v[0] - v[1]) / (2 * h)
        # a third derivative times h^2 / 6, and 2^-52 of the sum's terms over h
        assert torch.allclose(got[name][0], num, rtol=1e-7, atol=1e-8), name


mk = L.make_block_norm_desc


def test_descriptor_refusals():
    for bad, want in ((("fp16", 64, 1e-5), _lib.LORA_E_DTYPE),
                      (("bf16", 64.5, 1e-5), _lib.LORA_E_SHAPE),
                      (("bf16", 64, 1e-5, "row"), _lib.LORA_E_ARG),
                      (("bf16", 64, 1e-5, None), _lib.LORA_E_ARG)):
        with pytest.raises(L.LoraError) as e:
            mk(*bad)
        assert e.value.status == want


BAD = [(mk("e4m3", 1024, 1e-5), _lib.LORA_E_DTYPE), (mk("bf16", 0, 1e-5), _lib.LORA_E_SHAPE),
       (mk("bf16", 1028, 1e-5), _lib.LORA_E_ALIGN), (mk("bf16", 16392, 1e-5), _lib.LORA_E_SHAPE),
       (mk("bf16", 1024, -1.0), _lib.LORA_E_ARG), (mk("bf16", 1024, float("inf")), _lib.LORA_E_ARG),
       (mk("bf16", 1024, 1e-5, "none", float("nan")), _lib.LORA_E_ARG),
       (mk("bf16", 1024, 1e-5, "none", 1.0, float("inf")), _lib.LORA_E_ARG), (None, None)]


def test_forward_refusals():
    d = mk("bf16", 1024, 1e-5, "channel")
    ok = [d] + [FAKE] * 9 + [4]
    variants(L.lora_block_norm, ok, [(0, b, w) for b, w in BAD[:-1]] + [
        (0, mk("bf16", 1024, 1e-5), _lib.LORA_E_ARG),              # a gate that is not declared
        (3, None, _lib.LORA_E_ARG), (1, None, _lib.LORA_E_ARG), (2, None, _lib.LORA_E_ARG),
        (6, None, _lib.LORA_E_ARG), (5, None, _lib.LORA_E_ARG), (8, None, _lib.LORA_E_ARG),
        (9, None, _lib.LORA_E_ARG), (1, FAKE + 2, _lib.LORA_E_ALIGN),
        (9, FAKE + 4, _lib.LORA_E_ALIGN), (3, FAKE + 8, _lib.LORA_E_ALIGN),
        (10, -1, _lib.LORA_E_ARG), (10, (1 << 21) + 1, _lib.LORA_E_SHAPE)])
    assert status(L.lora_block_norm, d, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None, None, 4) \
        == _lib.LORA_E_ARG                                         # a weight without an output
    assert status(L.lora_block_norm, d, *[None] * 9, 0) == 0       # T = 0
    bad = mk("bf16", 1024, 1e-5, "channel")
    bad.gate = 3
    assert status(L.lora_block_norm, bad, *[FAKE] * 9, 4) == _lib.LORA_E_ARG


def test_backward_refusals():
    d = mk("bf16", 1024, 1e-5, "channel")
    need = L.lora_block_norm_backward_workspace_bytes(d, 4)
    assert need == 3 * 4 * 1024 * 4
    assert L.lora_block_norm_backward_workspace_bytes(d, 0) == 0
    assert L.lora_block_norm_backward_workspace_bytes(d, 1 << 21) == 3 * 2048 * 1024 * 4
    ok = [d] + [FAKE] * 12 + [0, 4, FAKE, need]
    variants(L.lora_block_norm_backward, ok, [(0, b, w) for b, w in BAD[:-1]] + [
        (0, mk("bf16", 1024, 1e-5), _lib.LORA_E_ARG), (1, None, _lib.LORA_E_ARG),
        (3, None, _lib.LORA_E_ARG), (4, None, _lib.LORA_E_ARG), (5, None, _lib.LORA_E_ARG),
        (6, None, _lib.LORA_E_ARG), (7, None, _lib.LORA_E_ARG), (12, FAKE + 4, _lib.LORA_E_ALIGN),
        (15, FAKE + 4, _lib.LORA_E_ALIGN), (13, 2, _lib.LORA_E_ARG), (14, -1, _lib.LORA_E_ARG),
        (14, (1 << 21) + 1, _lib.LORA_E_SHAPE), (15, None, _lib.LORA_E_ARG),
        (16, need - 1, _lib.LORA_E_WORKSPACE)])
    none = [d, None, None] + [FAKE] * 3 + [FAKE, None] + [FAKE] * 4 + [None, 0, 4, FAKE, need]
    assert status(L.lora_block_norm_backward, *none) == _lib.LORA_E_ARG   # no gradient comes in
    nothing = [d] + [FAKE] * 7 + [None] * 5 + [0, 4, FAKE, need]
    assert status(L.lora_block_norm_backward, *nothing) == _lib.LORA_E_ARG   # and none goes out
    # nothing to add to over no rows
    assert status(L.lora_block_norm_backward, d, *[None] * 12, 1, 0, None, 0) == 0
