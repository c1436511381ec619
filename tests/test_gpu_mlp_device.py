"""LoraMlp works on its weights' GPU, whichever GPU is the current one."""
import contextlib

import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import gen, normal
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def test_launches_go_to_the_weights_gpu(monkeypatch):
    """One GPU plays two: the current device is reported as another one until
    LoraMlp has made the weights' the current one.  Every launch asks for the
    current device's stream and has to find the weights'."""
    say("[gpu] test_launches_go_to_the_weights_gpu")
    H, I, T = 64, 72, 5
    g = gen(3)
    w = [normal(g, (H,), "bf16"), normal(g, (2 * I, H), "bf16"), normal(g, (H, I), "bf16")]
    x, dh = normal(g, (T, H), "bf16"), normal(g, (T, I), "bf16")
    mlp = L.LoraMlp(*w)
    want = mlp.forward(x, x, keep=True), *mlp.gate_up_backward(dh)
    current, entered, asked = [7], [], []

    @contextlib.contextmanager
    def device(d):
        entered.append(torch.device(d))
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    def stream():
        asked.append(current[0])
        return torch.cuda.default_stream(0).cuda_stream

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(L._lib, "_current_stream", stream)
    got = mlp.forward(x, x, keep=True), *mlp.gate_up_backward(dh)
    monkeypatch.undo()
    assert entered == [x.device] * 2 and current == [7]
    assert asked == [0] * 4          # norm, gate/up, down; the gradients
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_pool_on_another_device_is_refused():
    g = gen(4)
    w = [normal(g, (64,), "bf16"), normal(g, (144, 64), "bf16"), normal(g, (64, 72), "bf16")]
    with pytest.raises(L.LoraError) as e:
        L.LoraMlp(*w, gate_up=L.LoraPool("bf16", 2, 8, 64, [72, 72], device="cpu"))
    assert e.value.status == L._lib.LORA_E_ARG
