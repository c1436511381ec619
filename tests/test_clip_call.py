"""lora_clip_grads' way to the library: the current GPU is asked for once a call (with 14
small tensors the host's time is the call's), and the stream is the tensors' GPU's."""
from types import SimpleNamespace

import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib


@pytest.mark.parametrize("current", [0, 1])
def test_one_question_a_call(monkeypatch, current):
    now, asked, streams = [current], [], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, now[0] = now[0], self.device.index

        def __exit__(self, *_):
            now[0] = self.before

    def device():
        asked.append(now[0])
        return now[0]

    monkeypatch.setattr(torch.cuda, "current_device", device)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(_lib, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(_lib, "pycall", lambda: SimpleNamespace(
        clip_grads=lambda *a: streams.append((now[0], a[-1])) or 0))
    grads = SimpleNamespace(struct=_lib.lora_grad_list(), image=1 << 20,
                            device=torch.device("cuda", 1))
    L.lora_clip_grads(grads, 1.0, 1 << 20, 1 << 20, 1 << 20)
    assert asked == [current] and streams == [(1, 101)] and now == [current]
    L.lora_clip_grads(grads, 1.0, 1 << 20, 1 << 20, 1 << 20, stream=7)
    assert streams[1] == (1, 7)
