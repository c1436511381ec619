"""GPU tensors through the binding of the training operators: views that are not what a
kernel would read are refused before the call."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_norm_helpers import inputs
from delta_helpers import batch
from gpu_helpers import say
from lora_adapter_pool_amd import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def refused(f, args, i, value, status):
    a = list(args)
    a[i] = value
    with pytest.raises(L.LoraError) as e:
        f(*a)
    assert e.value.status == status, i


def bad_views(t):
    wide = torch.empty(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device="cuda")
    yield wide[..., :t.shape[-1]] if t.dim() > 1 else wide[::2], _lib.LORA_E_SHAPE
    yield t.flatten()[:-1], _lib.LORA_E_SHAPE
    yield t.cpu(), _lib.LORA_E_ARG


def test_block_norm_views():
    T, H = 6, 64
    s = inputs(1, T, H, "bf16", "element")
    d = L.make_block_norm_desc("bf16", H, 1e-5, "element")
    out8 = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    args = [d, s["y"], s["residual"], s["gate"], s["post"], s["pre"], torch.empty_like(s["y"]),
            torch.empty_like(s["y"]), out8, torch.empty(T, device="cuda"), T]
    L.lora_block_norm(*args)
    for i in range(1, 10):
        for v, status in bad_views(args[i]):
            refused(L.lora_block_norm, args, i, v, status)
    n = L.lora_block_norm_backward_workspace_bytes(d, T)
    new = lambda: torch.empty_like(s["y"])  # noqa: E731
    args = [d, s["dout"], s["dsum"], s["y"], s["sum"], s["gate"], s["post"], s["pre"], new(), new(),
            new(), torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), False, T,
            torch.empty(n, dtype=torch.uint8, device="cuda"), n]
    L.lora_block_norm_backward(*args)
    for i in range(1, 13):
        for v, status in bad_views(args[i]):
            refused(L.lora_block_norm_backward, args, i, v, status)
    refused(L.lora_block_norm_backward, args, 15, args[15][:-1], _lib.LORA_E_WORKSPACE)
    refused(L.lora_block_norm_backward, args, 12, torch.empty(H, device="cuda").bfloat16(),
            _lib.LORA_E_SHAPE)


def test_delta_views():
    s = batch(1, "bf16", [0, 1, -1, 1], 64, [72], 2, 8)
    d = L.make_desc("bf16", 2, 8, 64, [72])
    plan, image = L.lora_delta_backward_plan(d, s["ids"])
    n = L.lora_delta_backward_workspace_bytes(d, 4)
    args = [d, s["A"], s["B"], s["x"], s["dy"], s["dx_in"], torch.empty_like(s["x"]),
            torch.zeros(s["A"].shape, device="cuda"), torch.zeros(s["B"].shape, device="cuda"), 4,
            plan, torch.from_numpy(image.copy()).cuda(), False,
            torch.empty(n, dtype=torch.uint8, device="cuda"), n]
    L.lora_delta_backward(*args)
    for i in (1, 2, 3, 4, 5, 6, 7, 8, 11):
        for v, status in bad_views(args[i]):
            refused(L.lora_delta_backward, args, i, v, status)
    refused(L.lora_delta_backward, args, 7, args[7].bfloat16(), _lib.LORA_E_SHAPE)
    refused(L.lora_delta_backward, args, 13, args[13][:-1], _lib.LORA_E_WORKSPACE)


def test_pool_backward_views():
    pool = L.LoraPool("bf16", 2, 8, 64, [72])
    plan = pool.backward_plan([0, 1, -1, 1])
    x, dy = torch.randn(4, 64, device="cuda").bfloat16(), torch.randn(4, 72, device="cuda").bfloat16()
    dx, dA, dB = pool.backward(x, dy, plan)
    assert dx.shape == x.shape and dA.shape == (2, 1, 8, 64) and dB.shape == (2, 72, 8)
    for a, k, status in (((x[:3], dy, plan), {}, _lib.LORA_E_SHAPE),
                         ((x.float(), dy, plan), {}, _lib.LORA_E_DTYPE),
                         ((x.cpu(), dy, plan), {}, _lib.LORA_E_DTYPE),
                         ((x, dy, plan), {"dA": dA}, _lib.LORA_E_ARG),
                         ((x, dy, plan), {"dA": dA.bfloat16(), "dB": dB}, _lib.LORA_E_DTYPE),
                         ((x, dy, plan), {"dA": dA, "dB": dB, "need_grads": False},
                          _lib.LORA_E_ARG),
                         ((x, dy, plan), {"dx": dx, "need_dx": False}, _lib.LORA_E_ARG),
                         ((x, dy, plan), {"need_dx": False, "need_grads": False},
                          _lib.LORA_E_ARG)):
        with pytest.raises(L.LoraError) as e:
            pool.backward(*a, **k)
        assert e.value.status == status
    other = L.LoraPool("bf16", 3, 8, 64, [72])
    with pytest.raises(L.LoraError):
        other.backward(x, dy, plan)
