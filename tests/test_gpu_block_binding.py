"""GPU tensors through the binding of the decoder-block operators: views that are
not what a kernel would read are refused before the call, others are taken."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import gen, normal, run_linear
from gpu_helpers import say
from lora_adapter_pool_amd import _lib

pytestmark = pytest.mark.gpu
T, K, O = 24, 64, 40
LIN = L.make_linear_desc("bf16", "bf16", K, O)


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def _call(x, w, out, bias=None):
    n = L.lora_linear_workspace_bytes(LIN, T)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    L.lora_linear(LIN, x, w, None, None, bias, None, None, out, T, ws, n)


def test_views_that_are_refused():
    g = gen(1)
    x, w = normal(g, (T, K), "bf16"), normal(g, (O, K), "bf16")
    out = torch.full((T, O), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = [("w", normal(g, (K, O), "bf16").t(), _lib.LORA_E_SHAPE),
           ("w", normal(g, (O, 2 * K), "bf16")[:, :K], _lib.LORA_E_SHAPE),
           ("w", normal(g, (1, K), "bf16").expand(O, K), _lib.LORA_E_SHAPE),
           ("w", torch.nn.Parameter(normal(g, (K, O), "bf16")).t(), _lib.LORA_E_SHAPE),
           ("w", w[:-1], _lib.LORA_E_SHAPE), ("w", w.cpu(), _lib.LORA_E_ARG),
           ("w", w.cpu().pin_memory(), _lib.LORA_E_ARG),
           ("w", w.to(torch.float8_e4m3fn), _lib.LORA_E_SHAPE)]
    for name, t, status in bad:
        with pytest.raises(L.LoraError) as e:
            _call(x, t, out)
        assert e.value.status == status and f"linear: {name} " in str(e.value)
    for o in (out[:, :-8], out[:-1], torch.empty((O, T), dtype=out.dtype, device="cuda").t()):
        with pytest.raises(L.LoraError) as e:
            _call(x, w, o)
        assert e.value.status == _lib.LORA_E_SHAPE
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_tensors_that_are_taken():
    g = gen(2)
    x, w = normal(g, (T, K), "bf16"), normal(g, (O, K), "bf16")
    bias = normal(g, (O,), "bf16")
    want = run_linear(x, w, None, None, bias, None, None, "bf16", "bf16", "none")
    deep = normal(g, (O + 8, K), "bf16")
    deep[8:] = w
    for xx, ww, bb in ((x, torch.nn.Parameter(w), bias), (x.view(T, 1, K), w, bias[None]),
                       (x.view(torch.uint8), w.view(torch.int16), bias), (x, deep[8:], bias),
                       (torch.cat([x, x]), w, bias),
                       (x, w, torch.empty_strided((1, O), (5, 1), dtype=bias.dtype,
                                                  device="cuda").copy_(bias[None]))):
        out = torch.full((T, O), float("nan"), dtype=torch.bfloat16, device="cuda")
        _call(xx, ww, out, bb)
        assert torch.equal(out, want)
