"""LoraMlp.backward refuses gradient buffers that one of its operators could not take before
any of them has been added to."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from gpu_helpers import say
from lora_adapter_pool_amd import _lib

H, I, T = 64, 72, 4


def block(device):
    w = [torch.ones(H, device=device), torch.zeros(2 * I, H, device=device),
         torch.zeros(H, I, device=device)]
    pools = {"gate_up": L.LoraPool("f32", 2, 8, H, [I, I], device=device),
             "down": L.LoraPool("f32", 2, 8, I, [H], device=device)}
    m = L.LoraMlp(*w, gate=torch.ones(H, device=device), **pools)
    grads = {k: torch.full((H,), 3.0, device=device) for k in ("norm_weight", "gate")}
    for k, p in pools.items():
        grads[k] = tuple(torch.full(v.shape, 3.0, device=device) for v in (p.A_view(), p.B_view()))
    return m, pools, grads


def off(t):
    """The same tensor four bytes past 16."""
    return torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)


def wrong(pools, grads, dy, wt):
    """(status, dy, w_down_t, gradient buffers) that have to be refused."""
    (A, B), (Ad, Bd) = grads["gate_up"], grads["down"]
    yield _lib.LORA_E_ALIGN, dy, wt, dict(grads, norm_weight=off(grads["norm_weight"]))
    yield _lib.LORA_E_ALIGN, dy, wt, dict(grads, gate_up=(A, off(B)))
    yield _lib.LORA_E_ALIGN, off(dy), wt, grads
    yield _lib.LORA_E_ALIGN, dy, off(wt), grads
    yield _lib.LORA_E_ARG, dy, wt, dict(grads, norm_weight=grads["gate"])
    yield _lib.LORA_E_ARG, dy, wt, dict(grads, gate_up=(B.flatten()[8:8 + A.numel()].view(A.shape), B))
    yield _lib.LORA_E_ARG, dy, wt, dict(grads, norm_weight=dy.flatten()[H:2 * H])
    yield _lib.LORA_E_ARG, dy, wt, dict(grads, down=(pools["down"].A_view(), Bd))


def flat(grads):
    return [t for v in grads.values() for t in (v if isinstance(v, tuple) else (v,))]


def check(m, pools, grads, dy, wt):
    n = 0
    for status, d, w, g in wrong(pools, grads, dy, wt):
        with pytest.raises(L.LoraError) as e:
            m.backward(d, w, grads=g, accumulate=True)
        assert e.value.status == status, n
        assert all((t == 3).all() for t in flat(grads)), n
        n += 1
    assert n == 8 and m._saved is not None and m._saved_rest is not None


def test_refused_on_the_host():
    m, pools, grads = block("cpu")
    dy = torch.zeros(T, H)
    m._saved = dy, torch.zeros(T, 2 * I)
    m._saved_rest = dy, torch.zeros(T, I), dy, np.array([0, 1, -1, 0], np.int32)
    check(m, pools, grads, dy, torch.zeros(I, H))


@pytest.mark.gpu
def test_nothing_is_added():
    say("[gpu] test_nothing_is_added")
    m, pools, grads = block("cuda")
    x = torch.randn(T, H, device="cuda")
    m.forward(x, x, np.array([0, 1, -1, 0], np.int32), keep=True)
    check(m, pools, grads, torch.randn(T, H, device="cuda"), torch.zeros(I, H, device="cuda"))
    # (weights and adapters are zero, and so are the gradients)
    out = m.backward(x, torch.zeros(I, H, device="cuda"), grads=grads, accumulate=True)
    assert all((t == 3).all() for t in flat(grads)) and torch.equal(out["x"], x)
