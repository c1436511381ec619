"""What LoraMlp.forward holds for the gradients: for gate_up_backward alone no more than it
takes, for backward no tensor that the block's form does not need."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from gpu_helpers import say
from lora_adapter_pool_amd import _lib

H, I, T = 64, 72, 3
FORMS = [("plain", {}), ("scaled", {"residual_scale": 0.5, "block_scale": 0.7}),
         ("gated", {"gate": True}), ("normed", {"post": True, "gate": True})]


def block(device, form, down, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    k = dict(form)
    if k.pop("gate", False):
        k["gate"] = n(H)
    if k.pop("post", False):
        k["post_norm_weight"] = n(H)
    if down:
        k["down"] = L.LoraPool("f32", 2, 8, I, [H], device=device)
        for t in (k["down"].A, k["down"].B):
            t.copy_(n(t.numel()) * 0.1)
    return L.LoraMlp(n(H), n(2 * I, H) * 0.1, n(H, I) * 0.1, **k), n(T, H), n(T, H), n(T, H)


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("name,form", FORMS)
def test_kept_tensors(name, form, down):
    m, x, residual, _ = block("cpu", form, down)
    m._workspace = lambda need: torch.zeros(1)
    ids = np.array([0, -1, 1], np.int32)
    with pytest.MonkeyPatch.context() as patch:
        for f in ("lora_add_rms_norm", "lora_gated_ffn", "lora_linear", "lora_block_norm"):
            patch.setattr(_lib, f, lambda *a, **k: None)
        patch.setattr(L.LoraPool, "apply", lambda *a, **k: None)
        for given in (ids, None):
            m._forward(x, residual, given, None, True)
            s, h, kept_block, kept_ids = m._saved_rest
            assert s.shape == (T, H) and (kept_ids is None) == (given is None)
            assert (h is not None) == (down and given is not None)
            assert (kept_block is not None) == (name in ("gated", "normed"))
        m._forward(x, residual, ids, None, "gate_up")
        assert m._saved_rest is None and m._saved[1].shape == (T, 2 * I)
    with pytest.raises(L.LoraError) as e:
        m.backward(x, torch.zeros(I, H))
    assert e.value.status == _lib.LORA_E_ARG
    with pytest.raises(L.LoraError):
        m.forward(x, residual, ids, None, "down")


@pytest.mark.gpu
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("name,form", FORMS)
def test_gradients_of_every_form(name, form, down):
    """Against autograd in 64 bits: random signs, so that a sum of n fp32 products is off by at
    most sqrt(n) (n + 8) 2^-23 of its norm; the longest has 2 I = 144, and five follow each
    other."""
    say(f"[gpu] {name} down={down}")
    m, x, residual, dy = block("cuda", form, down, 3)
    ids = np.array([0, -1, 1], np.int32) if down else None
    m.forward(x, residual, ids, None, keep=True)
    wt = m.w_down.t().contiguous()
    got = m.backward(dy, wt)
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    X, gate, post, w = leaf(x), leaf(m.gate), leaf(m.post_norm_weight), leaf(m.norm_weight)
    norm = lambda t, v: t * (t.square().mean(1, keepdim=True) + 1e-5).rsqrt() * v  # noqa: E731
    s = X + residual.double()
    pre = norm(s, w) @ m.w_gate_up.double().t()
    h = torch.nn.functional.silu(pre[:, :I]) * pre[:, I:]
    b = h @ m.w_down.double().t()
    if down:
        A, B = leaf(m.down.A_view()), leaf(m.down.B_view())
        b = b + torch.stack([h[t] * 0 @ A[0, 0].t() @ B[0].t() if a < 0 else
                             h[t] @ A[a, 0].t() @ B[a].t() for t, a in enumerate(ids)])
    if post is not None:
        b = norm(b, post)
    if gate is not None:
        b = gate * b
    y = form.get("residual_scale", 1.0) * s + form.get("block_scale", 1.0) * b
    (y * dy.double()).sum().backward()
    want = {"x": X.grad, "norm_weight": w.grad}
    if gate is not None:
        want["gate"] = gate.grad
    if post is not None:
        want["post_norm_weight"] = post.grad
    pair = got.pop("down", None)
    if down:
        want["A"], want["B"] = A.grad, B.grad
        got["A"], got["B"] = pair
    assert set(got) == set(want)
    bound = 5 * 144 ** 0.5 * 152 * 2.0 ** -23
    for k, v in want.items():
        assert (got[k].double() - v).norm() <= bound * v.norm(), k
    m.forward(x, residual, ids, None, keep="gate_up")
    one = m.gate_up_backward(h.float().detach())
    m.forward(x, residual, ids, None, keep=True)
    assert all(torch.equal(a, c) for a, c in zip(one, m.gate_up_backward(h.float().detach())))
