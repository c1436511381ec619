"""LoraMlp.backward in fp32 against autograd in 64 bits, close enough that a value rounded to
bf16 on the way, or a term of 10^-4 of a gradient that is missing, shows.

Bound, relative to each gradient's norm: in a sum of n terms of random signs the k-th addition
rounds a partial sum of about sqrt(k) terms' size by at most a step, 2^-23 of it; these add up
as sqrt(1 + .. + n), n / sqrt 2 of 2^-23 terms, against a result of sqrt(n): sqrt(n / 2) 2^-23.
The widest has 384 rows.  Nine operators follow each other at most (norm, gate/up, activation,
down, norm after, and back), each passes earlier errors on at about their size, and a norm
over at least 100 elements stays within four times what is expected.  A bf16 rounding is
2^-8 / sqrt 12 of a value on average, some twenty times the bound, which the first test shows
with roundings planted in the 64-bit values."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from gpu_helpers import say

H, I, SLOTS, R = 136, 104, 4, 16
BOUND = 9 * 4 * (384 / 2) ** 0.5 * 2.0 ** -23


class Rounded(torch.autograd.Function):
    """The identity, whose gradient is rounded to bf16."""
    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


def data(seed, T, joined, device):
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(s, generator=g, device=device) * std  # noqa: E731
    w = {"norm": 1 + n(H, std=0.1), "gate_up": n(2 * I, H, std=H ** -0.5),
         "down": n(H, I, std=I ** -0.5)}
    if joined:
        w["post"], w["gate"] = 1 + n(H, std=0.1), n(H, std=0.5)
    adapters = []
    for K, O, S in ((H, 2 * I, 2), (I, H, 1)):
        adapters.append((n(SLOTS, S, R, K, std=K ** -0.5), n(SLOTS, O, R, std=0.3)))
    ids = torch.randint(-1, SLOTS, (T,), generator=torch.Generator().manual_seed(seed))
    return w, adapters, ids.int().numpy(), n(T, H), n(T, H), n(T, H, std=0.1)


def reference(w, adapters, ids, x, residual, dy, joined, rounded=None):
    """The leaves' gradients in 64 bits; `rounded` names a value whose gradient is rounded."""
    at = lambda name, t: Rounded.apply(t) if name == rounded else t  # noqa: E731
    leaf = lambda t: t.double().clone().requires_grad_()  # noqa: E731
    p = {k: leaf(v) for k, v in w.items()}
    A, B = [leaf(a) for a, _ in adapters], [leaf(b) for _, b in adapters]
    X = leaf(x)
    mine = (torch.from_numpy(ids)[:, None] == torch.arange(SLOTS)).double().to(x.device)
    norm = lambda t, v: t * (t.square().mean(1, keepdim=True) + 1e-5).rsqrt() * v  # noqa: E731

    def delta(t, a, b, outs):
        parts, o = [], 0
        for i, width in enumerate(outs):
            v = torch.stack([t @ a[k, i].t() @ b[k, o:o + width].t() for k in range(SLOTS)], 1)
            parts.append((v * mine[:, :, None]).sum(1))
            o += width
        return torch.cat(parts, 1)

    s = at("s", X + residual.double())
    n = at("n", norm(s, p["norm"]))
    pre = at("pre", n @ p["gate_up"].t() + delta(n, A[0], B[0], [I, I]))
    h = at("h", torch.nn.functional.silu(pre[:, :I]) * pre[:, I:])
    block = at("block", h @ p["down"].t() + delta(h, A[1], B[1], [H]))
    y = 0.8 * s + 0.5 * p["gate"] * norm(block, p["post"]) if joined else block + s
    (y * dy.double()).sum().backward()
    got = {"x": X.grad, "norm_weight": p["norm"].grad, "w_gate_up": p["gate_up"].grad,
           "gate_up.A": A[0].grad, "gate_up.B": B[0].grad, "down.A": A[1].grad,
           "down.B": B[1].grad}
    if joined:
        got["post_norm_weight"], got["gate"] = p["post"].grad, p["gate"].grad
    return y.detach(), got


def off(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("T", [1, 384])
@pytest.mark.parametrize("spot,seen", [("n", "x"), ("pre", "gate_up.A"), ("h", "gate_up.B"),
                                       ("block", "down.A"), ("s", "x")])
def test_a_rounding_on_the_way_shows(T, spot, seen):
    d = data(T, T, True, "cpu")
    d[2][0] = 1
    _, clean = reference(*d, True)
    _, rounded = reference(*d, True, spot)
    assert off(rounded[seen], clean[seen]) > 4 * BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("T", [1, 150, 384])
def test_gradients_of_the_block(joined, T):
    say(f"[gpu] T={T} joined={joined}")
    w, adapters, ids, x, residual, dy = data(T, T, joined, "cuda")
    ids[0] = 1
    pools = []
    for (a, b), K, outs in zip(adapters, (H, I), ([I, I], [H])):
        pool = L.LoraPool("f32", SLOTS, R, K, outs)
        pool.A.copy_(a.flatten())
        pool.B.copy_(b.flatten())
        pools.append(pool)
    k = {"post_norm_weight": w["post"], "gate": w["gate"], "residual_scale": 0.8,
         "block_scale": 0.5} if joined else {}
    m = L.LoraMlp(w["norm"], w["gate_up"], w["down"], eps=1e-5, gate_up=pools[0], down=pools[1],
                  **k)
    y = m.forward(x, residual, ids, np.ones(T, np.uint8), keep=True)
    out = m.backward(dy, w["down"].t().contiguous(), need_dw=True)
    got = {k: v for k, v in out.items() if not isinstance(v, tuple)}
    for name in ("gate_up", "down"):
        got[f"{name}.A"], got[f"{name}.B"] = out[name]
    want_y, want = reference(w, adapters, ids, x, residual, dy, joined)
    assert set(got) == set(want)
    got["y"], want["y"] = y, want_y
    for name, v in want.items():
        assert off(got[name], v) <= BOUND, (name, off(got[name], v))
