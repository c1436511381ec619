"""The operators together, as a training step takes them: a block's forward pass, its
gradients down to the adapters of both pools, norms of each slot's gradients and
clipping; against autograd in 64 bits of the same block.

Bounds: relative to each gradient's norm.  fp32: eight products and norms in turn, each
off by at most (n + 8) 2^-23 of its terms' magnitudes, whose sum is below sqrt(n) times
the result's norm for random signs: 8 sqrt(n) (n + 8) 2^-23 at most, n the widest sum
(384 rows or columns).  bf16: s, n, pre, h, y, dh, dpre and dn are rounded, half a step
2^-8 of each, and pass on at most about their own size through a product: 12 2^-8."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import TORCH
from gpu_helpers import say

pytestmark = pytest.mark.gpu
H, I, SLOTS, R = 136, 104, 4, 16
BOUND = {"f32": 8 * 384 ** 0.5 * 392 * 2.0 ** -23, "bf16": 12 * 2.0 ** -8}


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def make(dtype, seed, T, joined):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(  # noqa: E731
        TORCH[dtype])
    w = {"norm": 1 + n(H, std=0.1), "gate_up": n(2 * I, H, std=H ** -0.5),
         "down": n(H, I, std=I ** -0.5)}
    if joined:
        w["post"], w["gate"] = 1 + n(H, std=0.1), n(H, std=0.5)
    pools = []
    for K, outs in ((H, [I, I]), (I, [H])):
        p = L.LoraPool(dtype, SLOTS, R, K, outs)
        p.A.copy_(n(p.A.numel(), std=K ** -0.5))
        p.B.copy_(n(p.B.numel(), std=0.3))
        pools.append(p)
    k = {"post_norm_weight": w["post"], "gate": w["gate"], "residual_scale": 0.8,
         "block_scale": 0.5} if joined else {}
    mlp = L.LoraMlp(w["norm"], w["gate_up"], w["down"], eps=1e-5, gate_up=pools[0], down=pools[1],
                    **k)
    ids = torch.randint(-1, SLOTS - 1, (T,), generator=torch.Generator().manual_seed(seed))
    return mlp, w, pools, ids.int().numpy(), n(T, H), n(T, H), n(T, H, std=0.1)


def reference(w, pools, ids, x, residual, dy, joined):
    """Autograd of the block in 64 bits; the leaves' gradients."""
    leaf = lambda t: t.double().clone().requires_grad_()  # noqa: E731
    p = {k: leaf(v) for k, v in w.items()}
    A = [leaf(q.A_view()) for q in pools]
    B = [leaf(q.B_view()) for q in pools]
    x, residual = leaf(x), leaf(residual)
    at = torch.from_numpy(ids).cuda().long()
    mine = (at[:, None] == torch.arange(SLOTS, device="cuda")).double()

    def norm(t, weight):
        return t * (t.square().mean(1, keepdim=True) + 1e-5).rsqrt() * weight

    def delta(t, a, b, outs):
        parts, o = [], 0
        for i, width in enumerate(outs):
            v = torch.stack([t @ a[k, i].t() @ b[k, o:o + width].t() for k in range(SLOTS)], 1)
            parts.append((v * mine[:, :, None]).sum(1))
            o += width
        return torch.cat(parts, 1)

    s = x + residual
    n = norm(s, p["norm"])
    pre = n @ p["gate_up"].t() + delta(n, A[0], B[0], [I, I])
    h = torch.nn.functional.silu(pre[:, :I]) * pre[:, I:]
    block = h @ p["down"].t() + delta(h, A[1], B[1], [H])
    y = 0.8 * s + 0.5 * p["gate"] * norm(block, p["post"]) if joined else block + s
    (y * dy.double()).sum().backward()
    got = {"x": x.grad, "norm_weight": p["norm"].grad, "w_gate_up": p["gate_up"].grad,
           "gate_up.A": A[0].grad, "gate_up.B": B[0].grad, "down.A": A[1].grad,
           "down.B": B[1].grad}
    assert torch.equal(x.grad, residual.grad)
    if joined:
        got["post_norm_weight"], got["gate"] = p["post"].grad, p["gate"].grad
    return y.detach(), got


def flat(out):
    got = {k: v for k, v in out.items() if not isinstance(v, tuple)}
    for k in ("gate_up", "down"):
        if k in out:
            got[f"{k}.A"], got[f"{k}.B"] = out[k]
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("T", [1, 150, 384])
def test_gradients_of_the_block(dtype, joined, T):
    mlp, w, pools, ids, x, residual, dy = make(dtype, T, T, joined)
    if T == 1:
        ids[:] = 2
    y = mlp.forward(x, residual, ids, np.ones(T, np.uint8), keep=True)
    got = flat(mlp.backward(dy, w["down"].t().contiguous(), need_dw=True))
    want_y, want = reference(w, pools, ids, x, residual, dy, joined)
    assert set(got) == set(want)
    got["y"], want["y"] = y, want_y
    for k, v in want.items():
        rel = ((got[k].double() - v).norm() / v.norm()).item()
        assert rel <= BOUND[dtype], (k, rel)
    idle = [a for a in range(SLOTS) if a not in set(ids.tolist())]
    for k in ("gate_up.A", "down.B"):
        assert (got[k][idle] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_accumulation_and_clipping(dtype):
    """Two batches' gradients into one set of buffers; then a norm for each slot."""
    mlp, w, pools, _, *_ = make(dtype, 1, 1, True)
    wt = w["down"].t().contiguous()
    grads = {k: torch.zeros(H, device="cuda") for k in ("norm_weight", "post_norm_weight", "gate")}
    for k, p in zip(("gate_up", "down"), pools):
        grads[k] = (torch.zeros(p.A_view().shape, device="cuda"),
                    torch.zeros(p.B_view().shape, device="cuda"))
    want = {}
    for seed, T in ((5, 90), (6, 130)):
        _, _, _, ids, x, residual, dy = make(dtype, seed, T, True)
        mlp.forward(x, residual, ids, None, keep=True)
        out = mlp.backward(dy, wt, grads=grads, accumulate=True)
        assert out["gate_up"][0] is grads["gate_up"][0] and out["gate"] is grads["gate"]
        for k, v in reference(w, pools, ids, x, residual, dy, True)[1].items():
            if k != "x":     # (one a batch)
                want[k] = want.get(k, 0) + v
    got = flat(grads)
    for k in got:
        rel = ((got[k].double() - want[k]).norm() / want[k].norm()).item()
        assert rel <= BOUND[dtype], (k, rel)
    slots = [0, 2]
    for pool, k in zip(pools, ("gate_up", "down")):
        pair = grads[k]
        before = [t.clone() for t in pair]
        lst = pool.slot_grads(*pair, slots)
        n = L.lora_clip_grads_workspace_bytes(lst)
        ws, norms = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
        full = [torch.sqrt(sum(t[a].double().square().sum() for t in before)).item()
                for a in slots]
        limit = 0.7 * min(full)
        L.lora_clip_grads(lst, limit, norms, ws, n)
        for g, a in enumerate(slots):
            assert abs(norms[g].item() / full[g] - 1) <= 2.0 ** -22
            for t, b in zip(pair, before):
                f = limit / full[g]
                assert ((t[a].double() - b[a].double() * f).abs() <=
                        2.0 ** -21 * b[a].abs() * f + 1e-37).all()
                assert torch.equal(t[1], b[1])   # a slot outside the list


def test_no_rows_and_no_adapters():
    mlp, w, pools, *_ = make("bf16", 3, 8, False)
    wt = w["down"].t().contiguous()
    empty = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    mlp.forward(empty, empty, np.zeros(0, np.int32), None, keep=True)
    out = mlp.backward(empty, wt)
    assert out["x"].shape == (0, H) and (out["norm_weight"] == 0).all()
    assert all((t == 0).all() for t in out["down"] + out["gate_up"])
    x = torch.randn(5, H, device="cuda").bfloat16()
    mlp.forward(x, x, keep=True)
    out = mlp.backward(x, wt)
    assert set(out) == {"x", "norm_weight"} and out["x"].isfinite().all()
    with pytest.raises(L.LoraError):
        mlp.backward(x, wt)                       # the kept pass is gone


def test_captured_step():
    """Gradients of a kept pass captured once and replayed with new values in place."""
    mlp, w, pools, ids, x, residual, dy = make("bf16", 9, 120, True)
    plan = pools[0].backward_plan(ids)
    n = torch.randn(120, H, device="cuda").bfloat16()
    d = torch.randn(120, 2 * I, device="cuda").bfloat16()
    dn = torch.randn(120, H, device="cuda").bfloat16()
    dx = torch.empty_like(dn)
    dA, dB = (torch.zeros(v.shape, device="cuda") for v in (pools[0].A_view(), pools[0].B_view()))
    lst = pools[0].slot_grads(dA, dB, [0, 1, 2])
    need = L.lora_clip_grads_workspace_bytes(lst)
    ws, norms = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")

    def step():
        pools[0].backward(n, d, plan, dn, dx, dA, dB)
        L.lora_clip_grads(lst, 1.0, norms, ws, need)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pools[0].backward(torch.cat([n] * 9), torch.cat([d] * 9),
                      pools[0].backward_plan(np.tile(ids, 9)))   # outgrows the workspace
    for k in range(3):
        n.normal_()
        d.normal_()
        step()
        want = [t.clone() for t in (dx, dA, dB, norms)]
        for t in (dx, dA, dB, norms):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, dA, dB, norms), want)), k


def test_plans_from_outside_and_a_captured_pass():
    """The block's backward pass with plans made once: eager, and replayed from a graph."""
    mlp, w, pools, ids, x, residual, dy = make("bf16", 12, 150, True)
    wt = w["down"].t().contiguous()
    plans = {k: p.backward_plan(ids) for k, p in zip(("gate_up", "down"), pools)}
    mlp.forward(x, residual, ids, np.ones(150, np.uint8), keep=True)
    kept = mlp._saved, mlp._saved_rest
    want = flat(mlp.backward(dy, wt))

    def step():
        mlp._saved, mlp._saved_rest = kept
        return flat(mlp.backward(dy, wt, plans=plans))

    got = step()
    assert set(got) == set(want) and all(torch.equal(got[k], want[k]) for k in want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp._saved, mlp._saved_rest = kept
        with pytest.raises(L.LoraError):
            mlp.backward(dy, wt)
        out = step()
    for k in range(3):
        dy.normal_()
        want = {name: t.clone() for name, t in step().items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[name], want[name]) for name in want), k
