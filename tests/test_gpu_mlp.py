"""The feed-forward path (LoraMlp): the same as its operators one by one, near a
plain implementation in 64 bits, and the example that runs it."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import TORCH, act64, gen, normal, run_backward, run_gated, run_linear, slope64
from gpu_helpers import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def _pool(g, dtype, K, outs, rank=8, slots=3):
    pool = L.LoraPool(dtype, slots, rank, K, outs)
    for slot in range(slots):
        for s, o in enumerate(outs):
            pool.load(slot, s, normal(g, (rank, K), dtype, K ** -0.5),
                      normal(g, (o, rank), dtype, 0.2), rank, float(rank))
    return pool


def _delta64(pool, x, ids):
    A, B = pool.A_view().double(), pool.B_view().double()
    out = torch.zeros((x.shape[0], pool.O), dtype=torch.float64, device="cuda")
    for i, slot in enumerate(ids):
        if slot >= 0:
            c = 0
            for s, o in enumerate(pool.out_features):
                out[i, c:c + o] = B[slot, c:c + o] @ (A[slot, s] @ x[i])
                c += o
    return out


def _setup(seed, dtype, T, H, I):
    g = gen(seed)
    w = dict(norm_weight=(1 + 0.1 * normal(g, (H,), "f32")).to(TORCH[dtype]),
             w_gate_up=normal(g, (2 * I, H), dtype, H ** -0.5),
             w_down=normal(g, (H, I), dtype, I ** -0.5))
    pools = dict(gate_up=_pool(g, dtype, H, [I, I]), down=_pool(g, dtype, I, [H]))
    ids = np.random.default_rng(seed).integers(-1, 3, T).astype(np.int32)
    prefill = (np.arange(T) % 2).astype(np.uint8)
    return w, pools, normal(g, (T, H), dtype), normal(g, (T, H), dtype), ids, prefill


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 150])
def test_path_matches_operators_and_64_bits(dtype, T):
    H, I = 264, 520
    w, pools, x, r, ids, prefill = _setup(T, dtype, T, H, I)
    mlp = L.LoraMlp(**w, **pools)
    y = mlp.forward(x, r, ids, prefill, keep=True)
    # one by one
    s, n = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rms_norm(L.make_norm_desc(dtype, H, 1e-5), x, r, w["norm_weight"], s, n, None, None, T)
    d = torch.zeros((T, 2 * I), dtype=x.dtype, device="cuda")
    pools["gate_up"].apply(n, d, ids, prefill)
    h, pre = run_gated(n, w["w_gate_up"], None, None, d, True, dtype, dtype, "silu")
    d2 = torch.zeros((T, H), dtype=x.dtype, device="cuda")
    pools["down"].apply(h, d2, ids, prefill)
    want = run_linear(h, w["w_down"], None, None, None, d2, s, dtype, dtype, "none")
    assert torch.equal(y, want)
    dh = normal(gen(9), (T, I), dtype, 0.1)
    got = mlp.gate_up_backward(dh)
    for a, b in zip(got, run_backward(dh, pre, n, w["w_gate_up"], "silu", dtype)):
        assert torch.equal(a, b)
    # in 64 bits: six stored roundings (n, two deltas, h, s, y), each within half
    # a step of its values, passed on with the activation's slope and the other
    # factor (below 2 together)
    s64 = (x.double() + r.double())
    n64 = s64 * torch.rsqrt(s64.square().mean(1, keepdim=True) + 1e-5) * w["norm_weight"].double()
    z = n64 @ w["w_gate_up"].double().t() + _delta64(pools["gate_up"], n64, ids)
    h64 = act64("silu", z[:, :I]) * z[:, I:]
    y64 = h64 @ w["w_down"].double().t() + _delta64(pools["down"], h64, ids) + s64
    half = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    sums = {"bf16": 0.0, "f32": 2.0 ** -20}[dtype]   # fp32 sums of 520 terms, twice
    assert (y.double() - y64).norm() <= (6 * 2 * half + sums) * y64.norm()
    gate, up, d64 = pre[:, :I].double(), pre[:, I:].double(), dh.double()
    dz = torch.cat([d64 * up * slope64("silu", gate), d64 * act64("silu", gate)], 1)
    dn = dz @ w["w_gate_up"].double()
    assert (got[1].double() - dn).norm() <= (2 * 2 * half + sums) * dn.norm()


def test_eight_bit_gate_up():
    T, H, I = 70, 272, 528
    w, pools, x, r, ids, prefill = _setup(3, "bf16", T, H, I)
    scale = (w["w_gate_up"].float().abs().amax(1) / 448).clamp_min(2.0 ** -126)
    w8 = (w["w_gate_up"].float() / scale[:, None]).to(torch.float8_e4m3fn)
    y = L.LoraMlp(w["norm_weight"], w8, w["w_down"], gate_up_scale=scale, **pools).forward(
        x, r, ids, prefill)
    # the same weights' values in bf16 (e4m3 values times a scale round again)
    wb = (w8.float() * scale[:, None]).bfloat16()
    want = L.LoraMlp(w["norm_weight"], wb, w["w_down"], **pools).forward(x, r, ids, prefill)
    # the activations' rounding to 8 bits, half a step 2^-4 at most of every
    # value, and two factors of it in h
    assert (y.float() - want.float()).norm() <= 2 * 2.0 ** -4 * want.float().norm()


def test_no_adapters_and_empty_batch():
    w, pools, x, r, ids, prefill = _setup(4, "bf16", 9, 64, 72)
    a = L.LoraMlp(**w, **pools).forward(x, r)
    b = L.LoraMlp(**w).forward(x, r, ids, prefill)
    none = L.LoraMlp(**w, **pools).forward(x, r, np.full(9, -1, np.int32), prefill)
    assert torch.equal(a, b) and torch.equal(a, none)
    assert L.LoraMlp(**w, **pools).forward(x[:0], r[:0], ids[:0], prefill[:0]).shape == (0, 64)


def test_example_runs():
    p = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "mlp_block.py"), "--hidden",
                        "256", "--inter", "512", "--rows", "40"], capture_output=True, text=True,
                       timeout=100)
    assert p.returncode == 0, p.stderr
    assert "relative difference" in p.stdout
