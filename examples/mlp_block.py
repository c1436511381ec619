"""The feed-forward half of a decoder layer with adapters, on one GPU: a mixed
batch of prefill and decode rows through norm, gate/up, activation and down, each
row with its own adapter or none; then the gate/up gradients of the same pass;
then one training step's gradients of the adapters, clipped slot by slot; then the
same layer with its gate/up weights in 8 bits.

    python examples/mlp_block.py [--hidden 1024 --inter 2816 --rows 300]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lora_adapter_pool_amd as L  # noqa: E402


def pool_with_adapters(g, K, outs, slots=4, rank=16):
    pool = L.LoraPool("bf16", slots, rank, K, outs)
    for slot in range(slots):
        for s, o in enumerate(outs):
            A = (torch.randn(rank, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
            B = (torch.randn(o, rank, generator=g, device="cuda") * 0.1).bfloat16()
            pool.load(slot, s, A, B, rank, alpha=float(rank))
    return pool


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=2816)
    ap.add_argument("--rows", type=int, default=300)
    a = ap.parse_args()
    H, I, T = a.hidden, a.inter, a.rows
    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w_gate_up, w_down = (normal(2 * I, H) * H ** -0.5).bfloat16(), (normal(H, I) * I ** -0.5).bfloat16()
    weight = (1 + 0.1 * normal(H)).bfloat16()
    gate_up, down = pool_with_adapters(g, H, [I, I]), pool_with_adapters(g, I, [H])
    x, residual = normal(T, H).bfloat16(), normal(T, H).bfloat16()
    ids = np.random.default_rng(0).integers(-1, 4, T).astype(np.int32)
    prefill = (np.arange(T) < T // 2).astype(np.uint8)

    mlp = L.LoraMlp(weight, w_gate_up, w_down, gate_up=gate_up, down=down)
    y = mlp.forward(x, residual, ids, prefill, keep=True)
    dpre, dn, dw = mlp.gate_up_backward((normal(T, I) * 0.1).bfloat16())
    print("y", tuple(y.shape), "dn", tuple(dn.shape), "dW", tuple(dw.shape))

    dy, w_down_t = (normal(T, H) * 0.1).bfloat16(), w_down.t().contiguous()
    out = mlp.backward(dy, w_down_t)
    for name, pool in (("gate_up", gate_up), ("down", down)):
        grads = pool.slot_grads(*out[name], range(pool.max_loras))
        need = L.lora_clip_grads_workspace_bytes(grads)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        norms = torch.empty(pool.max_loras, device="cuda")
        L.lora_clip_grads(grads, 1.0, norms, ws, need)
        print(f"{name}: gradient norms of the slots before clipping to 1", norms.tolist())
    print("dx", tuple(out["x"].shape), "dnorm", tuple(out["norm_weight"].shape))

    scale = (w_gate_up.float().abs().amax(1) / 448).clamp_min(2.0 ** -126)
    w8 = (w_gate_up.float() / scale[:, None]).to(torch.float8_e4m3fn)
    y8 = L.LoraMlp(weight, w8, w_down, gate_up_scale=scale, gate_up=gate_up,
                   down=down).forward(x, residual, ids, prefill)
    rel = ((y8.float() - y.float()).norm() / y.float().norm()).item()
    print(f"gate/up weights and activations in 8 bits: relative difference {rel:.2e}")


if __name__ == "__main__":
    main()
