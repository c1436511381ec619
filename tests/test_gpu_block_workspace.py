"""One workspace, sized for the largest batch, for every smaller batch: the same
results as with a workspace of the batch's own, and nothing written past it."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import TORCH, gen, normal, run_backward, run_gated, run_linear
from gpu_helpers import say

pytestmark = pytest.mark.gpu
MOST = 4096


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,I", [(1024, 512), (264, 1032), (4096, 256)])
def test_one_workspace_for_all_batches(dtype, K, I):
    d = L.make_linear_desc(dtype, dtype, K, I)
    gd = L.make_gated_desc(dtype, dtype, K, I)
    need = max(L.lora_linear_workspace_bytes(d, MOST), L.lora_gated_ffn_workspace_bytes(gd, MOST),
               L.lora_gated_ffn_backward_workspace_bytes(gd, MOST))
    buf = torch.full((need + 4096,), 90, dtype=torch.uint8, device="cuda")
    ws = buf[:need]
    g = gen(K + I)
    w = normal(g, (2 * I, K), dtype, K ** -0.5)
    for T in (1, 8, 33, 64, 65, 129, 200, 300, 512, 1000, MOST):
        x, dout = normal(g, (T, K), dtype), normal(g, (T, I), dtype, 0.1)
        new = lambda *s: torch.full(s, float("nan"), dtype=TORCH[dtype], device="cuda")  # noqa: E731
        out, h, pre = new(T, I), new(T, I), new(T, 2 * I)
        dpre, dx, dw = new(T, 2 * I), new(T, K), new(2 * I, K)
        L.lora_linear(d, x, w[:I], None, None, None, None, None, out, T, ws, need)
        L.lora_gated_ffn(gd, x, w, None, None, None, pre, h, T, ws, need)
        L.lora_gated_ffn_backward(gd, dout, pre, x, w, dpre, dx, dw, T, ws, need)
        assert torch.equal(out, run_linear(x, w[:I], None, None, None, None, None, dtype, dtype,
                                           "none"))
        assert torch.equal(h, run_gated(x, w, None, None, None, False, dtype, dtype, "silu")[0])
        for a, b in zip((dpre, dx, dw), run_backward(dout, pre, x, w, "silu", dtype)):
            assert torch.equal(a, b), (T, K, I)
        # one gradient alone takes the same buffer
        L.lora_gated_ffn_backward(gd, dout, pre, x, None, dpre, None, dw.fill_(float("nan")), T, ws,
                                  need)
        assert torch.equal(dw, run_backward(dout, pre, x, w, "silu", dtype, dx=False)[2])
        assert (buf[need:] == 90).all(), T


def test_a_captured_forward_outlives_a_larger_call():
    """A graph of a small batch, then an eager call of a larger one, whose
    workspace is larger: the graph's replays are still right, and write into
    nobody else's memory."""
    H, I, T = 2048, 512, 8
    g = gen(21)
    w = [normal(g, (H,), "bf16"), normal(g, (2 * I, H), "bf16", H ** -0.5),
         normal(g, (H, I), "bf16", I ** -0.5)]
    mlp = L.LoraMlp(*w)
    x, r = normal(g, (T, H), "bf16"), normal(g, (T, H), "bf16")
    mlp.forward(x, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mlp.forward(x, r)
    before = mlp._ws.numel()
    xl = normal(g, (600, H), "bf16")
    mlp.forward(xl, torch.zeros_like(xl))
    assert mlp._ws.numel() > before
    # takes what the allocator has to give back of the old workspace's size
    others = [torch.full((before,), 85, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for k in range(4):
        x.copy_(normal(g, (T, H), "bf16"))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, L.LoraMlp(*w).forward(x, r)), k
        assert all((t == 85).all() for t in others), k
