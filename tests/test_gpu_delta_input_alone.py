"""The input's gradient alone (frozen adapters): the same bits as with the adapters' gradients,
cut reductions and rank blocks among them, and nothing made that those alone take: the
workspace begins with it."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from delta_helpers import batch, run_delta
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,outs,R,slots", [(1, 64, [64], 8, 1), (70, 2056, [520, 8, 136], 40, 3),
                                              (300, 520, [4104], 136, 5), (640, 4096, [72], 16, 2)])
def test_input_alone(dtype, T, K, outs, R, slots):
    ids = np.random.default_rng(T).integers(-1, slots, T)
    ids[0] = 0
    s = batch(T, dtype, ids, K, outs, slots, R)
    full = run_delta(s)
    assert torch.equal(run_delta(s, grads=False)["dx"], full["dx"])
    # (with x not read, what it holds is no matter)
    assert torch.equal(run_delta(dict(s, x=torch.full_like(s["x"], float("nan"))),
                                 grads=False)["dx"], full["dx"])
    desc = L.make_desc(dtype, slots, R, K, outs)
    plan, image = L.lora_delta_backward_plan(desc, ids)
    image = torch.from_numpy(image.copy()).cuda()
    n = L.lora_delta_backward_workspace_bytes(desc, T)
    ws = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(s["x"])
    L.lora_delta_backward(desc, s["A"], s["B"], s["x"], s["dy"], s["dx_in"], dx, None, None, T, plan,
                          image, False, ws, n)
    # u and v of every slice for the rows' tiles of 64, in bf16 three planes of them
    padded = -(-R // 16) * 16 if R <= 32 else -(-R // 64) * 64
    first = 2 * len(outs) * plan.tiles * 64 * padded * (6 if dtype == "bf16" else 4)
    assert torch.equal(dx, full["dx"]) and (ws[:first] == 0xAB).all()
