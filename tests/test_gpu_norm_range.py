"""Norm over the whole range of finite rows, against 64-bit values: also where the
factor of a row, (mean(t^2) + eps)^(-1/2), is past fp32's range or below its normal
numbers.  Bounds as in the norm's other tests: a few roundings to fp32, and the
output's."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import HALF_STEP, TORCH, gen
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [64, 1032, 8200])
def test_rows_of_any_size(dtype, H):
    say(f"[gpu] test_rows_of_any_size {dtype} {H}")
    g = gen(H)
    sizes = [2.0 ** -148, 2.0 ** -140, 2.0 ** -130, 2.0 ** -126, 2.0 ** -120, 2.0 ** -99, 1.0,
             2.0 ** 70, 2.0 ** 101, 2.0 ** 120, 2.0 ** 126]
    if dtype == "bf16":
        sizes[:2] = [2.0 ** -133, 2.0 ** -132]
    T = len(sizes)
    # whole multiples of the size, so that they are numbers of the type down there
    k = torch.randint(1, 4, (T, H), generator=g, device="cuda").double()
    sign = torch.randint(0, 2, (T, H), generator=g, device="cuda").double() * 2 - 1
    x = (k * sign * torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None]).to(TORCH[dtype])
    assert torch.isfinite(x).all() and (x != 0).all()
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(TORCH[dtype])
    out, out8 = torch.empty_like(x), torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(T, device="cuda")
    L.lora_add_rms_norm(L.make_norm_desc(dtype, H, 0.0), x, None, w, None, out, out8, scale, T)
    t = x.double()
    n = t / t.square().mean(1, keepdim=True).sqrt() * w.double()
    slack = 4 * 2.0 ** -24
    for i, size in enumerate(sizes):
        ok = (out[i].double() - n[i]).abs() <= (HALF_STEP[dtype] + slack) * n[i].abs()
        assert ok.all(), (size, out[i][~ok][:4].tolist(), n[i][~ok][:4].tolist())
        top = n[i].abs().max() / 448
        assert abs(scale[i].double() - top) <= (slack + 2.0 ** -24) * top, size
        v = out8[i].double() * scale[i].double()
        assert ((v - n[i]).abs() <= torch.maximum(HALF_STEP["e4m3"] * n[i].abs() * (1 + 2.0 ** -18),
                                                  scale[i].double() * 2.0 ** -10) +
                8 * 2.0 ** -24 * n[i].abs()).all(), size
