"""The activations and their slopes over the whole range of finite gates, through
every kernel that ends in them, against 64-bit values.

The operands are zeros and the gates come in as the delta, so a gate reaches the
curve as it is.  Bounds: with a(z) the size of the exponent's argument (|z| for
SiLU, z^2 / 2 for GELU, |2 u| for its tanh form), the factor beside z is off by
2^-19 (1 + a) of itself (exponent, exponential, reciprocal or erfc, products), or
by 2^-126 where it is flushed to zero; a slope by 2^-20 (1.2 + |z|), the bound of
the block's other tests.  Rounding to the output's type is half a step more."""
import math

import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import HALF_STEP, TORCH, act64, run_backward, run_gated, run_linear, slope64
from gpu_helpers import say

pytestmark = pytest.mark.gpu
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def _gates(dtype, rows, unit):
    """-130 to 130 in steps of 1/16 and -12 to 12 in steps of 1/512, as a matrix
    of `rows` rows and a multiple of `unit` columns (filled up with zeros)."""
    z = torch.cat([torch.arange(-130 * 16, 130 * 16 + 1, device="cuda") / 16.0,
                   torch.arange(-12 * 512, 12 * 512 + 1, device="cuda") / 512.0])
    cols = (-(-z.numel() // rows) + unit - 1) // unit * unit
    out = torch.zeros(rows * cols, device="cuda")
    out[:z.numel()] = z
    return out.view(rows, cols).to(TORCH[dtype])


def _check_value(got, z, act, dtype, label):
    z = z.double()
    want = act64(act, z)
    a = {"silu": z.abs(), "gelu": z * z / 2,
         "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3).abs()}.get(act, 0 * z)
    slack = 0 * z if act in ("none", "relu") else 2.0 ** -19 * (1 + a) * want.abs() + \
        z.abs() * 2.0 ** -126
    _within(got, want, slack, z, dtype, label)


def _check_slope(got, z, act, dtype, label):
    z = z.double()
    slack = 0 * z if act in ("none", "relu") else 2.0 ** -20 * (1.2 + z.abs())
    _within(got, slope64(act, z), slack, z, dtype, label)


def _within(got, want, slack, z, dtype, label):
    assert torch.isfinite(got).all(), (label, "not finite at", z[~torch.isfinite(got)][:8].tolist())
    b = slack + HALF_STEP[dtype] * (want.abs() + slack) + 2.0 ** -126
    bad = (got.double() - want).abs() > b
    assert not bad.any(), (label, z[bad][:8].tolist(), got[bad][:8].tolist(), want[bad][:8].tolist())


# a K split, the few-row kernel, and each tile shape's own epilogue
PLANS = [("4,1", 20), ("0,1", 40), ("1,1", 70), ("1,2", 70), ("2,1", 130), ("3,1", 260), ("3,2", 260)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,od", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"),
                                      ("e4m3", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("plan,T", PLANS)
def test_forward_curves(dtype, od, act, plan, T, monkeypatch):
    monkeypatch.setenv("LORA_GEMM_PLAN", plan)
    K = 512
    z = _gates(od, T, 16)
    N = z.shape[1]
    x = torch.zeros((T, K), device="cuda").to(TORCH[dtype])
    w = torch.zeros((2 * N, K), device="cuda").to(TORCH[dtype])
    xs = torch.ones(T, device="cuda") if dtype == "e4m3" else None
    ws = torch.ones(2 * N, device="cuda") if dtype == "e4m3" else None
    got = run_linear(x, w[:N], xs, None if ws is None else ws[:N], None, z, None, dtype, od, act)
    _check_value(got, z, act, od, f"linear {dtype}->{od} {act} {plan}")
    got, _ = run_gated(x, w, xs, ws, torch.cat([z, torch.ones_like(z)], 1), False, dtype, od, act)
    _check_value(got, z, act, od, f"gated {dtype}->{od} {act} {plan}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_curves(dtype, act):
    z = _gates(dtype, 37, 8)
    T, I = z.shape
    K = 64
    one = torch.ones_like(z)
    x = torch.ones((T, K), dtype=TORCH[dtype], device="cuda")
    w = torch.zeros((2 * I, K), dtype=TORCH[dtype], device="cuda")
    dpre, dx, dw = run_backward(one, torch.cat([z, one], 1), x, w, act, dtype)
    _check_slope(dpre[:, :I], z, act, dtype, f"slope {dtype} {act}")
    _check_value(dpre[:, I:], z, act, dtype, f"value {dtype} {act}")
    assert torch.equal(dx, torch.zeros_like(dx))
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_path_of_fp32_layer_stays_finite(act):
    """An fp32 LoraMlp whose gates reach far below zero: the down product and the
    gradients of the block would carry one NaN into whole rows."""
    H, I, T = 64, 128, 9
    g = torch.Generator(device="cuda").manual_seed(5)
    w_gu = torch.randn((2 * I, H), generator=g, device="cuda")
    mlp = L.LoraMlp(torch.ones(H, device="cuda"), w_gu * 4, torch.randn((H, I), generator=g,
                    device="cuda") * I ** -0.5, act=act)
    x = torch.randn((T, H), generator=g, device="cuda")
    y = mlp.forward(x, torch.zeros_like(x), keep=True)
    assert torch.isfinite(y).all()
    for t in mlp.gate_up_backward(torch.ones((T, I), device="cuda")):
        assert torch.isfinite(t).all()
