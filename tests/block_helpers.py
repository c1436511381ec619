"""Inputs, 64-bit values and error bounds of the decoder-block operators' tests.

Bounds: a product of K terms in fp32 is off by at most (K + 4) 2^-23 times the
sum of the terms' magnitudes (each addition by half a step of a partial sum
that the magnitudes bound; a whole step is allowed for adders that truncate).
e4m3 operands with bf16 outputs may use gfx950's 8-bit matrix instruction, which
adds neighbouring products on a grid of 2^-11 of the larger one: 2^-10 of the
magnitudes' sum on top.  An activation passes an error on with its steepest slope (below 1.2 for all of
them) and adds 2^-20 of its argument's size for its own exponential, reciprocal
and products.  An output's rounding is half a step, eps / 2 of its value."""
import math

import torch

import lora_adapter_pool_amd as L

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126}


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(TORCH[dtype])


def rows8(t):
    s = (t.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    return (t / s[:, None]).to(torch.float8_e4m3fn), s


def operand(g, rows, K, dtype, std, integer=False):
    if integer:
        t = torch.randint(-2, 3, (rows, K), generator=g, device=g.device).float()
        one = torch.ones(rows, device=g.device) if dtype == "e4m3" else None
        return t.to(TORCH[dtype]), one
    if dtype == "e4m3":
        return rows8(torch.randn((rows, K), generator=g, device=g.device) * std)
    return normal(g, (rows, K), dtype, std), None


def act64(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "relu":
        return z.clamp(min=0)
    return z


def slope64(name, z):
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).double()
    return torch.ones_like(z)


def product64(x, w, xs=None, ws=None):
    """The product in 64 bits and the sum of its terms' magnitudes."""
    a, b = x.double(), w.double()
    z, mag = a @ b.t(), a.abs() @ b.abs().t()
    if xs is not None:
        s = xs.double()[:, None] * ws.double()
        z, mag = z * s, mag * s
    return z, mag


def product_bound(K, mag, coarse=False):
    return ((K + 4) * 2.0 ** -23 + 2.0 ** -10 * coarse) * mag


def within(got, want, bound, dtype, label):
    """got is rounded to dtype: half a step of what the bound allows."""
    b = bound + HALF_STEP[dtype] * (want.abs() + bound) + TINY[dtype]
    err = (got.double() - want).abs()
    bad = ~(err <= b)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / b, torch.zeros_like(err))))
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: "
                             f"{got.flatten()[i]} for {want.flatten()[i]}, "
                             f"allowed {b.flatten()[i]}")


def run_linear(x, w, xs, ws_, bias, delta, residual, dtype, od, act, out=None, stream=None):
    T, K, O = x.shape[0], x.shape[1], w.shape[0]
    d = L.make_linear_desc(dtype, od, K, O, act)
    n = L.lora_linear_workspace_bytes(d, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    if out is None:
        out = torch.full((T, O), float("nan"), dtype=TORCH[od], device="cuda")
    L.lora_linear(d, x, w, xs, ws_, bias, delta, residual, out, T, ws, n, stream=stream)
    return out


def run_gated(x, w, xs, ws_, delta, keep, dtype, od, act, stream=None):
    T, K, I = x.shape[0], x.shape[1], w.shape[0] // 2
    d = L.make_gated_desc(dtype, od, K, I, act)
    n = L.lora_gated_ffn_workspace_bytes(d, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full((T, I), float("nan"), dtype=TORCH[od], device="cuda")
    pre = torch.full((T, 2 * I), float("nan"), dtype=TORCH[od], device="cuda") if keep else None
    L.lora_gated_ffn(d, x, w, xs, ws_, delta, pre, out, T, ws, n, stream=stream)
    return out, pre


def run_backward(dout, pre, x, w, act, dtype, dx=True, dw=True, dpre=None):
    T, K, I = x.shape[0], x.shape[1], w.shape[0] // 2
    d = L.make_gated_desc(dtype, dtype, K, I, act)
    n = L.lora_gated_ffn_backward_workspace_bytes(d, T, dx, dw)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    nan = lambda *s: torch.full(s, float("nan"), dtype=TORCH[dtype], device="cuda")  # noqa: E731
    dpre = nan(T, 2 * I) if dpre is None else dpre
    gx, gw = nan(T, K) if dx else None, nan(2 * I, K) if dw else None
    L.lora_gated_ffn_backward(d, dout, pre, x, w, dpre, gx, gw, T, ws, n)
    return dpre, gx, gw
