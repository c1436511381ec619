"""The delta's gradients in 64 bits, adapter by adapter, and how far they may be off.

Bounds: a sum of n products in fp32 is off by at most (n + 4) 2^-23 times the sum of
the terms' magnitudes.  u and v are such sums over out and in features.  dA and dB
pass their errors on and add a sum over the adapter's rows; a bf16 pool's u and v
are three bf16 values there, so that the sum has three times the terms and the value
is right to 2^-24.  In dx they are two values, right to 2^-17; its sum is over the
slices' ranks, twice.  dx_in and an output's rounding come on top."""
import numpy as np
import torch

import lora_adapter_pool_amd as L
from block_helpers import TORCH

UNIT = 2.0 ** -23


def batch(seed, dtype, ids, K, outs, slots, R, integer=False, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    T, O, S = len(ids), sum(outs), len(outs)

    def make(std, *shape):
        if integer:
            return torch.randint(-2, 3, shape, generator=g, device=device).to(TORCH[dtype])
        return (torch.randn(shape, generator=g, device=device) * std).to(TORCH[dtype])

    return {"ids": np.asarray(ids, np.int32), "x": make(1.0, T, K), "dy": make(0.1, T, O),
            "A": make(K ** -0.5, slots, S, R, K), "B": make(0.5, slots, O, R),
            "dx_in": make(1.0, T, K), "outs": list(outs), "dtype": dtype}


def delta64(s):
    """{name: (value, bound)}: dx of the delta alone, dA, dB."""
    x, dy, A, B = (s[k].double() for k in ("x", "dy", "A", "B"))
    n, S, R, K = A.shape
    planes = 3 if s["dtype"] == "bf16" else 1
    ids = torch.from_numpy(s["ids"]).to(x.device)
    zero = lambda t: torch.zeros_like(t)  # noqa: E731
    dx, dA, dB = zero(x), zero(A), zero(B)
    bx, bA, bB = zero(x), zero(A), zero(B)
    ends = np.cumsum([0] + s["outs"])
    for a in sorted(set(s["ids"].tolist()) - {-1}):
        t = torch.nonzero(ids == a)[:, 0]
        rows = len(t)
        for i in range(S):
            cols = slice(int(ends[i]), int(ends[i + 1]))
            d, xa, Aa, Ba = dy[t, cols], x[t], A[a, i], B[a, cols]
            u, v = d @ Ba, xa @ Aa.t()
            eu = (s["outs"][i] + 4) * UNIT * (d.abs() @ Ba.abs())
            ev = (K + 4) * UNIT * (xa.abs() @ Aa.abs().t())
            size = u.abs() @ Aa.abs()
            dx[t] += u @ Aa
            bx[t] += eu @ Aa.abs() + ((2 * S * R + 4) * UNIT + (planes == 3) * 2.0 ** -17) * size
            dA[a, i] = u.t() @ xa
            bA[a, i] = eu.t() @ xa.abs() + (planes * rows + 6) * UNIT * (u.abs().t() @ xa.abs())
            dB[a, cols] = d.t() @ v
            bB[a, cols] = d.abs().t() @ ev + (planes * rows + 6) * UNIT * (d.abs().t() @ v.abs())
    return {"dx": (dx, bx), "dA": (dA, bA), "dB": (dB, bB)}


def run_delta(s, dx_in=True, dx=True, grads=True, start=None, inplace=False, stream=None,
              plan=None):
    """Outputs by name, from buffers that hold NaN; start: a value that the gradients begin
    from (accumulated)."""
    n, S, R, K = s["A"].shape
    T = len(s["ids"])
    desc = L.make_desc(s["dtype"], n, R, K, s["outs"])
    plan, image = plan or L.lora_delta_backward_plan(desc, s["ids"])
    need = L.lora_delta_backward_workspace_bytes(desc, T)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    fill = float("nan") if start is None else start
    new = lambda t: torch.full(t.shape, fill, device="cuda")  # noqa: E731
    base = s["dx_in"] if dx_in else None
    o = {"dx": None if not dx else base if inplace else torch.full_like(s["x"], float("nan")),
         "dA": new(s["A"]) if grads else None, "dB": new(s["B"]) if grads else None}
    L.lora_delta_backward(desc, s["A"], s["B"], s["x"], s["dy"], base if dx else None, o["dx"],
                          o["dA"], o["dB"], T, plan,
                          torch.from_numpy(image.copy()).cuda() if isinstance(image, np.ndarray)
                          else image, start is not None, ws, need, stream=stream)
    return {k: v for k, v in o.items() if v is not None}
