"""lora_block_norm and its gradients in 64 bits, from the formulas, and how far
fp32 arithmetic may be from them.

Bounds, with e = 2^-24 (half a step of fp32): a norm's factor is right to e, and
each product or sum that follows adds e of its own result.  A branch beta g p is
off by at most 8 e of itself, the sum by that and 3 e of its terms.  In a norm's
gradient r (w - hat c) the terms w, hat and c carry 4 e each, so that it is off by at
most 16 e of r (|w| + |hat| <|w hat|>).  What comes in with an error passes it on
through the same formula.  A sum over T rows in fp32, in any order, adds T e of its
terms' magnitudes; an output's rounding half a step."""
import torch

import lora_adapter_pool_amd as L
from block_helpers import TORCH

E = 2.0 ** -24


def norm64(t, w, eps):
    return t * (t.square().mean(1, keepdim=True) + eps).rsqrt() * w


def join64(y, residual, gate, post, alpha, beta, eps):
    """The stream before it is rounded, and its bound."""
    p = y if post is None else norm64(y, post, eps)
    b = beta * (p if gate is None else p * gate)
    r = alpha * residual
    return r + b, 8 * E * b.abs() + 3 * E * (r.abs() + b.abs())


def norm_grad64(x, w, d, eps, err):
    """d (rms_norm(x) w) / dx applied to d, which is off by err; the weight's
    gradient; and both bounds."""
    r = (x.square().mean(1, keepdim=True) + eps).rsqrt()
    hat, v, e = x * r, d * w, err * w.abs()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    out = r * (v - hat * mean(v * hat))
    size = r * (v.abs() + hat.abs() * mean((v * hat).abs()))
    bound = 16 * E * size + r * (e + hat.abs() * mean(e * hat.abs()))
    rows = x.shape[0]
    dw = d * hat
    dw_bound = ((rows + 8) * E * dw.abs() + err * hat.abs()).sum(0)
    return out, bound, dw.sum(0), dw_bound


def join_grad64(dout, dsum, y, t, gate, post, pre, alpha, beta, eps):
    """{name: (value, bound)} of the gradients; gate [H] or [T][H] or None."""
    got = {}
    d, err = torch.zeros_like(y), torch.zeros_like(y)
    if dout is not None:
        d, err, dw, b = norm_grad64(t, pre, dout, eps, torch.zeros_like(y))
        got["dpre"] = (dw, b)
    if dsum is not None:
        d = d + dsum
        err = err + 2 * E * (d.abs() + dsum.abs())
    got["dresidual"] = (alpha * d, abs(alpha) * err + E * (alpha * d).abs())
    p = y if post is None else norm64(y, post, eps)
    d, err = beta * d, abs(beta) * err + E * (beta * d).abs()
    if gate is not None:
        dg, b = d * p, err * p.abs() + 8 * E * (d * p).abs()
        if gate.dim() == 1:
            dg, b = dg.sum(0), (b + (y.shape[0] + 8) * E * dg.abs()).sum(0)
        got["dgate"] = (dg, b)
        d, err = d * gate, err * gate.abs() + E * (d * gate).abs()
    if post is not None:
        d, err, dw, b = norm_grad64(y, post, d, eps, err)
        got["dpost"] = (dw, b)
    got["dy"] = (d, err)
    return got


def inputs(seed, T, H, dtype, gate="none", device="cuda", gain=1.0):
    g = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    wide = torch.exp(n(H)) * gain
    s = {"y": n(T, H) * wide, "residual": 2 * n(T, H) * wide, "post": 1 + 0.2 * n(H),
         "pre": 1 + 0.2 * n(H), "dout": 0.1 * n(T, H), "dsum": 0.1 * n(T, H),
         "sum": 2 * n(T, H) * wide}
    s["gate"] = None if gate == "none" else n(H) if gate == "channel" else n(T, H)
    return {k: None if v is None else v.to(TORCH[dtype]) for k, v in s.items()}


def run_join(s, dtype, gate, alpha=1.0, beta=1.0, eps=1e-5, post=True, pre=True, out=True,
             out8=True, stream=None, inplace=False):
    T, H = s["y"].shape
    d = L.make_block_norm_desc(dtype, H, eps, gate, alpha, beta)
    nan = lambda: torch.full_like(s["y"], float("nan"))  # noqa: E731
    total = s["residual"] if inplace else nan()
    o = (s["y"] if inplace else nan()) if pre and out else None
    o8 = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda") if pre and out8 else None
    sc = torch.full((T,), float("nan"), device="cuda") if pre and out8 else None
    L.lora_block_norm(d, s["y"], s["residual"], s["gate"], s["post"] if post else None,
                      s["pre"] if pre else None, total, o, o8, sc, T, stream=stream)
    return total, o, o8, sc


def run_join_backward(s, dtype, gate, alpha=1.0, beta=1.0, eps=1e-5, post=True, pre=True,
                      stream_grad=True, sums=True, start=None, inplace=False, stream=None):
    """Outputs by name; start: a value that the fp32 sums begin from (accumulated)."""
    T, H = s["y"].shape
    d = L.make_block_norm_desc(dtype, H, eps, gate, alpha, beta)
    n = L.lora_block_norm_backward_workspace_bytes(d, T)
    ws = torch.full((max(n, 16),), 0xAB, dtype=torch.uint8, device="cuda")
    new = lambda: torch.full_like(s["y"], float("nan"))  # noqa: E731
    row = lambda: torch.full((H,), float("nan") if start is None else start,  # noqa: E731
                             device="cuda")
    o = {"dy": s["y"] if inplace else new(), "dresidual": s["dsum"] if inplace else new(),
         "dgate": None if gate == "none" else row() if gate == "channel" else
         (s["gate"] if inplace else new()),
         "dpost": row() if post and sums else None, "dpre": row() if pre and sums else None}
    L.lora_block_norm_backward(
        d, s["dout"] if pre else None, s["dsum"] if stream_grad else None,
        s["y"] if post or gate != "none" else None, s["sum"] if pre else None, s["gate"],
        s["post"] if post else None, s["pre"] if pre else None, o["dy"], o["dresidual"],
        o["dgate"], o["dpost"], o["dpre"], start is not None, T, ws, n, stream=stream)
    return {k: v for k, v in o.items() if v is not None}
