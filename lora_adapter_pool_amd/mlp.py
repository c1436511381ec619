"""The feed-forward half of a decoder layer with adapters, as one path.

    s = x + residual                          (the residual stream)
    n = rms_norm(s) * norm_weight             (and, for 8-bit weights, n in e4m3)
    h = act(n Wg^T + dg) * (n Wu^T + du)      dg, du: the adapters' gate/up delta
    y = h Wd^T + dd + s                       dd: the adapters' down delta
or, in models with a norm after the block, a gate or scales of the two branches,
    y = residual_scale s + block_scale gate rms_norm(h Wd^T + dd) post_norm_weight

Every row names its adapter slot in each pool, or none (-1).  The adapters'
deltas are LoraPool.apply onto zeros; they join the base products before the
activation, inside the products' epilogues.  LoraMlp owns the descriptors and
one workspace; weights and pools belong to the caller.  Calls run on the current
stream of the weights' GPU, whichever GPU is the current one, and those of one
LoraMlp share its workspace: use one per stream.

A call that needs a larger workspace gets a new one, and the old one is kept as
long as the LoraMlp: a graph that was captured before holds its address.  Keep
the LoraMlp, then, as long as the graphs that its calls were captured in.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from . import _lib as L
from .pool import LoraPool


class LoraMlp:
    """norm_weight [H], w_gate_up [2 I][H] (gate rows, then up rows), w_down
    [H][I], all of the activations' dtype (fp32 or bf16); or w_gate_up in e4m3
    with one fp32 scale a row in gate_up_scale, for bf16 activations.  gate_up
    and down: pools of the activations' dtype with slices [I, I] and [H].
    post_norm_weight, gate [H] (of the activations' dtype), residual_scale,
    block_scale: of the second form of y; post_norm_weight and gate may be None."""

    def __init__(self, norm_weight, w_gate_up, w_down, eps: float = 1e-5, act: str = "silu",
                 gate_up_scale=None, gate_up: Optional[LoraPool] = None,
                 down: Optional[LoraPool] = None, post_norm_weight=None, gate=None,
                 residual_scale: float = 1.0, block_scale: float = 1.0):
        import torch

        self.torch = torch
        self.dtype = {torch.float32: "f32", torch.bfloat16: "bf16"}.get(w_down.dtype)
        if self.dtype is None or norm_weight.dtype != w_down.dtype:
            raise L.LoraError(L.LORA_E_DTYPE, "norm_weight and w_down must both be fp32 or bf16")
        self.eight = w_gate_up.dtype == torch.float8_e4m3fn
        if self.eight != (gate_up_scale is not None) or (self.eight and self.dtype != "bf16"):
            raise L.LoraError(L.LORA_E_DTYPE,
                              "an e4m3 w_gate_up needs gate_up_scale and bf16 activations")
        if not self.eight and w_gate_up.dtype != w_down.dtype:
            raise L.LoraError(L.LORA_E_DTYPE, "w_gate_up must be e4m3 or of w_down's dtype")
        if w_down.dim() != 2:
            raise L.LoraError(L.LORA_E_SHAPE, "w_down must be [H, I]")
        self.H, self.I = int(w_down.shape[0]), int(w_down.shape[1])
        if tuple(w_gate_up.shape) != (2 * self.I, self.H) or tuple(norm_weight.shape) != (self.H,):
            raise L.LoraError(L.LORA_E_SHAPE, "w_gate_up must be [2 I, H] and norm_weight [H]")
        if self.eight and (tuple(gate_up_scale.shape) != (2 * self.I,) or
                           gate_up_scale.dtype != torch.float32):
            raise L.LoraError(L.LORA_E_SHAPE, "gate_up_scale must be fp32 [2 I]")
        for pool, K, outs in ((gate_up, self.H, [self.I, self.I]), (down, self.I, [self.H])):
            if pool is not None and (pool.K != K or pool.out_features != outs or
                                     pool.dtype != self.dtype):
                raise L.LoraError(L.LORA_E_SHAPE, "a pool does not fit the block")
            if pool is not None and pool.A.device != w_down.device:
                raise L.LoraError(L.LORA_E_ARG, "a pool is not on the weights' device")
        for t in (post_norm_weight, gate):
            if t is not None and t.dtype != w_down.dtype:
                raise L.LoraError(L.LORA_E_DTYPE, "post_norm_weight and gate have w_down's dtype")
            if t is not None and tuple(t.shape) != (self.H,):
                raise L.LoraError(L.LORA_E_SHAPE, "post_norm_weight and gate must be [H]")
        for t in (norm_weight, w_gate_up, w_down, gate_up_scale, post_norm_weight, gate):
            if t is not None and not t.is_contiguous():
                raise L.LoraError(L.LORA_E_SHAPE, "weights must be contiguous")
            if t is not None and t.device != w_down.device:
                raise L.LoraError(L.LORA_E_ARG, "weights must be on one device")
        self.norm_weight, self.w_gate_up, self.w_down = norm_weight, w_gate_up, w_down
        self.gate_up_scale, self.gate_up, self.down = gate_up_scale, gate_up, down
        self.norm_desc = L.make_norm_desc(self.dtype, self.H, eps)
        self.gated_desc = L.make_gated_desc("e4m3" if self.eight else self.dtype, self.dtype,
                                            self.H, self.I, act)
        self.grad_desc = L.make_gated_desc(self.dtype, self.dtype, self.H, self.I, act)
        self.down_desc = L.make_linear_desc(self.dtype, self.dtype, self.I, self.H)
        self.post_norm_weight, self.gate = post_norm_weight, gate
        self.norm_grad_desc = L.make_block_norm_desc(self.dtype, self.H, eps)
        self.join_desc = None
        if post_norm_weight is not None or gate is not None or residual_scale != 1.0 or \
                block_scale != 1.0:
            self.join_desc = L.make_block_norm_desc(
                self.dtype, self.H, eps, "none" if gate is None else "channel", residual_scale,
                block_scale)
        self.dh_desc = L.make_linear_desc(self.dtype, self.dtype, self.H, self.I)
        self._ws = None
        self._outgrown = []
        self._saved = None
        self._saved_rest = None

    def _workspace(self, need: int):
        have = 0 if self._ws is None else self._ws.numel()
        if have < max(need, 1):
            if have:
                self._outgrown.append(self._ws)
            # at least twice as large: the outgrown ones add up to no more than the last
            self._ws = self.torch.empty(max(need, 2 * have, 256), dtype=self.torch.uint8,
                                        device=self.w_down.device)
        return self._ws

    def _check_device(self):
        if not self.w_down.is_cuda:
            raise L.LoraError(L.LORA_E_ARG, "the block's weights are not on a GPU")

    def _on_device(self, call, *args):
        """call(*args) with the weights' GPU as the current one (launches go to the
        current GPU's stream)."""
        if self.torch.cuda.current_device() == self.w_down.device.index:
            return call(*args)
        with self.torch.cuda.device(self.w_down.device):
            return call(*args)

    def _check_rows(self, t, width: int, name: str):
        if t.dtype != self.w_down.dtype or t.device != self.w_down.device:
            raise L.LoraError(L.LORA_E_DTYPE, f"{name} must have the weights' dtype and device")
        if t.dim() != 2 or t.shape[1] != width or not t.is_contiguous():
            raise L.LoraError(L.LORA_E_SHAPE, f"{name} must be a contiguous [T, {width}]")

    def forward(self, x, residual, ids=None, prefill=None, keep=False):
        """y [T][H] on the current stream of the weights' GPU.  ids, prefill: as
        LoraPool.apply takes them (None: no adapters).  keep: True holds what
        gate_up_backward and backward need, "gate_up" what gate_up_backward alone needs
        (T H values fewer, and T I fewer where down has adapters, T H fewer behind a norm
        after the block or a gate)."""
        if isinstance(keep, str) and keep != "gate_up":
            raise L.LoraError(L.LORA_E_ARG, f'keep must be True, False or "gate_up", got {keep!r}')
        self._check_rows(x, self.H, "x")
        self._check_rows(residual, self.H, "residual")
        if residual.shape != x.shape:
            raise L.LoraError(L.LORA_E_SHAPE, "x and residual must have the same shape")
        self._check_device()
        return self._on_device(self._forward, x, residual, ids, prefill, keep)

    def _forward(self, x, residual, ids, prefill, keep):
        torch = self.torch
        T, H, I = int(x.shape[0]), self.H, self.I
        new = lambda *s: torch.empty(s, dtype=x.dtype, device=x.device)  # noqa: E731
        # n in the activations' type is read by the adapters, or by 16- and 32-bit weights
        adapters = self.gate_up is not None and ids is not None
        n = new(T, H) if adapters or not self.eight else None
        s, h, y = new(T, H), new(T, I), new(T, H)
        n8 = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=x.device) if self.eight else None
        scale = torch.empty(T, device=x.device) if self.eight else None
        pre = new(T, 2 * I) if keep else None
        ws = self._workspace(max(L.lora_gated_ffn_workspace_bytes(self.gated_desc, T),
                                 L.lora_linear_workspace_bytes(self.down_desc, T)))
        L.lora_add_rms_norm(self.norm_desc, x, residual, self.norm_weight, s, n, n8, scale, T)
        d = self._delta(self.gate_up, n, ids, prefill, 2 * I)
        L.lora_gated_ffn(self.gated_desc, n8 if self.eight else n, self.w_gate_up, scale,
                         self.gate_up_scale, d, pre, h, T, ws, ws.numel())
        d = self._delta(self.down, h, ids, prefill, H)
        block = None
        if self.join_desc is None:
            L.lora_linear(self.down_desc, h, self.w_down, None, None, None, d, s, y, T, ws,
                          ws.numel())
        else:
            block = new(T, H)
            L.lora_linear(self.down_desc, h, self.w_down, None, None, None, d, None, block, T, ws,
                          ws.numel())
            L.lora_block_norm(self.join_desc, block, s, self.gate, self.post_norm_weight, None, y,
                              None, None, None, T)
        self._saved = (n, pre) if keep else None
        self._saved_rest = None
        if keep and keep != "gate_up" and not self.eight:
            kept = None if ids is None else np.array(ids, dtype=np.int32)
            if self.down is None or ids is None:
                h = None       # (its adapters alone take it)
            if self.post_norm_weight is None and self.gate is None:
                block = None   # (scales alone need no value of it)
            self._saved_rest = (s, h, block, kept)
        return y

    def _delta(self, pool, x, ids, prefill, width):
        if pool is None or ids is None or x.shape[0] == 0:
            return None
        d = self.torch.zeros((x.shape[0], width), dtype=x.dtype, device=x.device)
        pool.apply(x, d, ids, prefill)
        return d

    def gate_up_backward(self, dh, need_dw: bool = True):
        """Gradients of the kept forward pass from dh [T][I], the gradient of h:
        (dpre [T][2 I], which is also the delta's gradient, the base product's
        part of dn [T][H], dW_gate_up [2 I][H] or None).  w_gate_up must not be
        in e4m3."""
        if self._saved is None:
            raise L.LoraError(L.LORA_E_ARG, "no forward pass was kept (keep=True)")
        if self.eight:
            raise L.LoraError(L.LORA_E_DTYPE, "the gradients take weights in fp32 or bf16")
        self._check_rows(dh, self.I, "dh")
        if dh.shape[0] != self._saved[0].shape[0]:
            raise L.LoraError(L.LORA_E_SHAPE, "dh must have the kept pass's rows")
        return self._on_device(self._gate_up_backward, dh, need_dw)

    def _gate_up_backward(self, dh, need_dw):
        torch = self.torch
        n, pre = self._saved
        T = int(n.shape[0])
        dpre, dn = torch.empty_like(pre), torch.empty_like(n)
        dw = torch.empty_like(self.w_gate_up) if need_dw else None
        ws = self._workspace(L.lora_gated_ffn_backward_workspace_bytes(self.grad_desc, T, True,
                                                                       need_dw))
        L.lora_gated_ffn_backward(self.grad_desc, dh, pre, n if need_dw else None, self.w_gate_up,
                                  dpre, dn, dw, T, ws, ws.numel())
        return dpre, dn, dw

    def backward(self, dy, w_down_t, need_dw: bool = False, grads=None, accumulate: bool = False,
                 plans=None):
        """Gradients of the kept forward pass from dy [T][H], the gradient of y, as a dict:
        "x" (also residual's), "norm_weight" (fp32, as the next two), "post_norm_weight", "gate",
        "gate_up" and "down" ((dA, dB) of the pools, as LoraPool.backward gives them) and
        "w_gate_up" (need_dw).  w_down_t: w_down transposed, [I][H]; the base is frozen in this
        pass, so that a program makes it once.  grads: buffers for the fp32 sums by these names,
        which accumulate adds to (16-byte aligned, apart from each other); new ones are made for
        the others.  plans: the pools'
        backward_plan of the kept ids by "gate_up" and "down", where a program makes them once for
        a step's layers or captures the pass; made here otherwise, which waits for the GPU.
        Weights must not be in e4m3.  Takes the kept pass with it."""
        if self._saved is None:
            raise L.LoraError(L.LORA_E_ARG, "no forward pass was kept (keep=True)")
        if self.eight:
            raise L.LoraError(L.LORA_E_DTYPE, "the gradients take weights in fp32 or bf16")
        if self._saved_rest is None:
            raise L.LoraError(L.LORA_E_ARG, "the pass was kept for gate_up_backward alone")
        self._check_rows(dy, self.H, "dy")
        if dy.shape[0] != self._saved[0].shape[0]:
            raise L.LoraError(L.LORA_E_SHAPE, "dy must have the kept pass's rows")
        if tuple(w_down_t.shape) != (self.I, self.H) or not w_down_t.is_contiguous():
            raise L.LoraError(L.LORA_E_SHAPE, "w_down_t must be a contiguous [I, H]")
        if w_down_t.dtype != self.w_down.dtype or w_down_t.device != self.w_down.device:
            raise L.LoraError(L.LORA_E_DTYPE, "w_down_t must have w_down's dtype and device")
        grads = {k: v for k, v in (grads or {}).items() if v is not None}
        plans = dict(plans or {})
        pools = {k: p for k, p in (("gate_up", self.gate_up), ("down", self.down)) if p is not None}
        rows = {"norm_weight": self.norm_weight, "post_norm_weight": self.post_norm_weight,
                "gate": self.gate}
        rows = {k for k, v in rows.items() if v is not None}
        for k in ("norm_weight", "post_norm_weight", "gate"):
            t = grads.get(k)
            if t is not None and (t.dtype != self.torch.float32 or tuple(t.shape) != (self.H,) or
                                  not t.is_contiguous() or t.device != self.w_down.device):
                raise L.LoraError(L.LORA_E_SHAPE, f"the gradient of {k} must be fp32 [H]")
        for what, given, names in (("gradients", grads, rows | set(pools)),
                                   ("plans", plans, set(pools))):
            if set(given) - names:
                raise L.LoraError(L.LORA_E_ARG, f"{what} of {sorted(set(given) - names)}, which "
                                                "the block does not have")
        for k in set(grads) & set(pools):
            pools[k].check_grads(*grads[k])
        self._check_buffers(
            [(k, t) for k, v in grads.items() for t in (v if k in pools else (v,)) if t is not None],
            [("dy", dy), ("w_down_t", w_down_t)] +
            [(f"{k}'s pool", t) for k, p in pools.items() for t in (p.A, p.B)])
        ids = self._saved_rest[3]
        for k, pool in pools.items():
            if ids is None:
                plans.pop(k, None)
                continue
            if k not in plans:
                if dy.is_cuda and self.torch.cuda.is_current_stream_capturing():
                    raise L.LoraError(L.LORA_E_ARG, "a captured pass takes its plans from outside")
                plans[k] = pool.backward_plan(ids)
            pool.check_plan(plans[k], dy.shape[0])
        return self._on_device(self._backward, dy, w_down_t, need_dw, grads, accumulate, plans)

    def _check_buffers(self, written, read) -> None:
        """Refuses what an operator of the pass would refuse after others have added to their
        sums: tensors off 16 bytes, and gradients that overlap each other or what is read."""
        for name, t in written + read:
            if t.data_ptr() % 16:
                raise L.LoraError(L.LORA_E_ALIGN, f"{name} must be 16-byte aligned")
        span = lambda t: (t.data_ptr(), t.data_ptr() + t.nbytes)  # noqa: E731
        for i, (name, t) in enumerate(written):
            a, b = span(t)
            for other, u in written[i + 1:] + read:
                c, d = span(u)
                if max(a, c) < min(b, d):
                    raise L.LoraError(L.LORA_E_ARG, f"the gradient of {name} overlaps {other}")

    def _backward(self, dy, w_down_t, need_dw, grads, accumulate, plans):
        torch = self.torch
        (n, pre), (s, h, block, _) = self._saved, self._saved_rest
        T, out = int(dy.shape[0]), {}
        row = lambda k: (grads[k] if k in grads else  # noqa: E731
                         torch.zeros(self.H, device=dy.device))
        ws = self._workspace(max(
            L.lora_linear_workspace_bytes(self.dh_desc, T),
            L.lora_gated_ffn_backward_workspace_bytes(self.grad_desc, T, True, need_dw),
            L.lora_block_norm_backward_workspace_bytes(self.norm_grad_desc, T)))

        def adapters(name, pool, x, d, dx):
            """dx += the adapters' part; their gradients."""
            if name not in plans:
                return
            dA, dB = grads.get(name, (None, None))
            out[name] = pool.backward(x, d, plans[name], dx, dx, dA, dB,
                                      accumulate=accumulate)[1:]

        ds, db = dy, dy     # gradients of s and of the block's output
        if self.join_desc is not None:
            ds, db = torch.empty_like(dy), torch.empty_like(dy)
            if self.post_norm_weight is not None:
                out["post_norm_weight"] = row("post_norm_weight")
            if self.gate is not None:
                out["gate"] = row("gate")
            L.lora_block_norm_backward(
                self.join_desc, None, dy, block, None, self.gate, self.post_norm_weight, None, db,
                ds, out.get("gate"), out.get("post_norm_weight"), None, accumulate, T, ws,
                ws.numel())
        dh = torch.empty((T, self.I), dtype=dy.dtype, device=dy.device)
        L.lora_linear(self.dh_desc, db, w_down_t, None, None, None, None, None, dh, T, ws,
                      ws.numel())
        adapters("down", self.down, h, db, dh)
        dpre, dn = torch.empty_like(pre), torch.empty_like(n)
        dw = torch.empty_like(self.w_gate_up) if need_dw else None
        L.lora_gated_ffn_backward(self.grad_desc, dh, pre, n if need_dw else None, self.w_gate_up,
                                  dpre, dn, dw, T, ws, ws.numel())
        if need_dw:
            out["w_gate_up"] = dw
        adapters("gate_up", self.gate_up, n, dpre, dn)
        out["norm_weight"] = row("norm_weight")
        dx = torch.empty_like(dy)
        # (sum = x + residual: one gradient for both)
        L.lora_block_norm_backward(self.norm_grad_desc, dn, ds, None, s, None, None,
                                   self.norm_weight, None, dx, None, None, out["norm_weight"],
                                   accumulate, T, ws, ws.numel())
        out["x"] = dx
        self._saved = self._saved_rest = None
        return out
