"""The feed-forward half of a decoder layer with adapters, as one path.

    s = x + residual                          (the residual stream)
    n = rms_norm(s) * norm_weight             (and, for 8-bit weights, n in e4m3)
    h = act(n Wg^T + dg) * (n Wu^T + du)      dg, du: the adapters' gate/up delta
    y = h Wd^T + dd + s                       dd: the adapters' down delta

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

from . import _lib as L
from .pool import LoraPool


class LoraMlp:
    """norm_weight [H], w_gate_up [2 I][H] (gate rows, then up rows), w_down
    [H][I], all of the activations' dtype (fp32 or bf16); or w_gate_up in e4m3
    with one fp32 scale a row in gate_up_scale, for bf16 activations.  gate_up
    and down: pools of the activations' dtype with slices [I, I] and [H]."""

    def __init__(self, norm_weight, w_gate_up, w_down, eps: float = 1e-5, act: str = "silu",
                 gate_up_scale=None, gate_up: Optional[LoraPool] = None,
                 down: Optional[LoraPool] = None):
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
        for t in (norm_weight, w_gate_up, w_down, gate_up_scale):
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
        self._ws = None
        self._outgrown = []
        self._saved = None

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

    def forward(self, x, residual, ids=None, prefill=None, keep: bool = False):
        """y [T][H] on the current stream of the weights' GPU.  ids, prefill: as
        LoraPool.apply takes them (None: no adapters).  keep: hold what
        gate_up_backward needs."""
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
        L.lora_linear(self.down_desc, h, self.w_down, None, None, None, d, s, y, T, ws, ws.numel())
        self._saved = (n, pre) if keep else None
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
