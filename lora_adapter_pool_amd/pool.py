"""A rank-padded adapter pool in HBM plus the per-call workspace of lora_apply.

Thin owner of device memory (torch tensors) around the C ABI: it allocates the
pool once ([vLLM] step 2 of the vLLM offline multi-LoRA article: max_loras
slots pre-allocated at max_lora_rank), loads adapters through lora_pool_load and
calls lora_apply with a device workspace and a small ring of pinned host
staging buffers (a buffer is reused only after the stream has passed the call
that last read it).  It records the rank loaded into each slot and slice, so
apply(..., ragged=True) can pass each slot's true rank to lora_apply_ranked.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import numpy as np

from . import _lib as L


class DeltaPlan:
    """The plan of a batch's rows for LoraPool.backward: the host's records and their image
    on the pool's GPU.  It serves every pool of this geometry, and every call with these ids
    (the layers of a step); keep it as long as graphs that its calls were captured in."""

    def __init__(self, desc, ids, device):
        import torch

        self.struct, image = L.lora_delta_backward_plan(desc, ids)
        self.T = self.struct.rows + self.struct.none
        self.geometry = bytes(desc)
        self.image = torch.from_numpy(image).to(device)


class LoraPool:
    def __init__(self, dtype: str, max_loras: int, max_lora_rank: int, in_features: int,
                 out_features: Sequence[int], device: str = "cuda", staging_slots: int = 3):
        import torch

        self.torch = torch
        self.dtype = "bf16" if dtype in ("bf16", "bfloat16") else "f32"
        self.tdtype = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        self.desc = L.make_desc(self.dtype, max_loras, max_lora_rank, in_features, out_features)
        L.lora_pool_validate(self.desc)
        eb = 2 if self.dtype == "bf16" else 4
        self.max_loras = int(max_loras)
        self.R = int(max_lora_rank)
        self.K = int(in_features)
        self.out_features = [int(o) for o in out_features]
        self.O = sum(self.out_features)
        self.device = device
        self.A = torch.zeros(L.lora_pool_bytes_A(self.desc) // eb, dtype=self.tdtype, device=device)
        self.B = torch.zeros(L.lora_pool_bytes_B(self.desc) // eb, dtype=self.tdtype, device=device)
        # rank last loaded into each (slot, slice); 0 = nothing loaded (zeros)
        self.loaded_ranks = np.zeros((self.max_loras, len(self.out_features)), np.int32)
        self._ws = None
        self._bws = None
        self._outgrown: List = []
        self._staging: List[list] = [[None, None] for _ in range(max(1, staging_slots))]
        self._next = 0

    # views in the documented layouts
    def A_view(self):
        return self.A.view(self.max_loras, len(self.out_features), self.R, self.K)

    def B_view(self):
        return self.B.view(self.max_loras, self.O, self.R)

    def load(self, slot: int, slice_: int, A_src, B_src, rank: int, alpha: float,
             use_rslora: bool = False, stream=None) -> None:
        L.lora_pool_load(self.desc, self.A, self.B, slot, slice_, A_src, B_src, rank, alpha,
                         use_rslora, stream=stream)
        self.loaded_ranks[slot, slice_] = rank

    def clear(self, slot: int, stream=None) -> None:
        L.lora_pool_clear(self.desc, self.A, self.B, slot, stream=stream)
        self.loaded_ranks[slot, :] = 0

    def merge(self, slot: int, slice_: int, W, W_out=None, stream=None):
        """Merged-weight mode: W_out (default: a new tensor) = W + s B A of the
        adapter in `slot`, for the base weight W [out_s, in] of slice `slice_`."""
        if W.dtype != self.tdtype or not W.is_contiguous():
            raise L.LoraError(L.LORA_E_DTYPE, "W must be a contiguous tensor of the pool dtype")
        if tuple(W.shape) != (self.out_features[slice_], self.K):
            raise L.LoraError(L.LORA_E_SHAPE, f"W must be [{self.out_features[slice_]}, {self.K}]")
        out = self.torch.empty_like(W) if W_out is None else W_out
        if out.dtype != W.dtype or out.shape != W.shape or not out.is_contiguous():
            raise L.LoraError(L.LORA_E_SHAPE, "W_out must match W")
        st = self.torch.cuda.current_stream() if stream is None else stream
        L.lora_merge_weights(self.desc, self.A, self.B, slot, slice_, W, out, stream=st)
        return out

    def backward_plan(self, ids) -> DeltaPlan:
        """The plan that backward takes; ids int32 per row (-1 = none), on the host."""
        return DeltaPlan(self.desc, ids, self.A.device)

    def backward(self, x, dy, plan: DeltaPlan, dx_in=None, dx=None, dA=None, dB=None,
                 need_dx: bool = True, need_grads: bool = True, accumulate: bool = False):
        """Gradients of apply: (dx, dA, dB) from dy [T, O], the gradient of y, on the current
        stream of the pool's GPU.
        dx [T, K] = dx_in (the base projection's part; None: zeros) + the delta's; it may be
        dx_in itself.  dA, dB: fp32 gradients of A_view() and B_view(), overwritten or added to
        (accumulate) for the batch's slots, others left; new ones are zeros, of the whole pool's
        size, so that a program makes its own once.  peft's lora_B has the adapter's scale times
        dB's gradient.  A pool's calls share a workspace: two that run
        at once, or graphs of them, need pools of their own."""
        torch = self.torch
        if not self.A.is_cuda:
            raise L.LoraError(L.LORA_E_ARG, "the pool is not on a GPU")
        if not need_dx and not need_grads:
            raise L.LoraError(L.LORA_E_ARG, "neither dx nor the adapters' gradients are wanted")
        T, S = plan.T, len(self.out_features)
        self.check_plan(plan, T)
        want = {"x": (x, (T, self.K), self.tdtype), "dy": (dy, (T, self.O), self.tdtype),
                "dx_in": (dx_in, (T, self.K), self.tdtype), "dx": (dx, (T, self.K), self.tdtype)}
        self._check_tensors(want)
        if not need_dx and (dx is not None or dx_in is not None):
            raise L.LoraError(L.LORA_E_ARG, "dx is given and not wanted")
        if not need_grads and (dA is not None or dB is not None):
            raise L.LoraError(L.LORA_E_ARG, "dA or dB is given and not wanted")
        self.check_grads(dA, dB)
        with torch.cuda.device(self.A.device):
            if need_grads and dA is None:
                dA = torch.zeros((self.max_loras, S, self.R, self.K), device=self.A.device)
                dB = torch.zeros((self.max_loras, self.O, self.R), device=self.A.device)
            if need_dx and dx is None:
                dx = torch.empty_like(x)
            ws = self._backward_workspace(T)
            if T:
                L.lora_delta_backward(self.desc, self.A, self.B, x, dy, dx_in, dx, dA, dB, T,
                                      plan.struct, plan.image, accumulate, ws, ws.numel())
        return dx, dA, dB

    def check_plan(self, plan: DeltaPlan, T: int) -> None:
        """Refuses a plan of other rows, another geometry or another GPU."""
        if plan.T != T or plan.geometry != bytes(self.desc):
            raise L.LoraError(L.LORA_E_ARG, "the plan is not of these rows and this pool's geometry")
        if plan.image.device != self.A.device:
            raise L.LoraError(L.LORA_E_ARG, "the plan is not on the pool's GPU")

    def check_grads(self, dA, dB) -> None:
        """Refuses what backward cannot take as dA and dB (both None: new ones)."""
        if (dA is None) != (dB is None):
            raise L.LoraError(L.LORA_E_ARG, "dA and dB go together: one of them is None")
        f32 = self.torch.float32
        self._check_tensors({
            "dA": (dA, (self.max_loras, len(self.out_features), self.R, self.K), f32),
            "dB": (dB, (self.max_loras, self.O, self.R), f32)})

    def _check_tensors(self, want) -> None:
        """{name: (tensor or None, shape, dtype)}: contiguous and on the pool's GPU."""
        for name, (t, shape, dtype) in want.items():
            if t is None:
                continue
            if t.dtype != dtype or t.device != self.A.device:
                raise L.LoraError(L.LORA_E_DTYPE, f"{name} must be {dtype} on the pool's GPU")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise L.LoraError(L.LORA_E_SHAPE, f"{name} must be a contiguous {list(shape)}")

    def _backward_workspace(self, T: int):
        need = L.lora_delta_backward_workspace_bytes(self.desc, T)
        have = 0 if self._bws is None else self._bws.numel()
        if have < max(need, 1):
            if have:   # graphs that were captured before hold its address
                self._outgrown.append(self._bws)
            self._bws = self.torch.empty(max(need, 2 * have, 256), dtype=self.torch.uint8,
                                         device=self.A.device)
        return self._bws

    def slot_grads(self, dA, dB, slots, outs=None) -> L.GradList:
        """The gradients of some slots as lora_clip_grads takes them, a group for each slot in
        turn; outs: (dA, dB) that the clipped gradients go to (None: in place)."""
        for pair in (dA, dB), outs or (None, None):
            self.check_grads(*pair)
        slots = [int(k) for k in slots]
        for k in slots:
            if not 0 <= k < self.max_loras:
                raise L.LoraError(L.LORA_E_ID, f"slot {k} of {self.max_loras}")
        pick = lambda a, b: [t[k] for k in slots for t in (a, b)]  # noqa: E731
        return L.GradList(pick(dA, dB), [g for g in range(len(slots)) for _ in range(2)],
                          None if outs is None else pick(*outs), num_groups=len(slots))

    def slot_ranks(self) -> np.ndarray:
        """int32[max_loras]: the largest rank loaded into each slot; a slot with
        nothing loaded holds zeros and reports 1 (any rank gives a zero delta)."""
        return np.maximum(self.loaded_ranks.max(axis=1), 1).astype(np.int32)

    def workspace(self, T: int):
        need = L.lora_apply_workspace_bytes(self.desc, T)
        if self._ws is None or self._ws.numel() < need:
            self._ws = self.torch.empty(max(need, 256), dtype=self.torch.uint8, device=self.device)
        return self._ws

    def _staging_buffer(self, T: int, stream):
        need = L.lora_apply_host_meta_bytes(self.desc, T)
        slot = self._staging[self._next]
        self._next = (self._next + 1) % len(self._staging)
        buf, ev = slot
        if ev is not None:
            ev.synchronize()  # the stream has passed the call that last read this buffer
        if buf is None or buf.numel() < need:
            buf = self.torch.empty(max(need, 64), dtype=self.torch.uint8, pin_memory=True)
            slot[0] = buf
        return slot, buf, need

    def apply(self, x, y, ids, prefill=None, bgmv_max_rank: int = 0, stream=None,
              ragged: bool = False) -> None:
        """y (in place) += per-row LoRA delta for x; ids int32 per row (-1 = none).
        ragged: skip each slot's padded ranks (same result)."""
        torch = self.torch
        T = int(x.shape[0])
        ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
        pre = None if prefill is None else np.ascontiguousarray(np.asarray(prefill, dtype=np.uint8))
        if ids.shape[0] != T or (pre is not None and pre.shape[0] != T):
            raise L.LoraError(L.LORA_E_SHAPE, "ids / prefill length must equal the token count")
        ws = self.workspace(T)
        slot, buf, need = self._staging_buffer(T, stream)
        st = torch.cuda.current_stream() if stream is None else stream
        if ragged:
            L.lora_apply_ranked(self.desc, self.A, self.B, x, y, T, ids, pre, bgmv_max_rank,
                                self.slot_ranks(), ws, ws.numel(), buf, buf.numel(), stream=st)
        else:
            L.lora_apply(self.desc, self.A, self.B, x, y, T, ids, pre, bgmv_max_rank, ws,
                         ws.numel(), buf, buf.numel(), stream=st)
        ev = slot[1] or torch.cuda.Event()
        ev.record(st)
        slot[1] = ev
