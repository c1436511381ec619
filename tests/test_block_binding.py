"""What the binding of the decoder-block operators takes as device memory: an
address as it is, and a tensor only if a kernel may be handed it.  On the CPU: a
stand-in with a tensor's attributes plays the GPU tensor, and what would pass is
stopped by an entry point's own check (a misaligned address) before any GPU call."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib

FAKE = 1 << 20   # an aligned address that is never read


class Gpu:
    """A tensor of `nbytes` in GPU memory, by its attributes."""

    def __init__(self, nbytes, contiguous=True, at=FAKE, is_cuda=True):
        self.nbytes, self.contiguous, self.at, self.is_cuda = nbytes, contiguous, at, is_cuda

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.at


T, K, O, I, H = 5, 64, 48, 32, 64
LIN = L.make_linear_desc("bf16", "f32", K, O)
LIN8 = L.make_linear_desc("e4m3", "bf16", K, O)
GATED = L.make_gated_desc("e4m3", "bf16", K, I)
GRAD = L.make_gated_desc("f32", "f32", K, I)
NORM = L.make_norm_desc("bf16", H, 1e-5)
WS = 1 << 27
# entry point, its arguments with each tensor's size, and where the entry point's
# own check is provoked
CALLS = [
    (L.lora_add_rms_norm, [NORM, ("x", T * H * 2), ("residual", T * H * 2), ("weight", H * 2),
                           ("sum", T * H * 2), ("out", T * H * 2), ("out8", T * H),
                           ("scale", T * 4), T]),
    (L.lora_linear, [LIN, ("x", T * K * 2), ("w", O * K * 2), None, None, ("bias", O * 4),
                     ("delta", T * O * 4), ("residual", T * O * 4), ("out", T * O * 4), T,
                     ("ws", WS), WS]),
    (L.lora_linear, [LIN8, ("x", T * K), ("w", O * K), ("x_scale", T * 4), ("w_scale", O * 4),
                     ("bias", O * 2), ("delta", T * O * 2), ("residual", T * O * 2),
                     ("out", T * O * 2), T, ("ws", WS), WS]),
    (L.lora_gated_ffn, [GATED, ("x", T * K), ("w", 2 * I * K), ("x_scale", T * 4),
                        ("w_scale", 2 * I * 4), ("delta", T * 2 * I * 2), ("pre", T * 2 * I * 2),
                        ("out", T * I * 2), T, ("ws", WS), WS]),
    (L.lora_gated_ffn_backward, [GRAD, ("dout", T * I * 4), ("pre", T * 2 * I * 4),
                                 ("x", T * K * 4), ("w", 2 * I * K * 4), ("dpre", T * 2 * I * 4),
                                 ("dx", T * K * 4), ("dw", 2 * I * K * 4), T, ("ws", WS), WS])]


def args(spec, change=None, by=None):
    """The call's arguments as stand-ins of just the size, one of them changed.
    The first is misaligned in every call, so that none gets past the entry
    point's own checks (LORA_E_ALIGN)."""
    out = []
    for a in spec:
        if isinstance(a, tuple):
            a = by(a[1]) if a[0] == change else Gpu(a[1], at=FAKE + 8 * (len(out) == 1))
        out.append(a)
    return out


def refused(f, a, status, says=""):
    with pytest.raises(L.LoraError) as e:
        f(*a, stream=0)
    assert e.value.status == status and says in str(e.value), str(e.value)


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_tensors_that_are_refused(call):
    f, spec = CALLS[call]
    for name, size in [a for a in spec if isinstance(a, tuple)]:
        short = _lib.LORA_E_WORKSPACE if name == "ws" else _lib.LORA_E_SHAPE
        refused(f, args(spec, name, lambda n: Gpu(n, contiguous=False)), _lib.LORA_E_SHAPE,
                f"{name} is not contiguous")
        refused(f, args(spec, name, lambda n: Gpu(n, is_cuda=False)), _lib.LORA_E_ARG,
                f"{name} is not GPU memory")
        refused(f, args(spec, name, lambda n: Gpu(n - 1)), short, f"{name} is smaller")
        # just the size passes the binding, and so does an address, as it is: the
        # entry point's own check is reached
        refused(f, args(spec, name, lambda n: Gpu(n, at=FAKE + 8)), _lib.LORA_E_ALIGN)
        refused(f, args(spec, name, lambda n: FAKE + 8), _lib.LORA_E_ALIGN)


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_tensors_of_the_host_and_other_objects(call):
    f, spec = CALLS[call]
    for name in [a[0] for a in spec if isinstance(a, tuple)]:
        refused(f, args(spec, name, lambda n: torch.zeros(n, dtype=torch.uint8)), _lib.LORA_E_ARG,
                f"{name} is not GPU memory")
        for other in (np.zeros(4096, np.uint8), "x", 1.5, object()):
            with pytest.raises(TypeError) as e:
                f(*args(spec, name, lambda n: other), stream=0)
            assert name in str(e.value)


def test_torch_tensors_by_their_c_interface():
    """Host tensors are told apart before their layout is looked at, whatever their
    type: parameters, 8-bit and empty tensors, strided views."""
    t = torch.zeros(2 * I, K)
    for w in (t, torch.nn.Parameter(t), t.t(), t.to(torch.float8_e4m3fn), t[:0], t[:, ::2]):
        a = args(CALLS[3][1], "w", lambda n: w)
        refused(L.lora_gated_ffn, a, _lib.LORA_E_ARG, "w is not GPU memory")


def test_arguments_that_a_call_does_not_read():
    f, spec = CALLS[4]
    # x is read for dw alone, w for dx alone; over no rows dw alone is touched
    a = args(spec, "x", lambda n: Gpu(0))
    a[7] = None                                             # no dw
    refused(f, a, _lib.LORA_E_ALIGN)
    a = args(spec, "w", lambda n: Gpu(0))
    a[6] = None                                             # no dx
    refused(f, a, _lib.LORA_E_ALIGN)
    f(*[GRAD] + [Gpu(0)] * 6 + [None, 0, None, 0], stream=0)
    refused(f, [GRAD] + [Gpu(0)] * 7 + [0, None, 0], _lib.LORA_E_SHAPE, "dw is smaller")
    for f, spec in CALLS[:4]:                               # an empty batch reads nothing
        a = [Gpu(0) if isinstance(v, tuple) else v for v in spec]
        a[a.index(T)] = 0
        f(*a, stream=0)


def test_sizes_past_32_bits():
    big = L.make_linear_desc("bf16", "bf16", 1 << 20, 1 << 20)      # w: 2 TiB
    a = [big, Gpu(1 << 42), Gpu((1 << 41) - 1), None, None, None, None, None, Gpu(1 << 42), 1 << 20,
         None, 0]
    refused(L.lora_linear, a, _lib.LORA_E_SHAPE, "w is smaller")
    a[2] = Gpu(1 << 41, at=FAKE + 8)
    refused(L.lora_linear, a, _lib.LORA_E_ALIGN, "w")
