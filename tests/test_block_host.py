"""The decoder-block operators' checks of arguments and workspace sizes, all
made on the host before any GPU call, and the two binding routes' agreement on
them."""
import ctypes

import pytest

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib

FAKE = 1 << 20   # an aligned address that is never read


def status(f, *a):
    try:
        f(*a, stream=0)
        return 0
    except L.LoraError as e:
        assert L.last_error()
        return e.status


def variants(f, ok, cases):
    for i, v, want in cases:
        a = list(ok)
        a[i] = v
        assert status(f, *a) == want, (i, v)


def test_norm_refusals():
    d = L.make_norm_desc("bf16", 1024, 1e-5)
    ok = [d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4]
    mk = L.make_norm_desc
    variants(L.lora_add_rms_norm, ok, [
        (0, mk("e4m3", 1024, 1e-5), _lib.LORA_E_DTYPE), (0, mk("bf16", 0, 1e-5), _lib.LORA_E_SHAPE),
        (0, mk("bf16", 1028, 1e-5), _lib.LORA_E_ALIGN),
        (0, mk("bf16", 32776, 1e-5), _lib.LORA_E_SHAPE),
        (0, mk("bf16", 1024, -1.0), _lib.LORA_E_ARG),
        (0, mk("bf16", 1024, float("nan")), _lib.LORA_E_ARG),
        (1, None, _lib.LORA_E_ARG), (3, None, _lib.LORA_E_ARG), (2, None, _lib.LORA_E_ARG),
        (4, None, _lib.LORA_E_ARG), (6, None, _lib.LORA_E_ARG), (7, None, _lib.LORA_E_ARG),
        (1, FAKE + 2, _lib.LORA_E_ALIGN), (6, FAKE + 8, _lib.LORA_E_ALIGN),
        (8, -1, _lib.LORA_E_ARG), (8, (1 << 21) + 1, _lib.LORA_E_SHAPE)])
    assert status(L.lora_add_rms_norm, d, FAKE, None, FAKE, None, None, None, None, 4) == \
        _lib.LORA_E_ARG                                            # no output at all
    assert status(L.lora_add_rms_norm, d, *[None] * 7, 0) == 0     # T = 0


def test_linear_refusals():
    mk = L.make_linear_desc
    d = mk("bf16", "bf16", 4096, 300)
    need = L.lora_linear_workspace_bytes(d, 8)
    assert need > 0
    ok = [d, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 8, FAKE, need]
    variants(L.lora_linear, ok, [
        (0, mk("f32", "bf16", 4096, 300), _lib.LORA_E_DTYPE),
        (0, mk("bf16", "e4m3", 4096, 300), _lib.LORA_E_DTYPE),
        (0, mk("bf16", "bf16", 0, 300), _lib.LORA_E_SHAPE),
        (0, mk("bf16", "bf16", 4100, 300), _lib.LORA_E_ALIGN),
        (0, mk("bf16", "bf16", 4096, 0), _lib.LORA_E_SHAPE),
        (0, mk("bf16", "bf16", 4096, (1 << 20) + 1), _lib.LORA_E_SHAPE),
        (0, mk("e4m3", "bf16", 4096, 300), _lib.LORA_E_ARG),       # no scales
        (0, mk("e4m3", "bf16", 4104, 300), _lib.LORA_E_ALIGN),
        (3, FAKE, _lib.LORA_E_ARG), (4, FAKE, _lib.LORA_E_ARG),    # scales without e4m3
        (1, None, _lib.LORA_E_ARG), (2, None, _lib.LORA_E_ARG), (8, None, _lib.LORA_E_ARG),
        (1, FAKE + 8, _lib.LORA_E_ALIGN), (5, FAKE + 2, _lib.LORA_E_ALIGN),
        (6, FAKE + 2, _lib.LORA_E_ALIGN), (7, FAKE + 4, _lib.LORA_E_ALIGN),
        (9, -1, _lib.LORA_E_ARG), (9, (1 << 21) + 1, _lib.LORA_E_SHAPE),
        (10, None, _lib.LORA_E_ARG), (11, need - 1, _lib.LORA_E_WORKSPACE)])
    bad = mk("bf16", "bf16", 4096, 300)
    bad.act = 5
    variants(L.lora_linear, ok, [(0, bad, _lib.LORA_E_ARG)])
    bad.act, bad.dtype = 0, 7
    variants(L.lora_linear, ok, [(0, bad, _lib.LORA_E_DTYPE)])
    assert status(L.lora_linear, d, *[None] * 8, 0, None, 0) == 0  # T = 0
    for T in (-1, (1 << 21) + 1):
        with pytest.raises(L.LoraError):
            L.lora_linear_workspace_bytes(d, T)


def test_gated_refusals():
    mk = L.make_gated_desc
    d = mk("bf16", "bf16", 4096, 256)
    need = L.lora_gated_ffn_workspace_bytes(d, 8)
    assert need > 0
    ok = [d, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 8, FAKE, need]
    variants(L.lora_gated_ffn, ok, [
        (0, mk("bf16", "bf16", 4096, 252), _lib.LORA_E_ALIGN),
        (0, mk("e4m3", "bf16", 4096, 264), _lib.LORA_E_ALIGN),
        (0, mk("e4m3", "bf16", 4096, 256), _lib.LORA_E_ARG),
        (0, mk("f32", "bf16", 4096, 256), _lib.LORA_E_DTYPE),
        (3, FAKE, _lib.LORA_E_ARG), (1, None, _lib.LORA_E_ARG), (7, None, _lib.LORA_E_ARG),
        (5, FAKE + 2, _lib.LORA_E_ALIGN), (6, FAKE + 2, _lib.LORA_E_ALIGN),
        (8, -1, _lib.LORA_E_ARG), (10, need - 1, _lib.LORA_E_WORKSPACE)])
    assert status(L.lora_gated_ffn, d, *[None] * 7, 0, None, 0) == 0


def test_backward_refusals():
    mk = L.make_gated_desc
    d = mk("bf16", "bf16", 512, 256)
    size = L.lora_gated_ffn_backward_workspace_bytes
    need = size(d, 8)
    assert size(d, 8, True, False) <= need and size(d, 8, False, True) <= need
    assert size(d, 8, False, False) == 0
    ok = [d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, FAKE, need]
    variants(L.lora_gated_ffn_backward, ok, [
        (0, mk("e4m3", "bf16", 512, 256), _lib.LORA_E_DTYPE),
        (0, mk("bf16", "f32", 512, 256), _lib.LORA_E_DTYPE),
        (1, None, _lib.LORA_E_ARG), (2, None, _lib.LORA_E_ARG), (3, None, _lib.LORA_E_ARG),
        (4, None, _lib.LORA_E_ARG), (5, None, _lib.LORA_E_ARG),
        (6, FAKE + 2, _lib.LORA_E_ALIGN), (7, FAKE + 2, _lib.LORA_E_ALIGN),
        (8, -1, _lib.LORA_E_ARG)])
    if need:
        variants(L.lora_gated_ffn_backward, ok, [(10, need - 1, _lib.LORA_E_WORKSPACE)])
    assert status(L.lora_gated_ffn_backward, d, *[None] * 7, 0, None, 0) == 0


def test_null_descriptors():
    lib = _lib.lib()
    assert lib.lora_linear_workspace_bytes(None, 4) == _lib.LORA_E_ARG
    assert lib.lora_gated_ffn_workspace_bytes(None, 4) == _lib.LORA_E_ARG
    assert lib.lora_gated_ffn_backward_workspace_bytes(None, 4, 1, 1) == _lib.LORA_E_ARG
    assert lib.lora_add_rms_norm(None, *[FAKE] * 7, 4, 0) == _lib.LORA_E_ARG


def test_workspace_grows_with_nothing_but_sizes():
    """The workspace covers what the call's plan needs at every size of a range
    (the call checks against the same plan)."""
    for dtype in ("bf16", "f32", "e4m3"):
        for T in (1, 7, 64, 65, 500, 8960):
            for K, O in ((64, 17), (4096, 100), (14336, 4096), (4096, 14336)):
                n = L.lora_linear_workspace_bytes(L.make_linear_desc(dtype, "f32", K, O), T)
                assert 0 <= n <= 64 << 20, (dtype, T, K, O, n)


def test_routes_agree_on_refusals():
    d = L.make_linear_desc("bf16", "bf16", 4100, 300)
    with pytest.raises(L.LoraError) as e:
        L.lora_linear(d, FAKE, FAKE, None, None, None, None, None, FAKE, 4, None, 0, stream=0)
    message = str(e.value)
    st = _lib.lib().lora_linear(ctypes.byref(d), FAKE, FAKE, None, None, None, None, None, FAKE, 4,
                                None, 0, None)
    assert st == e.value.status and L.last_error() in message
