"""The host plan of the delta's gradients: every row once, sorted by adapter; tiles and
pieces of one adapter; buffers of exactly the documented size; refusals."""
import ctypes

import numpy as np
import pytest

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib
from test_block_host import FAKE, status, variants


def check(desc, ids):
    ids = np.asarray(ids, np.int32)
    T = len(ids)
    words = L.lora_delta_backward_image_bytes(desc, T) // 4
    guarded = np.full(words + 8, 0x5A5A5A5A, np.int32)
    p, image = L.lora_delta_backward_plan(desc, ids, guarded[4:-4])
    assert (guarded[:4] == 0x5A5A5A5A).all() and (guarded[-4:] == 0x5A5A5A5A).all()
    perm = image[:T]
    assert p.rows == int((ids >= 0).sum()) and p.none == T - p.rows
    order = np.lexsort((np.arange(T), np.where(ids < 0, 1 << 30, ids)))
    assert (perm == order).all()
    tiles = image[p.off_tiles:p.off_tiles + 4 * (p.tiles + p.none_tiles)].reshape(-1, 4)
    seen = []
    for k, (slot, rows, first, _) in enumerate(tiles):
        assert 1 <= rows <= 64 and (slot == -1) == (k >= p.tiles)
        assert (ids[perm[first:first + rows]] == slot).all()
        seen += range(first, first + rows)
    assert seen == list(range(T))
    parts = image[p.off_parts:p.off_parts + 4 * p.parts].reshape(-1, 4)
    seen, partials = [], []
    for slot, rows, tile, to in parts:
        first = tiles[tile][2]
        assert rows >= 1 and (ids[perm[first:first + rows]] == slot).all()
        whole = rows == (ids == slot).sum()
        assert (to == -1) == whole
        partials += [] if whole else [(to, slot)]
        seen += range(first, first + rows)
    assert sorted(seen) == list(range(p.rows)) and (np.diff(parts[:, 1]) <= 0).all()
    partials.sort()
    assert [q for q, _ in partials] == list(range(p.partials))
    multi = image[p.off_multi:p.off_multi + 4 * p.multi].reshape(-1, 4)
    flat = [(q, slot) for slot, at, n, _ in multi for q in range(at, at + n)]
    assert flat == partials and p.image_bytes == 4 * (p.off_multi + 4 * p.multi)
    # the kernels read up to seven words behind perm's last row with an adapter
    assert not p.rows or p.image_bytes // 4 >= p.rows + 7
    return p


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 700, 9000])
@pytest.mark.parametrize("slots", [1, 5, 64])
def test_plans(T, slots):
    rng = np.random.default_rng(T + slots)
    desc = L.make_desc("bf16", slots, 16, 256, [256])
    for ids in (np.full(T, -1), np.zeros(T), np.full(T, slots - 1), np.arange(T) % slots,
                rng.integers(-1, slots, T), np.sort(rng.integers(-1, slots, T)),
                np.where(rng.random(T) < 0.9, 0, rng.integers(-1, slots, T))):
        p = check(desc, ids)
        assert p.chunk % 64 == 0


def test_pieces_and_parts():
    """Long runs are cut where there are few columns; reductions where there are few tiles."""
    small = L.make_desc("bf16", 4, 16, 256, [256])
    assert check(small, np.zeros(9000)).partials > 1
    assert check(small, np.zeros(100)).partials == 0
    wide = L.make_desc("bf16", 4, 64, 16384, [131072])
    assert check(wide, np.zeros(9000)).partials == 0
    p = check(L.make_desc("bf16", 4, 16, 4096, [4096]), np.zeros(64))
    assert 256 <= p.chunk < 4096
    assert check(L.make_desc("bf16", 64, 64, 4096, [4096]),
                 np.arange(40000) % 64).chunk == 4096


def test_workspace_does_not_shrink():
    rng = np.random.default_rng(1)
    for dtype, R, K, outs in (("bf16", 16, 256, [256]), ("bf16", 64, 4096, [14336, 14336]),
                              ("f32", 8, 64, [64, 128, 72]), ("bf16", 512, 1024, [1024])):
        desc, last = L.make_desc(dtype, 8, R, K, outs), 0
        assert L.lora_delta_backward_workspace_bytes(desc, 0) == 0
        for T in sorted(rng.integers(1, 1 << 21, 200).tolist() + list(range(1, 40)) + [1 << 21]):
            n = L.lora_delta_backward_workspace_bytes(desc, T)
            assert n >= last
            last = n


def test_plan_refusals():
    desc = L.make_desc("bf16", 4, 16, 256, [256])
    for ids, want in (([0, 4], _lib.LORA_E_ID), ([0, -2], _lib.LORA_E_ID),
                      ([[0, 1]], _lib.LORA_E_SHAPE)):
        assert status(lambda i, stream: L.lora_delta_backward_plan(desc, i), ids) == want
    small = np.empty(L.lora_delta_backward_image_bytes(desc, 9) // 4 - 1, np.int32)
    assert status(lambda stream: L.lora_delta_backward_plan(desc, [0] * 9, small)) == \
        _lib.LORA_E_WORKSPACE
    lib, p = L.lib(), _lib.lora_delta_plan()
    d, at = ctypes.byref(desc), small.ctypes.data
    assert lib.lora_delta_backward_plan(d, -1, at, at, 1 << 20, ctypes.byref(p)) == _lib.LORA_E_ARG
    assert lib.lora_delta_backward_plan(d, 4, None, at, 1 << 20, ctypes.byref(p)) == \
        _lib.LORA_E_ARG
    assert lib.lora_delta_backward_plan(d, 4, at, None, 1 << 20, ctypes.byref(p)) == \
        _lib.LORA_E_ARG
    assert lib.lora_delta_backward_image_bytes(d, (1 << 21) + 1) == _lib.LORA_E_SHAPE
    bad = L.make_desc("bf16", 4, 12, 256, [256])
    assert lib.lora_delta_backward_workspace_bytes(ctypes.byref(bad), 4) == _lib.LORA_E_ALIGN


def test_call_refusals():
    desc = L.make_desc("bf16", 4, 16, 256, [256])
    plan, _ = L.lora_delta_backward_plan(desc, [0, 1, -1, 3, 0])
    need = L.lora_delta_backward_workspace_bytes(desc, 5)
    ok = [desc] + [FAKE] * 8 + [5, plan, FAKE, 0, FAKE, need]
    other, _ = L.lora_delta_backward_plan(desc, [0, 1])
    forged = _lib.lora_delta_plan.from_buffer_copy(plan)
    forged.off_parts += 4
    wide = L.make_desc("bf16", 4, 16, 256, [4096])
    variants(L.lora_delta_backward, ok, [
        (0, L.make_desc("bf16", 4, 12, 256, [256]), _lib.LORA_E_ALIGN),
        (0, wide, _lib.LORA_E_ARG),                                   # another pool's plan
        (1, None, _lib.LORA_E_ARG), (2, None, _lib.LORA_E_ARG), (3, None, _lib.LORA_E_ARG),
        (4, None, _lib.LORA_E_ARG), (6, None, _lib.LORA_E_ARG),       # dx_in without dx
        (7, None, _lib.LORA_E_ARG), (8, None, _lib.LORA_E_ARG),       # dA without dB
        (9, 4, _lib.LORA_E_ARG), (9, -1, _lib.LORA_E_ARG), (9, (1 << 21) + 1, _lib.LORA_E_SHAPE),
        (10, other, _lib.LORA_E_ARG), (10, forged, _lib.LORA_E_ARG), (11, None, _lib.LORA_E_ARG),
        (12, 2, _lib.LORA_E_ARG), (13, None, _lib.LORA_E_ARG),
        (14, need - 1, _lib.LORA_E_WORKSPACE), (3, FAKE + 2, _lib.LORA_E_ALIGN),
        (7, FAKE + 4, _lib.LORA_E_ALIGN), (11, FAKE + 4, _lib.LORA_E_ALIGN)])
    none = [desc] + [FAKE] * 4 + [None] * 4 + ok[9:]
    assert status(L.lora_delta_backward, *none) == _lib.LORA_E_ARG    # nothing to compute
    empty, _ = L.lora_delta_backward_plan(desc, [])
    assert status(L.lora_delta_backward, desc, *[None] * 8, 0, empty, None, 0, None, 0) == 0


def test_overlaps_and_limits():
    """dx is dx_in or apart; nothing else that is written overlaps a buffer."""
    desc = L.make_desc("bf16", 4, 16, 256, [256])
    plan, _ = L.lora_delta_backward_plan(desc, [0, 1, -1, 3, 0])
    need = L.lora_delta_backward_workspace_bytes(desc, 5)
    apart = [(i + 1) << 30 for i in range(10)]   # A, B, x, dy, dx_in, dx, dA, dB, image, ws

    def call(at, d=desc, p=plan):
        return status(L.lora_delta_backward, d, *at[:8], 5, p, at[8], 0, at[9], need)

    x_bytes = 5 * 256 * 2
    for i, j, shift in ((5, 2, 0), (5, 3, 16), (5, 4, 512), (5, 4, -x_bytes + 16), (6, 7, 0),
                        (6, 0, 0), (7, 1, 0), (9, 8, 0), (9, 2, x_bytes - 16), (8, 9, need - 16)):
        at = list(apart)
        at[i] = apart[j] + shift
        assert call(at) == _lib.LORA_E_ARG, (i, j)
    tall = L.make_desc("bf16", 1, (1 << 16) + 8, 64, [64])
    p, _ = L.lora_delta_backward_plan(tall, [0] * 5)
    assert call(apart, tall, p) == _lib.LORA_E_SHAPE
