"""lora_grad_list_build and lora_clip_grads on the CPU: the chunks of a list cover
every element once, group after group; refusals before any GPU call."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from lora_adapter_pool_amd import _lib
from test_block_host import FAKE

CHUNK = np.dtype([("in", "<u8"), ("out", "<u8"), ("count", "<i4"), ("dtype", "<i4"),
                  ("group", "<i4"), ("reserved", "<i4")])


def entries(rows):
    """rows: (address, out, count, dtype, group)"""
    return np.array([tuple(r) for r in rows], dtype=_lib.GRAD_DTYPE)


def unpack(lst, image):
    starts = image[:4 * (lst.groups + 1)].view(np.int32)
    at = -(-4 * (lst.groups + 1) // 32) * 32
    chunks = image[at:].view(CHUNK)
    assert len(image) == lst.bytes and len(chunks) == lst.chunks
    return starts, chunks


@pytest.mark.parametrize("sizes", [[1], [0, 7, 0], [2048, 2049, 5], [40000, 1, 70001, 333],
                                   [100_000_000, 3, 60_000_000]])
@pytest.mark.parametrize("groups", [1, 3])
def test_chunks_cover_the_tensors(sizes, groups):
    at, rows = FAKE, []
    for i, n in enumerate(sizes):
        e = 2 if i % 2 else 4
        rows.append((at, 0 if i % 3 else at + (1 << 40), n, i % 2, (i * 2) % groups))
        at = (at + n * e + 7) // 8 * 8
    lst, image = L.lora_grad_list_build(entries(rows), groups)
    starts, chunks = unpack(lst, image)
    assert starts[0] == 0 and starts[-1] == lst.chunks and (np.diff(starts) >= 0).all()
    assert lst.most_chunks == np.diff(starts).max() and lst.empty == (np.diff(starts) == 0).sum()
    assert lst.separate == int(any(r[1] and r[2] for r in rows))
    for g in range(groups):
        assert (chunks["group"][starts[g]:starts[g + 1]] == g).all()
    seen = 0
    for a, out, n, dt, g in rows:
        e = 2 if dt else 4
        mine = chunks[(chunks["in"] >= a) & (chunks["in"] < a + n * e)]
        assert (np.diff(mine["in"].astype(np.int64)) == mine["count"][:-1].astype(np.int64) * e
                ).all()
        assert int(mine["count"].sum()) == n and (mine["dtype"] == dt).all()
        assert (mine["group"] == g).all()
        assert (mine["out"] - (out or a) == mine["in"] - a).all()
        if n:
            assert mine["in"][0] == a and (mine["count"] > 0).all()
        seen += len(mine)
    assert seen == lst.chunks


def build_status(rows, groups):
    try:
        L.lora_grad_list_build(entries(rows), groups)
        return 0
    except L.LoraError as e:
        return e.status


def test_list_refusals():
    ok = [(FAKE, 0, 100, 0, 0), (FAKE + 400, FAKE + 4000, 100, 1, 1)]
    assert build_status(ok, 2) == 0
    for rows, groups, want in (
            (ok, 0, _lib.LORA_E_SHAPE), (ok, (1 << 20) + 1, _lib.LORA_E_SHAPE),
            (ok, 1, _lib.LORA_E_ID), ([(FAKE, 0, 100, 0, -1)], 2, _lib.LORA_E_ID),
            ([(FAKE, 0, -1, 0, 0)], 1, _lib.LORA_E_SHAPE),
            ([(0, 0, 4, 0, 0)], 1, _lib.LORA_E_ARG),
            ([(FAKE, 0, 4, 2, 0)], 1, _lib.LORA_E_DTYPE),
            ([(FAKE + 2, 0, 4, 0, 0)], 1, _lib.LORA_E_ALIGN),
            ([(FAKE, FAKE + 4001, 4, 1, 0)], 1, _lib.LORA_E_ALIGN),
            ([(FAKE, 0, 100, 0, 0), (FAKE, 0, 100, 0, 0)], 1, _lib.LORA_E_ARG),      # twice
            ([(FAKE, 0, 100, 0, 0), (FAKE + 396, 0, 1, 0, 0)], 1, _lib.LORA_E_ARG),  # overlap
            ([(FAKE, FAKE + 4, 100, 0, 0)], 1, _lib.LORA_E_ARG),                     # shifted out
            ([(FAKE, FAKE + 4000, 100, 0, 0), (FAKE + 400, FAKE + 4000, 100, 0, 0)], 1,
             _lib.LORA_E_ARG)):                                                      # one out
        assert build_status(rows, groups) == want, rows
    assert build_status([(FAKE, FAKE, 4, 0, 0), (0, 0, 0, 0, 0)], 1) == 0   # in place; empty


def test_call_refusals():
    lst, _ = L.lora_grad_list_build(entries([(FAKE, 0, 100, 0, 0)]), 1)

    class Grads:
        struct, image = lst, FAKE

    need = L.lora_clip_grads_workspace_bytes(Grads)

    def status(max_norm=1.0, norms=FAKE, ws=FAKE, n=need, image=FAKE):
        Grads.image = image
        try:
            L.lora_clip_grads(Grads, max_norm, norms, ws, n, stream=0)
            return 0
        except L.LoraError as e:
            return e.status

    assert status(-1.0) == status(float("nan")) == _lib.LORA_E_ARG
    assert status(norms=None) == status(ws=None) == status(image=None) == _lib.LORA_E_ARG
    assert status(n=need - 1) == _lib.LORA_E_WORKSPACE
    assert status(norms=FAKE + 4) == status(ws=FAKE + 8) == status(image=FAKE + 8) == \
        _lib.LORA_E_ALIGN
    lst.chunks = 2                                    # not what the image holds
    assert status() == _lib.LORA_E_ARG


def test_tensors_that_a_list_refuses():
    t = torch.zeros(8)
    for a, k, want in (([t], {}, _lib.LORA_E_ARG), ([], {}, _lib.LORA_E_ARG),
                       ([t.half()], {}, _lib.LORA_E_DTYPE),
                       ([t], {"groups": [0, 1]}, _lib.LORA_E_SHAPE),
                       ([t], {"outs": []}, _lib.LORA_E_SHAPE),
                       ([t], {"outs": [t.bfloat16()]}, _lib.LORA_E_DTYPE)):
        with pytest.raises(L.LoraError) as e:
            L.GradList(a, **k)
        assert e.value.status == want


def test_lists_past_a_grids_limit():
    """A workgroup of 256 threads a chunk, and a grid holds less than 2^32 threads."""
    lib = L.lib()

    def size(counts):
        a = entries([(FAKE + (i << 48), 0, n, 1, 0) for i, n in enumerate(counts)])
        return lib.lora_grad_list_bytes(a.ctypes.data, len(a), 1)

    most = ((1 << 24) - 1) * 32768
    assert size([most]) == 32 * ((1 << 24) - 1) + 32
    assert size([most, 1]) == size([most + 1]) == size([1 << 40] * 9) == _lib.LORA_E_SHAPE
    assert size([most - 1, 1]) == _lib.LORA_E_SHAPE      # two chunks that are not full


def test_a_lists_gpu(monkeypatch):
    """A list is clipped on its tensors' GPU, whichever is the current one."""
    lst, _ = L.lora_grad_list_build(entries([(FAKE, 0, 100, 0, 0)]), 1)
    now, calls = [0], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, now[0] = now[0], self.device.index

        def __exit__(self, *_):
            now[0] = self.before

    class Grads:
        struct, image, device = lst, FAKE, torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(_lib, "_clip_grads", lambda *a: calls.append(now[0]))
    L.lora_clip_grads(Grads, 1.0, FAKE, FAKE, 1 << 20)
    now[0] = 1
    L.lora_clip_grads(Grads, 1.0, FAKE, FAKE, 1 << 20)
    assert calls == [1, 1] and now == [1]
    with pytest.raises(L.LoraError):                  # the norms lie elsewhere
        L.lora_clip_grads(Grads, 1.0, torch.zeros(4), FAKE, 1 << 20)
