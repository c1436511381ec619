"""Gradients of the adapters' delta against 64 bits: every rank block, sizes off every
tile, slices, rows of one adapter each to one adapter for all, rows without one,
untouched slots, runs that are cut, exact integers, in place, sums added to a start,
extreme values, far offsets, streams and replayed graphs; and the forward path's
differences."""
import numpy as np
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import HALF_STEP, TORCH, within
from delta_helpers import batch, delta64, run_delta
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def check(s, got, label, dx_in=True, start=None):
    want = delta64(s)
    used = sorted(set(s["ids"].tolist()) - {-1})
    idle = [a for a in range(s["A"].shape[0]) if a not in used]
    if "dx" in got:
        value, bound = want["dx"]
        if dx_in:
            value = value + s["dx_in"].double()
            bound = bound + 2.0 ** -24 * value.abs()
        within(got["dx"], value, bound, s["dtype"], f"{label}: dx")
    for k in ("dA", "dB"):
        if k not in got:
            continue
        value, bound = want[k][0] + (start or 0.0), want[k][1]
        bound = bound + 2.0 ** -24 * value.abs()
        within(got[k][used], value[used], bound[used], "f32", f"{label}: {k}")
        rest = got[k][idle]
        assert (rest.isnan() if start is None else rest == start).all(), f"{label}: idle {k}"


def some_ids(kind, T, slots, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(T, slots - 1)
    if kind == "each":
        return np.arange(T) % slots
    if kind == "none":
        return np.full(T, -1)
    if kind == "runs":
        return np.sort(rng.integers(-1, slots, T))
    return rng.integers(-1, slots, T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128, 136])
def test_ranks(dtype, R):
    for k, (T, K, outs) in enumerate(((1, 64, [64]), (70, 136, [200, 72]), (131, 520, [264]))):
        for kind in ("mixed", "one"):
            s = batch(R + k, dtype, some_ids(kind, T, 3, k), K, outs, 3, R)
            check(s, run_delta(s), f"R={R} T={T} {kind}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,outs", [(8, [8]), (16, [8, 24, 8]), (264, [1032]), (1032, [72, 64]),
                                    (2056, [520, 8, 16, 32, 64, 128, 8, 40]), (4096, [1024]),
                                    (72, [4104])])
def test_widths(dtype, K, outs):
    for k, (T, kind) in enumerate(((1, "one"), (65, "mixed"), (200, "runs"), (40, "each"))):
        s = batch(K + k, dtype, some_ids(kind, T, 7, k), K, outs, 7, 16)
        check(s, run_delta(s), f"K={K} {outs} T={T} {kind}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_integers_are_exact(dtype):
    """Products and sums of small whole numbers have no rounding in fp32 (|u| <= 4 64, sums
    below 2^24): every element is the exact one."""
    for k, (T, K, outs, R, kind) in enumerate(((300, 64, [64, 32], 16, "mixed"),
                                               (513, 128, [72], 40, "one"),
                                               (64, 64, [64], 8, "each"))):
        s = batch(k, dtype, some_ids(kind, T, 5, k), K, outs, 5, R, integer=True)
        got, want = run_delta(s), delta64(s)
        used = sorted(set(s["ids"].tolist()) - {-1})
        for name in ("dA", "dB"):
            assert torch.equal(got[name][used].double(), want[name][0][used]), (k, name)
        dx = (want["dx"][0] + s["dx_in"].double()).to(TORCH[dtype])
        assert torch.equal(got["dx"], dx), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_runs(dtype):
    """One adapter of many rows (cut into pieces whose partials are added), next to short ones."""
    rng = np.random.default_rng(3)
    ids = np.where(rng.random(5000) < 0.85, 2, rng.integers(-1, 6, 5000))
    s = batch(1, dtype, ids, 136, [72], 6, 16)
    desc = L.make_desc(dtype, 6, 16, 136, [72])
    assert L.lora_delta_backward_plan(desc, ids)[0].partials > 2
    check(s, run_delta(s), "long")
    a, b = run_delta(s), run_delta(s)
    assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)
    check(s, run_delta(s, start=0.5), "long, added", start=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forms(dtype):
    ids = some_ids("mixed", 150, 4, 9)
    s = batch(2, dtype, ids, 264, [136, 64], 4, 24)
    full = run_delta(s)
    check(s, full, "full")
    check(s, run_delta(s, dx_in=False), "no dx_in", dx_in=False)
    only = run_delta(s, grads=False)
    assert list(only) == ["dx"] and torch.equal(only["dx"], full["dx"])
    only = run_delta(s, dx=False)
    assert list(only) == ["dA", "dB"]
    assert all(torch.equal(only[k].view(torch.int32), full[k].view(torch.int32)) for k in only)
    check(s, run_delta(s, start=-2.0), "added", start=-2.0)
    t = dict(s, dx_in=s["dx_in"].clone())
    assert torch.equal(run_delta(t, inplace=True)["dx"], full["dx"])
    none = batch(3, dtype, np.full(70, -1), 264, [136, 64], 4, 24)
    got = run_delta(none)
    assert torch.equal(got["dx"], none["dx_in"]) and got["dA"].isnan().all()
    assert (run_delta(none, dx_in=False)["dx"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_stay_with_their_rows(dtype):
    """A row with an infinity or a NaN spoils its adapter's sums and its own dx, nothing else."""
    ids = some_ids("mixed", 200, 4, 1)
    s = batch(4, dtype, ids, 136, [72], 4, 16)
    clean = run_delta(s)
    for name in ("x", "dy"):
        for v in (float("inf"), float("nan")):
            t = dict(s, **{name: s[name].clone()})
            row = int(np.nonzero(ids == 2)[0][3])
            t[name][row, 5] = v
            got = run_delta(t)
            others = [a for a in range(4) if a != 2]
            assert torch.equal(got["dA"][others], clean["dA"][others])
            assert torch.equal(got["dB"][others], clean["dB"][others])
            assert not got["dA"][2].isfinite().all() or not got["dB"][2].isfinite().all()
            rows = [i for i in range(200) if i != row]
            assert torch.equal(got["dx"][rows], clean["dx"][rows])
            assert torch.equal(got["dx"][row].isfinite(), clean["dx"][row].isfinite()) == (
                name == "x")
    # a slot that no row names is not read
    t = dict(s, A=s["A"].clone(), B=s["B"].clone(), ids=np.where(ids == 1, -1, ids))
    t["A"][1], t["B"][1] = float("nan"), float("inf")
    got = run_delta(t)
    assert got["dx"].isfinite().all() and got["dA"][[0, 2, 3]].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_values(dtype):
    """Gradients of 2^-60 and of 2^60 keep all their bits."""
    for k, scale in enumerate((2.0 ** -60, 2.0 ** 60)):
        s = batch(5 + k, dtype, some_ids("runs", 100, 3), 136, [72], 3, 16)
        s["dy"] = s["dy"] * scale
        check(s, run_delta(s, dx_in=False), f"{scale}", dx_in=False)


def test_far_offsets():
    """Rows past 2^32 bytes and slots past 2^31 values."""
    T, K = 280_000, 8192
    ids = np.full(T, -1, np.int32)
    rows = [0, 1000, 262_143, 262_144, T - 2, T - 1]
    ids[rows] = [0, 1, 0, 1, 1, 0]
    g = torch.Generator(device="cuda").manual_seed(0)
    make = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    s = {"ids": ids, "x": torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"),
         "dy": make(T, 64), "A": make(2, 1, 16, K), "B": make(2, 64, 16), "outs": [64],
         "dx_in": torch.full((T, K), 2.0, dtype=torch.bfloat16, device="cuda"), "dtype": "bf16"}
    s["x"][rows] = make(len(rows), K)
    got = run_delta(s)
    few = dict(s, ids=ids[rows], x=s["x"][rows], dy=s["dy"][rows], dx_in=s["dx_in"][rows])
    check(few, dict(got, dx=got["dx"][rows]), "far")
    ids_gpu = torch.from_numpy(ids).cuda()
    assert (got["dx"][ids_gpu < 0] == 2).all()
    del s, got
    slots = 40_000   # 40000 x 16 x 4096 values of A: past 2^31
    s = {"ids": np.array([0, slots - 1, -1, slots - 1], np.int32), "x": make(4, 4096),
         "dy": make(4, 64), "A": torch.empty(slots, 1, 16, 4096, dtype=torch.bfloat16,
                                             device="cuda"),
         "B": torch.empty(slots, 64, 16, dtype=torch.bfloat16, device="cuda"), "outs": [64],
         "dx_in": make(4, 4096), "dtype": "bf16"}
    ends = [0, slots - 1]
    s["A"][ends], s["B"][ends] = make(2, 1, 16, 4096), make(2, 64, 16)
    got = run_delta(s)
    few = dict(s, A=s["A"][ends], B=s["B"][ends],
               ids=np.array([0, 1, -1, 1], np.int32))
    check(few, {"dx": got["dx"], "dA": got["dA"][ends], "dB": got["dB"][ends]}, "far slots")
    assert got["dA"][1:-1].isnan().all()


def test_against_differences_of_the_forward_path():
    """The scalar <dy, lora_apply(x)> is linear in x, in A and in B: its difference along any
    direction is the gradient's product with it."""
    ids = some_ids("mixed", 90, 3, 4)
    s = batch(6, "f32", ids, 136, [72, 40], 3, 16)
    got = run_delta(s, dx_in=False)
    pool = L.LoraPool("f32", 3, 16, 136, [72, 40])
    g = torch.Generator(device="cuda").manual_seed(1)

    def value(x, A, B):
        pool.A.copy_(A.flatten())
        pool.B.copy_(B.flatten())
        y = torch.zeros_like(s["dy"])
        pool.apply(x, y, ids)
        return (y.double() * s["dy"].double())

    for k, (name, grad) in enumerate((("x", "dx"), ("A", "dA"), ("B", "dB"))):
        at = [s["x"], s["A"], s["B"]]
        step = torch.randn(at[k].shape, generator=g, device="cuda")
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + step, at[k] - step
        a, b = value(*up), value(*down)
        d = got[grad].double()
        used = torch.from_numpy(ids).cuda() >= 0
        terms = (d * step.double())[used] if name == "x" else (d * step.double())
        assert name == "x" or set(ids.tolist()) >= {0, 1, 2}
        # three fp32 sums of up to 136 terms on either side
        tol = 600 * 2.0 ** -23 * (a.abs().sum() + b.abs().sum() + terms.abs().sum())
        assert abs((a.sum() - b.sum()) / 2 - terms.sum()) <= tol, name


def test_streams_and_replays():
    ids = some_ids("mixed", 300, 5, 2)
    s = batch(7, "bf16", ids, 520, [264, 72], 5, 32)
    want = run_delta(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run_delta(s)
    st.synchronize()
    for k in want:
        assert torch.equal(want[k].view(torch.uint8), got[k].view(torch.uint8)), k
    desc = L.make_desc("bf16", 5, 32, 520, s["outs"])
    plan, image = L.lora_delta_backward_plan(desc, ids)
    image = torch.from_numpy(image).cuda()
    n = L.lora_delta_backward_workspace_bytes(desc, 300)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dA, dB = torch.empty_like(s["x"]), want["dA"].clone(), want["dB"].clone()
    call = lambda: L.lora_delta_backward(  # noqa: E731
        desc, s["A"], s["B"], s["x"], s["dy"], s["dx_in"], dx, dA, dB, 300, plan, image, False, ws,
        n)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        new = batch(20 + k, "bf16", ids, 520, [264, 72], 5, 32)
        for name in ("x", "dy", "A", "B", "dx_in"):
            s[name].copy_(new[name])
        call()
        keep = [t.clone() for t in (dx, dA, dB)]
        for t in (dx, dA, dB):
            t.zero_()
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, dA, dB), keep)), k
