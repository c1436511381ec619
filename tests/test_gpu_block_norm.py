"""lora_block_norm and its gradients against 64 bits: one element a thread to the
largest rows, with and without each part, in place, rows of zeros, infinities, NaN
and extreme sizes, sums over rows that start from a value, no rows, another stream,
replayed graphs."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import HALF_STEP, within
from block_norm_helpers import (E, inputs, join64, join_grad64, norm64, run_join,
                                run_join_backward)
from gpu_helpers import say

pytestmark = pytest.mark.gpu
HIDDEN = [8, 64, 520, 1032, 4096, 5128, 8192, 8200, 16384]


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def f64(s):
    return {k: None if v is None else v.double() for k, v in s.items()}


def check_forward(s, got, dtype, gate, alpha, beta, eps, post, pre, label):
    total, out, out8, scale = got
    d = f64(s)
    t, bound = join64(d["y"], d["residual"], d["gate"], d["post"] if post else None, alpha, beta,
                      eps)
    within(total, t, bound, dtype, f"{label}: sum")
    if not pre:
        return
    n = norm64(total.double(), d["pre"], eps)   # from the stream as it was rounded
    if out is not None:
        within(out, n, 4 * E * n.abs(), dtype, f"{label}: out")
    if out8 is not None:
        want = (n.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        assert ((scale.double() - want).abs() <= 5 * E * want).all(), label
        v = out8.double() * scale.double()[:, None]
        b = torch.maximum(HALF_STEP["e4m3"] * n.abs(), scale.double()[:, None] * 2.0 ** -10)
        assert ((v - n).abs() <= b * (1 + 2.0 ** -18) + 8 * E * n.abs()).all(), label


def check_backward(s, got, dtype, alpha, beta, eps, post, pre, stream_grad, label, start=0.0):
    d = f64(s)
    want = join_grad64(d["dout"] if pre else None, d["dsum"] if stream_grad else None, d["y"],
                       d["sum"], d["gate"], d["post"] if post else None, d["pre"], alpha, beta,
                       eps)
    for k, v in got.items():
        value, bound = want[k]
        # past the type's largest value the nearest value of the type is infinite: two
        # norms of rows of 2^-100 give gradients of 2^200
        far = value.abs() > 3.41e38
        assert torch.equal(v[far].double(), value[far].sign() * float("inf")), label
        v, value, bound = v[~far] if far.any() else v, value[~far] if far.any() else value, \
            bound[~far] if far.any() else bound
        if want[k][0].dim() == 1:   # added to the start, with a rounding of its own
            value = value + start
            bound = bound + E * value.abs()
        within(v, value, bound, "f32" if want[k][0].dim() == 1 else dtype, f"{label}: {k}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", HIDDEN)
def test_forward_sizes(dtype, H):
    for k, T in enumerate((1, 3, 65)):
        for gate, post, alpha, beta in (("none", True, 1.0, 1.0), ("channel", False, 0.5, 0.22),
                                        ("element", True, 1.0, -1.5), ("none", False, 1.0, 1.0)):
            s = inputs(10 * H + k, T, H, dtype, gate)
            for pre, out, out8 in ((True, True, True), (True, True, False), (True, False, True),
                                   (False, False, False)):
                got = run_join(s, dtype, gate, alpha, beta, post=post, pre=pre, out=out, out8=out8)
                check_forward(s, got, dtype, gate, alpha, beta, 1e-5, post, pre,
                              f"T={T} H={H} {gate} post={post} pre={pre}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", HIDDEN)
def test_backward_sizes(dtype, H):
    for k, T in enumerate((1, 3, 65)):
        for gate, post, pre, stream_grad, alpha, beta in (
                ("none", True, True, True, 1.0, 1.0), ("channel", False, True, False, 0.5, 0.22),
                ("element", True, True, True, 1.0, -1.5), ("channel", True, False, True, 1.0, 1.0),
                ("none", False, True, True, 1.0, 1.0), ("none", False, False, True, 2.0, 0.5)):
            s = inputs(20 * H + k, T, H, dtype, gate)
            got = run_join_backward(s, dtype, gate, alpha, beta, post=post, pre=pre,
                                    stream_grad=stream_grad)
            check_backward(s, got, dtype, alpha, beta, 1e-5, post, pre, stream_grad,
                           f"T={T} H={H} {gate} post={post} pre={pre}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(513, 264), (1500, 4096), (2049, 72)])
def test_backward_many_rows(dtype, T, H):
    """More rows than workgroups that keep sums; sums added to a start; frozen weights."""
    s = inputs(T, T, H, dtype, "channel")
    for start in (None, 3.0):
        got = run_join_backward(s, dtype, "channel", start=start)
        check_backward(s, got, dtype, 1.0, 1.0, 1e-5, True, True, True, f"T={T} start={start}",
                       start or 0.0)
    s = inputs(T + 1, T, H, dtype, "element")
    frozen = run_join_backward(s, dtype, "element", sums=False)
    full = run_join_backward(s, dtype, "element")
    for k, v in frozen.items():
        assert torch.equal(v, full[k]), k
    again = run_join_backward(s, dtype, "element")
    assert all(torch.equal(v, full[k]) for k, v in again.items()), "a second run differs"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [520, 4096, 8192, 16384])
def test_in_place(dtype, H):
    for gate in ("none", "channel", "element"):
        s = inputs(H, 9, H, dtype, gate)
        copy = lambda: {k: None if v is None else v.clone() for k, v in s.items()}  # noqa: E731
        want = run_join(s, dtype, gate)
        for a, b in zip(want, run_join(copy(), dtype, gate, inplace=True)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), gate
        want = run_join_backward(s, dtype, gate)
        got = run_join_backward(copy(), dtype, gate, inplace=True)
        for k in want:
            assert torch.equal(want[k], got[k]), (gate, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [520, 8192, 16384])
def test_outputs_that_are_not_wanted(dtype, H):
    for gate, post in (("channel", True), ("element", False), ("none", False)):
        s = inputs(H + 1, 9, H, dtype, gate)
        want = run_join_backward(s, dtype, gate, post=post)
        d = L.make_block_norm_desc(dtype, H, 1e-5, gate)
        n = L.lora_block_norm_backward_workspace_bytes(d, 9)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        y = s["y"] if post or gate != "none" else None
        for name in ("dy", "dresidual", "dpre"):
            out = torch.full_like(want[name], float("nan"))
            o = {name: out}
            L.lora_block_norm_backward(
                d, s["dout"], s["dsum"], y, s["sum"], s["gate"], s["post"] if post else None,
                s["pre"], o.get("dy"), o.get("dresidual"), None, None, o.get("dpre"), False, 9, ws,
                n)
            assert torch.equal(out, want[name]), (gate, post, name)


def test_plain_norm_is_the_same():
    """No gate, scales of one and no norm after the block: lora_add_rms_norm, bit for bit."""
    for dtype in ("bf16", "f32"):
        s = inputs(3, 33, 1032, dtype)
        total, out, out8, scale = run_join(s, dtype, "none", post=False)
        want = [torch.empty_like(v) for v in (total, out, out8, scale)]
        L.lora_add_rms_norm(L.make_norm_desc(dtype, 1032, 1e-5), s["y"], s["residual"], s["pre"],
                            *want, 33)
        for a, b in zip((total, out, out8, scale), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_at_the_ends(dtype):
    """Rows of zeros, of the smallest and largest numbers, with an infinity or a NaN: the
    other rows are as they are without them."""
    T, H = 12, 264
    s = inputs(8, T, H, dtype)
    for k in ("y", "residual", "sum"):
        s[k][1] = 0
        s[k][3] *= 2.0 ** -100
        s[k][5] *= 2.0 ** 100
    s["residual"][1] = 0
    got = run_join(s, dtype, "none", eps=0.0, beta=1.0)
    keep = [0, 2, 3, 4, 5] + list(range(6, T))
    part = {k: v if v is None or v.dim() == 1 else v[keep] for k, v in s.items()}
    check_forward(part, [v[keep] for v in got], dtype, "none", 1.0, 1.0, 0.0, True, True, "ends")
    grads = run_join_backward(s, dtype, "none", eps=0.0, sums=False, stream_grad=False)
    check_backward(part, {k: v[keep] for k, v in grads.items()}, dtype, 1.0, 1.0, 0.0, True, True,
                   False, "ends")
    bad = inputs(8, T, H, dtype)
    clean = run_join(bad, dtype, "none")
    cleang = run_join_backward(bad, dtype, "none", sums=False)
    bad["y"][1, 7], bad["residual"][2, 9] = float("nan"), float("inf")
    bad["dout"][1, 7], bad["sum"][2, 9], bad["dsum"][1, 0] = float("nan"), float("inf"), 1.0
    dirty = run_join(bad, dtype, "none")
    dirtyg = run_join_backward(bad, dtype, "none", sums=False)
    rows = [0] + list(range(3, T))
    for a, b in zip(clean, dirty):
        assert torch.equal(a[rows].view(torch.uint8), b[rows].view(torch.uint8))
    assert dirty[0][1].isnan().all() and dirty[3][1].isnan() and dirty[3][2].isnan()
    for k in cleang:
        assert torch.equal(cleang[k][rows], dirtyg[k][rows]), k
        assert dirtyg[k][1].isnan().any() and not dirtyg[k][2].isfinite().all()


def test_no_rows():
    d = L.make_block_norm_desc("bf16", 64, 1e-5, "channel")
    sums = [torch.full((64,), 7.0, device="cuda") for _ in range(3)]
    call = lambda acc: L.lora_block_norm_backward(  # noqa: E731
        d, *[None] * 9, *sums, acc, 0, None, 0)
    call(True)
    assert all((t == 7).all() for t in sums)
    call(False)
    assert all((t == 0).all() for t in sums)
    L.lora_block_norm(d, *[None] * 9, 0)


def test_another_stream_and_replays():
    s = inputs(4, 70, 1032, "bf16", "channel")
    want = run_join(s, "bf16", "channel")
    wantg = run_join_backward(s, "bf16", "channel")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run_join(s, "bf16", "channel")
        gotg = run_join_backward(s, "bf16", "channel")
    st.synchronize()
    for a, b in list(zip(want, got)) + [(wantg[k], gotg[k]) for k in wantg]:
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    T, H = s["y"].shape
    d = L.make_block_norm_desc("bf16", H, 1e-5, "channel")
    n = L.lora_block_norm_backward_workspace_bytes(d, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(s["y"]) for _ in range(3)]
    sums = [torch.empty(H, device="cuda") for _ in range(3)]

    def calls():
        L.lora_block_norm(d, s["y"], s["residual"], s["gate"], s["post"], s["pre"], outs[0],
                          outs[1], None, None, T)
        L.lora_block_norm_backward(d, s["dout"], s["dsum"], s["y"], outs[0], s["gate"], s["post"],
                                   s["pre"], outs[1], outs[2], *sums, False, T, ws, n)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        for name in ("y", "residual", "dout"):
            s[name].copy_(inputs(40 + k, T, H, "bf16", "channel")[name])
        calls()
        want = [t.clone() for t in outs + sums]
        for t in outs + sums:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + sums, want)), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(2048, 3600), (4100, 1024), (2500, 2048), (9000, 72), (530, 8192)])
def test_backward_by_rows_and_width(dtype, T, H):
    """Two pieces a thread, more workgroups for narrow rows, fewer for wide ones; a row's
    gradients are the same whether the sums are wanted or not."""
    s = inputs(T + H, T, H, dtype, "channel")
    got = run_join_backward(s, dtype, "channel", start=0.5)
    check_backward(s, got, dtype, 1.0, 1.0, 1e-5, True, True, True, f"T={T} H={H}", 0.5)
    bare = run_join_backward(s, dtype, "channel", sums=False)
    for k in ("dy", "dresidual"):
        assert torch.equal(bare[k], got[k]), k
