"""The decoder-block operators (norm, linear, gated feed-forward block and its
gradients) against plain implementations in 64 bits, at the sizes where they
can go wrong: one token, one column past a tile, reductions that end inside a
tile step, odd output widths, K splits, in-place forms, empty batches, rows of
zeros, infinities and NaN; exact on integers; replayed graphs; other streams."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import (HALF_STEP, TORCH, act64, gen, normal, operand, product64,
                           product_bound, run_backward, run_gated, run_linear, slope64, within)
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


# -------------------------------------------------------------------- norm

def _norm(x, residual, weight, eps, dtype, out8=True, out=True, inplace=False, stream=None):
    T, H = x.shape
    d = L.make_norm_desc(dtype, H, eps)
    total = None if residual is None else (residual if inplace else torch.empty_like(x))
    o = (x if inplace else torch.empty_like(x)) if out else None
    o8 = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda") if out8 else None
    sc = torch.empty(T, device="cuda") if out8 else None
    L.lora_add_rms_norm(d, x, residual, weight, total, o, o8, sc, T, stream=stream)
    return total, o, o8, sc


def _norm_inputs(seed, T, H, dtype, residual=True):
    g = gen(seed)
    gain = torch.exp(torch.randn(H, generator=g, device="cuda"))
    x = (torch.randn((T, H), generator=g, device="cuda") * gain).to(TORCH[dtype])
    r = (torch.randn((T, H), generator=g, device="cuda") * 2 * gain).to(TORCH[dtype])
    return x, r if residual else None, (1 + 0.2 * normal(g, (H,), "f32")).to(TORCH[dtype])


def _norm64(t, weight, eps):
    t = t.double()
    return t / (t.square().mean(1, keepdim=True) + eps).sqrt() * weight.double()


def _check_norm(x, r, w, eps, dtype, got, label):
    total, out, out8, scale = got
    t = x
    if r is not None:
        t = (x.double() + r.double()).to(TORCH[dtype])   # one rounding
        assert torch.equal(total, t), f"{label}: sum"
    n = _norm64(t, w, eps)
    # t * rstd * weight in fp32: the statistic's rounding and two products'
    slack = 4 * 2.0 ** -24
    if out is not None:
        within(out, n, slack * n.abs(), dtype, f"{label}: out")
    if out8 is not None:
        want = (n.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        assert ((scale.double() - want).abs() <= (slack + 2.0 ** -24) * want).all(), label
        v = out8.double() * scale.double()[:, None]
        # half a step of e4m3 (2^-10 where it is subnormal), two more fp32 roundings
        b = torch.maximum(HALF_STEP["e4m3"] * n.abs(), scale.double()[:, None] * 2.0 ** -10)
        assert ((v - n).abs() <= b * (1 + 2.0 ** -18) + 8 * 2.0 ** -24 * n.abs()).all(), label


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [8, 64, 136, 512, 1032, 4096, 8192, 8200, 20480, 32768])
def test_norm_sizes(dtype, H):
    for k, T in enumerate((1, 3, 65)):
        for residual in (False, True):
            x, r, w = _norm_inputs(100 * H + k, T, H, dtype, residual)
            for out8, out in ((True, True), (True, False), (False, True)):
                got = _norm(x, r, w, 1e-5, dtype, out8=out8, out=out)
                _check_norm(x, r, w, 1e-5, dtype, got, f"T={T} H={H} res={residual}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(dtype):
    x, r, w = _norm_inputs(5, 37, 1032, dtype)
    x0, r0 = x.clone(), r.clone()
    got = _norm(x, r, w, 1e-6, dtype, inplace=True)
    _check_norm(x0, r0, w, 1e-6, dtype, got, "in place")


def test_norm_rows_of_zeros_infinities_and_nan():
    x, r, w = _norm_inputs(6, 6, 264, "bf16")
    x[0] = 0
    r[0] = 0
    x[1, 7] = float("inf")
    x[2, 250] = float("nan")
    x[3] = 3e38      # squares past fp32
    r[3] = 0
    x[4] = 1e-30     # squares below fp32
    r[4] = 0
    total, out, out8, scale = _norm(x, r, w, 1e-5, "bf16")
    t = (x.double() + r.double()).to(torch.bfloat16)
    for i in (0, 3, 4, 5):
        one = slice(i, i + 1)
        _check_norm(x[one], r[one], w, 1e-5, "bf16",
                    (total[one], out[one], out8[one], scale[one]), f"row {i}")
    assert scale[0].item() == 2.0 ** -126 and not out8[0].float().any()
    assert torch.equal(total[:2], t[:2])
    for i in (1, 2):
        assert torch.isnan(scale[i]) and torch.isnan(out[i].float()).any()
        assert torch.isnan(out8[i].float()).all()


def test_norm_long_batch_past_32_bit_offsets():
    T, H = 140000, 32768     # 4.6e9 elements
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x[-2:] = normal(gen(7), (2, H), "bf16")
    got = _norm(x, None, w, 1e-5, "bf16", out8=False)
    _check_norm(x[-2:].clone(), None, w, 1e-5, "bf16", (None, got[1][-2:], None, None), "tail")
    assert not got[1][:2].any()


# ------------------------------------------------------------------ linear

def _check_linear(T, K, O, dtype, od, act, bias, delta, residual, seed, inplace=False):
    g = gen(seed)
    x, xs = operand(g, T, K, dtype, 1.0)
    w, ws = operand(g, O, K, dtype, K ** -0.5)
    b = normal(g, (O,), od, 0.5) if bias else None
    d = normal(g, (T, O), od, 0.3) if delta else None
    r = normal(g, (T, O), od) if residual else None
    z, mag = product64(x, w, xs, ws)
    for t in (b, d):
        if t is not None:
            z, mag = z + t.double(), mag + t.double().abs()
    want = act64(act, z)
    bound = 1.2 * product_bound(K, mag, (dtype, od) == ("e4m3", "bf16")) + 2.0 ** -20 * z.abs() * (act != "none")
    if r is not None:
        want = want + r.double()
        bound = bound + 2.0 ** -23 * (want.abs() + r.double().abs())
    got = run_linear(x, w, xs, ws, b, d, r, dtype, od, act, out=r if inplace else None)
    within(got, want, bound, od, f"linear {T}x{K}x{O} {dtype}->{od} {act}")


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T", [1, 2, 15, 17, 64, 129, 300])
def test_linear_sizes(dtype, od, T):
    unit = 16 if dtype == "e4m3" else 8
    for k, (K, O) in enumerate(((unit, 1), (64, 17), (264 // unit * unit, 33), (1040, 251),
                                (528, 256), (2048, 129))):
        _check_linear(T, K, O, dtype, od, "none", k % 2 == 0, k % 3 == 0, k % 2 == 1,
                      1000 * T + k)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype,od", TYPES)
def test_linear_activations(dtype, od, act):
    for k, (T, K, O) in enumerate(((5, 272, 200), (150, 144, 391))):
        _check_linear(T, K, O, dtype, od, act, True, True, True, 70 + k, inplace=k == 0)


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T,K,O", [(700, 1040, 3000), (2050, 528, 4100), (1300, 4112, 2064),
                                   (4097, 192, 2049)])
def test_linear_large(dtype, od, T, K, O):
    _check_linear(T, K, O, dtype, od, "silu", True, False, True, T + O)


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T,K,O", [(1, 4096, 100), (9, 8208, 37), (70, 16384, 64),
                                   (33, 2064, 520), (257, 6160, 300), (16, 14336, 4096)])
def test_linear_long_reductions(dtype, od, T, K, O):
    _check_linear(T, K, O, dtype, od, "gelu_tanh", True, True, True, T + K)


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T,K,O", [(3, 528, 77), (65, 1040, 130), (1100, 400, 3001),
                                   (2304, 272, 2560), (20, 8192, 48)])
def test_linear_exact_integers(dtype, od, T, K, O):
    g = gen(T + K)
    x, xs = operand(g, T, K, dtype, 1.0, integer=True)
    w, ws = operand(g, O, K, dtype, 1.0, integer=True)
    r = torch.randint(-8, 9, (T, O), generator=g, device="cuda").to(TORCH[od])
    z = x.double() @ w.double().t() + r.double()
    got = run_linear(x, w, xs, ws, None, None, r, dtype, od, "none")
    assert torch.equal(got, z.to(TORCH[od]))


# tile shapes, each with and without a K split (the plan would take some of
# them at large sizes alone)
SHAPES = ["0,1", "0,3", "1,1", "1,2", "2,1", "2,3", "3,1", "3,3"]


@pytest.mark.parametrize("plan", SHAPES)
@pytest.mark.parametrize("dtype,od", TYPES)
def test_every_shape(dtype, od, plan, monkeypatch):
    monkeypatch.setenv("LORA_GEMM_PLAN", plan)
    unit = 16 if dtype == "e4m3" else 8
    for k, (T, K, O) in enumerate(((1, unit, 17), (255, 64, 255), (257, 272, 513), (600, 1040, 301),
                                   (300, 2064, 260), (513, 384, 777))):
        _check_linear(T, K, O, dtype, od, "none", k % 2 == 0, k % 3 == 0, k % 2 == 1, k)
        I = max(unit, O // unit * unit)
        _check_gated(T, K, I, dtype, od, "silu", k % 2 == 0, k % 3 == 0, k)
    g = gen(2)
    for T, K, O in ((300, 528, 270), (130, 64, 1000)):
        x, xs = operand(g, T, K, dtype, 1.0, integer=True)
        w, ws = operand(g, O, K, dtype, 1.0, integer=True)
        got = run_linear(x, w, xs, ws, None, None, None, dtype, "f32" if dtype == "f32" else od,
                         "none")
        assert torch.equal(got, (x.double() @ w.double().t()).to(got.dtype))


@pytest.mark.parametrize("T", [1, 15, 16, 17, 32])
@pytest.mark.parametrize("dtype,od", TYPES)
def test_few_rows(dtype, od, T, monkeypatch):
    """The kernel of up to 32 rows: reductions of less than a step, that end inside
    one, and of more steps than its waves take at once; more workgroups than the
    compute units hold; columns that end inside a tile; NaN around the operands."""
    monkeypatch.setenv("LORA_GEMM_PLAN", "4,1")
    unit, es = {"bf16": (8, 2), "e4m3": (16, 1), "f32": (8, 4)}[dtype]
    g = gen(500 + T)
    for k, (K, O) in enumerate(((unit, 1), (64, 17), (272, 513), (2064, 250), (8208, 40),
                                (144, 16391))):
        _check_linear(T, K, O, dtype, od, "gelu", k % 2 == 0, k % 3 == 0, k % 2 == 1, T + k)
        _check_gated(T, K, (O + 15) // 16 * 16, dtype, od, "silu", k % 2 == 0, k % 3 != 1, T + k)
        x, xs = operand(g, T, K, dtype, 1.0, integer=True)
        w, ws = operand(g, O, K, dtype, 1.0, integer=True)
        around = []
        for t in (x, w):
            n = t.numel() * es
            buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")  # NaN in every type
            view = buf[240:240 + n]
            view.copy_(t.contiguous().view(torch.uint8).reshape(-1))
            around.append(view.view(t.dtype).view(t.shape))
        got = run_linear(*around, xs, ws, None, None, None, dtype, od, "none")
        assert torch.equal(got, (x.double() @ w.double().t()).to(got.dtype)), (T, K, O)


def test_linear_inf_and_nan_stay_in_their_rows():
    # K ends inside a tile step and T inside a tile: what lies past a row's end
    # is the next row, whose infinities and NaN must not come in
    g = gen(3)
    for T, K, O in ((40, 72, 50), (300, 1032, 300)):
        x, w = normal(g, (T, K), "bf16"), normal(g, (O, K), "bf16", K ** -0.5)
        x[7, 0] = float("inf")
        x[9, K - 1] = float("nan")
        w[11, 3] = float("nan")
        got = run_linear(x, w, None, None, None, None, None, "bf16", "f32", "none")
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        cols = torch.ones(O, dtype=torch.bool, device="cuda")
        rows[[7, 9]] = False
        cols[11] = False
        assert torch.isnan(got[:, 11]).all() and torch.isnan(got[9]).all()
        assert not torch.isfinite(got[7]).any()
        z, mag = product64(x[rows], w[cols])
        within(got[rows][:, cols], z, product_bound(K, mag), "f32", "finite part")


@pytest.mark.parametrize("plan", [None, "0,1", "0,3", "1,1", "1,2", "2,1", "2,2", "3,1"])
@pytest.mark.parametrize("dtype,od", TYPES)
def test_rows_off_the_cache_lines(dtype, od, plan, monkeypatch):
    """Every distance of a row from a cache line, by odd row lengths and by
    operands that start 16 bytes apart; what lies around them is not a number."""
    if plan:
        monkeypatch.setenv("LORA_GEMM_PLAN", plan)
        monkeypatch.setenv("LORA_GEMM_LINES", "1")
    es = {"bf16": 2, "e4m3": 1, "f32": 4}[dtype]
    g = gen(11)

    def placed(t, chunks):
        n = t.numel() * es
        buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")   # NaN in every type
        view = buf[128 + 16 * chunks:128 + 16 * chunks + n]
        view.copy_(t.contiguous().view(torch.uint8).reshape(-1))
        return view.view(t.dtype).view(t.shape)

    for k, (T, chunks, O) in enumerate(((1, 1, 16), (5, 7, 32), (33, 13, 48), (70, 33, 96),
                                        (130, 70, 144), (64, 66, 80))):
        K = chunks * 16 // es
        K = max(8, K // 8 * 8)    # (fp32 rows are multiples of 32 bytes)
        for da, db in ((0, 0), (k + 1, 0), (3, (k + 5) % 8)):
            x, xs = operand(g, T, K, dtype, 1.0, integer=True)
            w, ws = operand(g, 2 * O, K, dtype, 1.0, integer=True)
            z = x.double() @ w.double().t()
            x, w = placed(x, da), placed(w, db)
            got = run_linear(x, w, xs, ws, None, None, None, dtype, od, "none")
            assert torch.equal(got, z.to(got.dtype)), (T, K, O, da, db)
            got, _ = run_gated(x, w, xs, ws, None, False, dtype, od, "none")
            assert torch.equal(got, (z[:, :O] * z[:, O:]).to(got.dtype)), (T, K, O, da, db)


def test_linear_output_past_32_bit_offsets():
    T, K, O = 70001, 64, 16387     # 4.6 GB of fp32 outputs, odd rows
    g = gen(4)
    x, w = normal(g, (T, K), "bf16"), normal(g, (O, K), "bf16", K ** -0.5)
    got = run_linear(x, w, None, None, None, None, None, "bf16", "f32", "none")
    for rows in (slice(0, 3), slice(65530, 65540), slice(T - 3, T)):
        z, mag = product64(x[rows], w)
        within(got[rows], z, product_bound(K, mag), "f32", f"rows {rows}")


def test_empty_batches():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), normal(gen(1), (48, 64), "bf16")
    assert run_linear(x, w, None, None, None, None, None, "bf16", "bf16", "none").shape == (0, 48)
    out, pre = run_gated(x, w, None, None, None, True, "bf16", "bf16", "silu")
    assert out.shape == (0, 24)
    for dtype in ("bf16", "f32"):
        e = lambda n: torch.empty((0, n), dtype=TORCH[dtype], device="cuda")  # noqa: E731
        _, _, dw = run_backward(e(24), e(48), e(64), w.to(TORCH[dtype]), "silu", dtype)
        assert torch.equal(dw, torch.zeros_like(dw))


# ------------------------------------------------------------------- gated

def _check_gated(T, K, I, dtype, od, act, delta, keep, seed):
    g = gen(seed)
    x, xs = operand(g, T, K, dtype, 1.0)
    w, ws = operand(g, 2 * I, K, dtype, K ** -0.5)
    d = normal(g, (T, 2 * I), od, 0.3) if delta else None
    z, mag = product64(x, w, xs, ws)
    if d is not None:
        z, mag = z + d.double(), mag + d.double().abs()
    e = product_bound(K, mag, (dtype, od) == ("e4m3", "bf16"))
    got, pre = run_gated(x, w, xs, ws, d, keep, dtype, od, act)
    label = f"gated {T}x{K}x{I} {dtype}->{od} {act}"
    if keep:
        within(pre, z, e, od, label + " pre")
    v, u = act64(act, z[:, :I]), z[:, I:]
    ev = 1.2 * e[:, :I] + 2.0 ** -20 * z[:, :I].abs()
    within(got, v * u, ev * u.abs() + (v.abs() + ev) * e[:, I:] + 2.0 ** -23 * (v * u).abs(), od,
           label)


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T", [1, 2, 16, 17, 65, 130])
def test_gated_sizes(dtype, od, T):
    for k, (K, I) in enumerate(((16, 16), (64, 48), (528, 272), (1040, 64), (2064, 144))):
        _check_gated(T, K, I, dtype, od, "silu", k % 2 == 0, k % 3 != 1, 50 * T + k)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype,od", TYPES)
def test_gated_activations(dtype, od, act):
    _check_gated(7, 272, 208, dtype, od, act, True, True, 8)
    _check_gated(200, 144, 400, dtype, od, act, True, True, 9)


@pytest.mark.parametrize("dtype,od", TYPES)
@pytest.mark.parametrize("T,K,I", [(777, 1040, 528), (2050, 528, 2064), (1500, 2064, 1424),
                                   (1, 4096, 2048), (40, 8208, 160)])
def test_gated_large(dtype, od, T, K, I):
    _check_gated(T, K, I, dtype, od, "silu", T % 2 == 1, T % 3 == 0, T + I)


def test_gated_units_of_eight():
    # bf16 and fp32 take sizes that are multiples of 8 alone
    for dtype in ("bf16", "f32"):
        for T, K, I in ((3, 8, 8), (70, 1032, 520), (600, 72, 1304)):
            _check_gated(T, K, I, dtype, dtype, "gelu", True, True, T)


# ---------------------------------------------------------------- backward

def _check_backward(T, K, I, dtype, act, seed, dx=True, dw=True, inplace=False):
    g = gen(seed)
    x, w = normal(g, (T, K), dtype), normal(g, (2 * I, K), dtype, K ** -0.5)
    pre, dout = normal(g, (T, 2 * I), dtype), normal(g, (T, I), dtype, 0.1)
    gate, up, d = pre[:, :I].double(), pre[:, I:].double(), dout.double()
    want = torch.cat([d * up * slope64(act, gate), d * act64(act, gate)], 1)
    # the curve's own error (2^-20 of the gate's size, the slope's terms below
    # 1.2 + |gate|) and the products'
    near = 2.0 ** -20 * torch.cat([(d * up).abs() * (1.2 + gate.abs()), d.abs() * gate.abs()], 1)
    label = f"backward {T}x{K}x{I} {dtype} {act}"
    dpre, gx, gw = run_backward(dout, pre.clone() if inplace else pre, x, w, act, dtype, dx, dw,
                                dpre=None)
    if inplace:
        p2 = pre.clone()
        again = run_backward(dout, p2, x, w, act, dtype, dx, dw, dpre=p2)
        assert torch.equal(again[0], dpre) and torch.equal(again[1], gx)
        assert torch.equal(again[2], gw)
    within(dpre, want, near, dtype, label + " dpre")
    # the products take dpre as it is stored
    s = dpre.double()
    if dx:
        m = s.abs() @ w.double().abs()
        within(gx, s @ w.double(), product_bound(2 * I, m), dtype, label + " dx")
    if dw:
        st = s.t().contiguous()
        m = st.abs() @ x.double().abs()
        within(gw, st @ x.double(), product_bound(T, m), dtype, label + " dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 7, 33, 64, 129, 257])
def test_backward_sizes(dtype, T):
    for k, (K, I) in enumerate(((8, 8), (64, 72), (520, 264), (136, 1032))):
        _check_backward(T, K, I, dtype, "silu", 10 * T + k, inplace=k == 1)


@pytest.mark.parametrize("plan", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_every_shape(dtype, plan, monkeypatch):
    monkeypatch.setenv("LORA_GEMM_PLAN", plan)
    for k, (T, K, I) in enumerate(((1, 8, 8), (31, 264, 136), (257, 520, 264), (600, 304, 72),
                                   (67, 72, 520))):
        _check_backward(T, K, I, dtype, "silu", 30 + k)


@pytest.mark.parametrize("pair", ["0,0,0", "0,2,1", "1,0,0", "1,1,3", "2,0,0", "2,3,1", "off"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_in_one_launch(dtype, pair, monkeypatch):
    """Both products in one launch, every tile shape with and without K splits
    (bf16 rounds sums of another order: the bounds, not each other)."""
    monkeypatch.setenv("LORA_GRAD_PAIR", pair)
    for k, (T, K, I) in enumerate(((1, 8, 8), (31, 264, 136), (257, 520, 264), (600, 304, 72),
                                   (67, 72, 520), (1500, 40, 1600))):
        _check_backward(T, K, I, dtype, "silu", 60 + k, inplace=k == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_exact_integers(dtype):
    # relu over positive gates: dpre, and with it every product, is whole
    for T, K, I in ((3, 136, 72), (129, 264, 392), (1031, 520, 648)):
        g = gen(T)
        whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(  # noqa: E731
            TORCH[dtype])
        x, w, dout = whole(T, K), whole(2 * I, K), whole(T, I)
        pre = torch.cat([whole(T, I).abs() + 1, whole(T, I)], 1)
        dpre, gx, gw = run_backward(dout, pre, x, w, "relu", dtype)
        d = dout.double()
        want = torch.cat([d * pre[:, I:].double(), d * pre[:, :I].double()], 1)
        assert torch.equal(dpre.double(), want)
        assert torch.equal(gx, (want @ w.double()).to(TORCH[dtype]))
        assert torch.equal(gw, (want.t().contiguous() @ x.double()).to(TORCH[dtype]))


def test_backward_rows_past_the_end_stay_out():
    # the reduction over the tokens ends inside a step; what lies behind it in
    # memory is not a number
    for dtype in ("bf16", "f32"):
        for T in (5, 70):
            K, I = 72, 40
            g = gen(T)
            buf = lambda n: torch.full((T + 70, n), float("nan"), dtype=TORCH[dtype],  # noqa: E731
                                       device="cuda")
            x, pre, dout = buf(K), buf(2 * I), buf(I)
            for t in (x, pre, dout):
                t[:T] = normal(g, t[:T].shape, dtype)
            w = normal(g, (2 * I, K), dtype)
            dpre = buf(2 * I)
            _, gx, gw = run_backward(dout[:T], pre[:T], x[:T], w, "silu", dtype, dpre=dpre[:T])
            assert torch.isfinite(gx).all() and torch.isfinite(gw).all()
            assert torch.isnan(dpre[T:]).all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_activations(dtype, act):
    _check_backward(150, 200, 88, dtype, act, 5)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activations_at_the_ends_of_their_range(dtype, act):
    """Gates of zero, far values and infinities get the curve's limits, forward
    and backward; NaN stays."""
    inf, nan = float("inf"), float("nan")
    gate = [0.0, -0.0, 3e-39, 150.0, -150.0, 2.5e19, -2.5e19, 3e38, -3e38, inf, -inf, nan]
    I = 16
    pre = torch.ones((1, 2 * I), dtype=TORCH[dtype], device="cuda")
    pre[0, :len(gate)] = torch.tensor(gate).to(TORCH[dtype])
    one = torch.ones((1, I), dtype=TORCH[dtype], device="cuda")
    x = torch.zeros((1, 8), dtype=TORCH[dtype], device="cuda")
    w = torch.zeros((2 * I, 8), dtype=TORCH[dtype], device="cuda")
    dpre, _, _ = run_backward(one, pre, x, w, act, dtype, dx=False, dw=False)
    out, _ = run_gated(x, w, None, None, pre, False, dtype, dtype, act)
    z = pre[0, :len(gate)].double()
    value = torch.where(z > 100, z, torch.where(z < -100, torch.zeros_like(z), z / 2))
    slope = torch.where(z > 100, 1.0, torch.where(z < -100, 0.0, 0.5))
    if act == "relu":
        value = torch.where(z > 0, z, torch.zeros_like(z))
        slope = (z > 0).double()
    for got, want in ((out[0], value), (dpre[0, I:], value), (dpre[0, :I], slope)):
        got = got[:len(gate)]
        assert torch.isnan(got[-1])
        bound = 2.0 ** -20 + HALF_STEP[dtype]
        same = got[:-1].double() == want[:-1]
        assert (same | ((got[:-1].double() - want[:-1]).abs() <= bound * want[:-1].abs() +
                        2.0 ** -126)).all(), (act, got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,I", [(1030, 1032, 1304), (2500, 776, 520), (4099, 264, 136)])
def test_backward_large(dtype, T, K, I):
    _check_backward(T, K, I, dtype, "silu", T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_one_gradient_alone(dtype):
    _check_backward(100, 136, 72, dtype, "gelu_tanh", 6, dw=False)
    _check_backward(100, 136, 72, dtype, "gelu_tanh", 7, dx=False)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_backward_against_differences(act):
    """The kernels' gradients against central differences of the block's
    definition in 64 bits: L = sum(dout * out)."""
    T, K, I = 5, 16, 24
    g = gen(12)
    x, w = normal(g, (T, K), "f32"), normal(g, (2 * I, K), "f32", K ** -0.5)
    dout = normal(g, (T, I), "f32")

    def loss(xx, ww):
        z = xx @ ww.t()
        return (dout.double() * act64(act, z[:, :I]) * z[:, I:]).sum()

    x64, w64, h = x.double(), w.double(), 1e-5
    pre = (x64 @ w64.t()).float()
    _, gx, gw = run_backward(dout, pre, x, w, act, "f32")
    for got, base, f in ((gx, x64, lambda t: loss(t, w64)), (gw, w64, lambda t: loss(x64, t))):
        want = torch.empty_like(base)
        for i in range(base.numel()):
            step = torch.zeros(base.numel(), dtype=torch.float64, device="cuda")
            step[i] = h
            step = step.view_as(base)
            want.view(-1)[i] = (f(base + step) - f(base - step)) / (2 * h)
        # differences: h^2 of the third derivative; fp32 sums of some 50 terms of size 1
        assert (got.double() - want).abs().max() < 2e-5 * (1 + want.abs().max())


# ------------------------------------------------- streams, graphs, repeats

def _everything(seed, stream=None):
    g = gen(seed)
    T, K, I = 70, 520, 264
    x, r, w = normal(g, (T, K), "bf16"), normal(g, (T, K), "bf16"), normal(g, (K,), "bf16")
    wg, wd = normal(g, (2 * I, K), "bf16", 0.05), normal(g, (K, I), "bf16", 0.05)
    return x, r, w, wg, wd


def test_results_repeat_bit_for_bit():
    for T, K, O in ((1, 4096, 300), (300, 2064, 700), (2000, 528, 3000)):
        g = gen(T)
        x, w = normal(g, (T, K), "bf16"), normal(g, (O, K), "bf16", K ** -0.5)
        first = run_linear(x, w, None, None, None, None, None, "bf16", "f32", "silu")
        for _ in range(3):
            again = run_linear(x, w, None, None, None, None, None, "bf16", "f32", "silu")
            assert torch.equal(first, again)


def test_other_stream():
    x, r, w, wg, wd = _everything(1)
    want, _ = run_gated(x, wg, None, None, None, False, "bf16", "bf16", "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = run_gated(x, wg, None, None, None, False, "bf16", "bf16", "silu", stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_graph_replays():
    """Norm, gated block, down projection and the gradients in one graph,
    replayed with new inputs and eager work between the replays."""
    x, r, w, wg, wd = _everything(2)
    T, K, I = x.shape[0], x.shape[1], wg.shape[0] // 2
    dn, dg = L.make_norm_desc("bf16", K, 1e-5), L.make_gated_desc("bf16", "bf16", K, I, "silu")
    dl = L.make_linear_desc("bf16", "bf16", I, K)
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = dict(total=new(T, K), n=new(T, K), h=new(T, I), pre=new(T, 2 * I), y=new(T, K),
             dpre=new(T, 2 * I), dx=new(T, K), dw=new(2 * I, K))
    n = max(L.lora_gated_ffn_workspace_bytes(dg, T), L.lora_linear_workspace_bytes(dl, T),
            L.lora_gated_ffn_backward_workspace_bytes(dg, T), 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        L.lora_add_rms_norm(dn, x, r, w, o["total"], o["n"], None, None, T)
        L.lora_gated_ffn(dg, o["n"], wg, None, None, None, o["pre"], o["h"], T, ws, n)
        L.lora_linear(dl, o["h"], wd, None, None, None, None, o["total"], o["y"], T, ws, n)
        L.lora_gated_ffn_backward(dg, o["h"], o["pre"], o["n"], wg, o["dpre"], o["dx"], o["dw"],
                                  T, ws, n)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = gen(9)
    for k in range(4):
        x.copy_(normal(g, (T, K), "bf16"))
        r.copy_(normal(g, (T, K), "bf16"))
        for t in o.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = {a: t.clone() for a, t in o.items()}
        for t in o.values():
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for a, t in o.items():
            assert torch.equal(got[a], t), (k, a)
