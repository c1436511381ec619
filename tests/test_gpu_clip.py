"""Gradient norms and clipping against 64 bits: sizes and addresses off every vector,
groups with and without elements, in place and into other arrays, norms that clip and
that do not, squares past fp32's range, infinities and NaN, replayed graphs."""
import math

import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import HALF_STEP, TORCH, gen
from gpu_helpers import say
from lora_adapter_pool_amd import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def clip(lst, max_norm, norms=None, stream=None):
    n = L.lora_clip_grads_workspace_bytes(lst)
    ws = torch.full((max(n, 16),), 0xAB, dtype=torch.uint8, device="cuda")
    norms = torch.full((lst.num_groups,), float("nan"), device="cuda") if norms is None else norms
    L.lora_clip_grads(lst, max_norm, norms, ws, n, stream=stream)
    return norms


def tensors(seed, sizes, dtypes, scale=1.0):
    """Views into larger buffers, at odd addresses, with a border that has to stay."""
    g, out, whole = gen(seed), [], []
    for i, n in enumerate(sizes):
        b = (torch.randn(n + 12, generator=g, device="cuda") * scale).to(
            TORCH[dtypes[i % len(dtypes)]])
        whole.append(b)
        out.append(b[1 + i % 7:1 + i % 7 + n])
    return out, whole


def check(before, after, groups, count, max_norm, norms, label):
    for g in range(count):
        mine = [i for i, k in enumerate(groups) if k == g]
        want = math.sqrt(sum(before[i].double().square().sum().item() for i in mine))
        # a sum in 64 bits, a root and a rounding to fp32
        assert abs(norms[g].item() - want) <= 2.0 ** -23 * want, (label, g)
        f = max_norm / want if want > max_norm else 1.0
        for i in mine:
            x = before[i].double() * f
            half = HALF_STEP["bf16" if before[i].dtype == torch.bfloat16 else "f32"]
            # the factor's rounding (2^-24 and a norm's 2^-40), the product's and the output's
            b = (half + 2.0 ** -23) * x.abs() + 2.0 ** -126
            assert ((after[i].double() - x).abs() <= (b if f != 1.0 else 0)).all(), (label, i)


SIZES = [[1], [8], [9], [2047, 2048, 2049], [5, 0, 70000, 31, 4096], [3] * 40,
         [1 << 20, 17, 300_001], [40_000_003, 1_000_000]]


@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f32", "bf16"]])
@pytest.mark.parametrize("k", range(len(SIZES)))
def test_sizes(dtypes, k):
    sizes = SIZES[k]
    for count in sorted({1, min(3, len(sizes)), len(sizes)}):
        groups = [i % count for i in range(len(sizes))]
        for max_norm in (0.5 * math.sqrt(sum(sizes) / count), 1e6, 0.0, math.inf):
            grads, whole = tensors(k, sizes, dtypes)
            before = [t.clone() for t in grads]
            border = [w.clone() for w in whole]
            norms = clip(L.GradList(grads, groups), max_norm)
            check(before, grads, groups, count, max_norm, norms, f"{sizes[:4]} {count} {max_norm}")
            outs, wo = tensors(k + 100, sizes, dtypes)
            edge = [w.clone() for w in wo]
            grads, _ = tensors(k, sizes, dtypes)
            again = clip(L.GradList(grads, groups, outs), max_norm)
            assert torch.equal(norms, again)
            check(before, outs, groups, count, max_norm, norms, "out")
            for i, n in enumerate(sizes):
                assert torch.equal(grads[i], before[i])
                for w, b in ((whole[i], border[i]), (wo[i], edge[i])):
                    keep = torch.ones(n + 12, dtype=torch.bool, device="cuda")
                    keep[1 + i % 7:1 + i % 7 + n] = False
                    assert torch.equal(w[keep], b[keep]), "outside a tensor"


def test_pool_slots():
    """Slots of a pool's gradients as groups; slots outside the list are left alone."""
    dA = torch.randn(5, 2, 16, 72, generator=gen(1), device="cuda")
    dB = torch.randn(5, 104, 16, generator=gen(2), device="cuda") * torch.arange(
        5, device="cuda").view(5, 1, 1)
    use = [0, 2, 4]
    grads = [t[a] for a in use for t in (dA, dB)]
    before, whole = [t.clone() for t in grads], (dA.clone(), dB.clone())
    groups = [g for g in range(3) for _ in range(2)]
    norms = clip(L.GradList(grads, groups, num_groups=4), 60.0)
    check(before, grads, groups, 3, 60.0, norms, "slots")
    assert norms[3] == 0
    for a in (1, 3):
        assert torch.equal(dA[a], whole[0][a]) and torch.equal(dB[a], whole[1][a])


def test_extreme_values():
    big = torch.full((3000,), 3e38, device="cuda")
    small = torch.full((3000,), 1e-38, device="cuda")
    mixed = torch.randn(3000, generator=gen(3), device="cuda")
    lst = L.GradList([big, small, mixed], [0, 1, 2])
    keep = big.clone()
    norms = clip(lst, 1e-37)
    # 3e38 sqrt(3000) is past fp32: reported as infinite, and left
    assert norms[0] == math.inf and torch.equal(big, keep)
    assert abs(norms[1].item() / (1e-38 * math.sqrt(3000)) - 1) < 1e-6
    assert abs(small.double().norm().item() / 1e-37 - 1) < 1e-6
    assert abs(mixed.double().norm().item() / 1e-37 - 1) < 1e-6
    big.fill_(1e25)     # squares past fp32's range, the norm within it
    assert abs(clip(lst, 2.0)[0].item() / (1e25 * math.sqrt(3000)) - 1) < 1e-6
    assert abs(big.double().norm().item() / 2.0 - 1) < 1e-6
    for v in (math.inf, -math.inf, math.nan):
        mixed.normal_(generator=gen(4))
        small.normal_(generator=gen(5))
        mixed[1234] = v
        keep = mixed.clone()
        norms = clip(lst, 1.0)
        assert not norms[2].isfinite() and norms[1].isfinite()
        assert torch.equal(mixed.view(torch.int32), keep.view(torch.int32))
        assert abs(small.double().norm().item() - 1) < 1e-6


def test_refusals_of_gpu_tensors():
    t = torch.randn(64, 64, device="cuda")
    for a, k, want in (([t.t()], {}, _lib.LORA_E_SHAPE), ([t, t], {}, _lib.LORA_E_ARG),
                       ([t, t[3]], {}, _lib.LORA_E_ARG),
                       ([t], {"outs": [t[:32]]}, _lib.LORA_E_SHAPE),
                       ([t], {"outs": [t.cpu()]}, _lib.LORA_E_ARG),
                       ([t], {"groups": [1], "num_groups": 1}, _lib.LORA_E_ID),
                       ([t[:32], t[32:]], {"outs": [t[32:], None]}, _lib.LORA_E_ARG)):
        with pytest.raises(L.LoraError) as e:
            L.GradList(a, **k)
        assert e.value.status == want
    lst = L.GradList([t], [1])
    with pytest.raises(L.LoraError) as e:
        clip(lst, 1.0, norms=torch.empty(1, device="cuda"))
    assert e.value.status == _lib.LORA_E_SHAPE


def test_streams_and_replays():
    sizes, groups = [5000, 70001, 333, 1 << 19], [0, 1, 1, 2]
    grads, _ = tensors(9, sizes, ["f32", "bf16"])
    outs = [torch.empty_like(t) for t in grads]
    lst = L.GradList(grads, groups, outs)
    n = L.lora_clip_grads_workspace_bytes(lst)
    ws, norms = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    call = lambda: L.lora_clip_grads(lst, 50.0, norms, ws, n)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    check(grads, outs, groups, 3, 50.0, norms, "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        new, _ = tensors(20 + k, sizes, ["f32", "bf16"], scale=0.2 + k)
        for a, b in zip(grads, new):
            a.copy_(b)
        call()
        want = [t.clone() for t in outs] + [norms.clone()]
        for t in outs + [norms]:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + [norms], want)), k
