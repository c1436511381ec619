"""The decoder-block operators on a stream of the caller's: ordered after what that
stream did before, and before what it does next, with the default stream idle.

Inputs, outputs and workspace are made on the stream itself, behind a wait of some
milliseconds, so that a launch on another stream would find them unwritten."""
import pytest
import torch

import lora_adapter_pool_amd as L
from block_helpers import gen, normal, run_backward, run_gated, run_linear
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


def _calls(x, r, w, wg, wd, stream=None):
    """Everything that the operators write, as copies made on the current stream."""
    T, K, I = x.shape[0], x.shape[1], wg.shape[0] // 2
    total, n = torch.empty_like(x), torch.empty_like(x)
    L.lora_add_rms_norm(L.make_norm_desc("bf16", K, 1e-5), x, r, w, total, n, None, None, T,
                        stream=stream)
    h, pre = run_gated(n, wg, None, None, None, True, "bf16", "bf16", "silu", stream=stream)
    y = run_linear(h, wd, None, None, None, None, total, "bf16", "bf16", "none", stream=stream)
    return [t.clone() for t in (total, n, h, pre, y)]


@pytest.mark.parametrize("given", [False, True])
def test_calls_are_ordered_on_their_stream(given):
    """given: the stream is handed to the calls, else it is the current one."""
    g = gen(31)
    T, K, I = 70, 520, 264
    src = [normal(g, s, "bf16", d) for s, d in (((T, K), 1), ((T, K), 1), ((K,), 1),
                                                 ((2 * I, K), 0.05), ((K, I), 0.05))]
    want = _calls(*src)
    dh = normal(g, (T, I), "bf16", 0.1)
    want += list(run_backward(dh, want[3], want[1], src[3], "silu", "bf16"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            late = [torch.full_like(t, float("nan")) for t in src]
            torch.cuda._sleep(20_000_000)
            for a, b in zip(late, src):
                a.copy_(b)
            got = _calls(*late, stream=s if given else None)
            got += list(run_backward(dh, got[3], got[1], late[3], "silu", "bf16"))
            for t in late:                       # what follows on the stream comes after
                t.fill_(float("nan"))
        assert torch.cuda.default_stream().query()
        s.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), k
