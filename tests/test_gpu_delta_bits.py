"""The input's gradient of a bf16 pool keeps fp32 products: whole numbers in rank space that
need all three bf16 pieces (17 to 20 bits), whose large parts cancel in the sum over the
ranks.  Every product and partial sum is a whole number below 2^24, so that the sum is exact
in fp32 and what is left, at most 128, is exact in bf16.  And an infinite dy."""
import numpy as np
import pytest
import torch

from block_helpers import TORCH
from delta_helpers import delta64, run_delta
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,slots,kind", [(1, 8, 1, "one"), (70, 136, 3, "mixed"),
                                            (200, 520, 2, "runs")])
def test_ranks_that_cancel(dtype, T, K, slots, kind):
    """B takes three features into each rank: dy's are multiples of 2^12, of 2^4 and small, and
    two neighbouring ranks differ in the small one alone; A has them with opposite signs."""
    rng = np.random.default_rng(T)
    ids = np.zeros(T, np.int32) if kind == "one" else rng.integers(-1, slots, T)
    ids = np.sort(ids) if kind == "runs" else ids
    R, O = 16, 32
    g = torch.Generator(device="cuda").manual_seed(T)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g,  # noqa: E731
                                             device="cuda").float()
    dy = torch.cat([whole(32, 255, T, 8) * 4096, whole(-255, 255, T, 8) * 16,
                    whole(-8, 8, T, 16)], 1)
    B = torch.zeros(slots, O, R, device="cuda")
    for r in range(R):
        for j in (r // 2, 8 + r // 2, 16 + r):
            B[:, j, r] = 1
    A = torch.zeros(slots, 1, R, K, device="cuda")
    sign = whole(0, 1, slots, R // 2, K) * 2 - 1
    A[:, 0, 0::2], A[:, 0, 1::2] = sign, -sign
    to = TORCH[dtype]
    s = {"ids": ids.astype(np.int32), "x": whole(-2, 2, T, K).to(to), "dy": dy.to(to),
         "A": A.to(to), "B": B.to(to), "dx_in": torch.zeros(T, K, device="cuda", dtype=to),
         "outs": [O], "dtype": dtype}
    assert torch.equal(s["dy"].float(), dy)
    want = delta64(s)["dx"][0]
    assert want.abs().max() <= 128
    for dx_in in (False, True):
        assert torch.equal(run_delta(s, dx_in=dx_in)["dx"].double(), want), dx_in


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 24, 40, 64, 72])
def test_an_infinity_stays_one(dtype, R):
    """A row whose dy has one infinity, through positive A and B: its dx is infinite (and not
    NaN, whatever the ranks are padded to), its dA infinite or NaN by x's sign alone."""
    T, K, O = 5, 136, 72
    g = torch.Generator(device="cuda").manual_seed(R)
    pos = lambda *s: (torch.rand(s, generator=g, device="cuda") + 0.5).to(TORCH[dtype])  # noqa: E731
    s = {"ids": np.array([0, 1, -1, 1, 0], np.int32), "x": pos(T, K), "dy": pos(T, O),
         "A": pos(2, 1, R, K), "B": pos(2, O, R), "dx_in": pos(T, K), "outs": [O], "dtype": dtype}
    clean = run_delta(s)
    for sign in (1, -1):
        t = dict(s, dy=s["dy"].clone())
        t["dy"][3, 7] = sign * float("inf")
        got = run_delta(t)
        assert (got["dx"][3] == sign * float("inf")).all(), sign
        rows = [0, 1, 2, 4]
        assert torch.equal(got["dx"][rows], clean["dx"][rows])
        assert (got["dA"][1] == sign * float("inf")).all()
        assert torch.equal(got["dA"][0], clean["dA"][0])
        # v of a bf16 pool is a sum of pieces p + q + r, and q is of either sign: an infinite dy
        # times p and times q are infinities whose sum is NaN where the signs differ
        assert (got["dB"][1, 7] == sign * float("inf")).all() if dtype == "f32" else \
            not got["dB"][1, 7].isfinite().any()
        assert torch.equal(got["dB"][1, 8:], clean["dB"][1, 8:])
