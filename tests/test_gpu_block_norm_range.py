"""Block norm's gradients where dout and the stream are of very different sizes, rows of
zeros, and rows near fp32's ends in every form of the kernel (one, two and four pieces a
thread), against 64 bits with the bounds of the other tests."""
import pytest
import torch

from block_norm_helpers import inputs, run_join, run_join_backward
from gpu_helpers import say
from test_gpu_block_norm import check_backward

pytestmark = pytest.mark.gpu
# (one, two and four pieces a thread; two also where rows are many)
SIZES = [(7, 264), (7, 4096), (2052, 4096), (7, 8192), (7, 16384)]


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"[gpu] {request.node.name}")
    yield


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("post", [False, True])
def test_gradients_far_from_the_stream(dtype, T, H, post):
    """dout times the stream is past fp32's range or below its numbers, the stream's squares
    are not, and no gradient is."""
    s = inputs(T + H, T, H, dtype)
    rows = torch.arange(T, device="cuda") % 7
    of_t = torch.tensor([50., 50., -30., -36., 0., 0., 0.], device="cuda")[rows]
    of_dout = torch.tensor([85., 100., -100., -106., 100., -100., 0.], device="cuda")[rows]
    s["sum"] *= torch.exp2(of_t).to(s["sum"].dtype)[:, None]
    s["dout"] *= torch.exp2(of_dout).to(s["dout"].dtype)[:, None]
    got = run_join_backward(s, dtype, "none", eps=0.0, post=post, stream_grad=False, sums=False)
    check_backward(s, got, dtype, 1.0, 1.0, 0.0, post, True, False, f"T={T} H={H}")


@pytest.mark.parametrize("T,H", [(1, 520), (1, 4096), (1, 8192), (1, 16384)])
def test_a_rows_factor_is_the_forward_pass_own(T, H):
    """With dout and the weight 1, the weight's gradient of a single row is the row times its
    factor, which is the forward pass's output: the same bits."""
    for seed in range(24):
        s = inputs(seed, T, H, "f32")
        s["pre"], s["dout"] = torch.ones_like(s["pre"]), torch.ones_like(s["dout"])
        total, out, _, _ = run_join(s, "f32", "none", post=False, out8=False)
        got = run_join_backward(dict(s, sum=total), "f32", "none", post=False)
        assert torch.equal(got["dpre"], out[0]), seed
        # the norm after the block: its factor by the forward pass of y alone
        s["residual"], s["post"] = torch.zeros_like(s["residual"]), s["pre"]
        total, _, _, _ = run_join(s, "f32", "none", pre=False)
        got = run_join_backward(dict(s, dsum=s["dout"]), "f32", "none", pre=False)
        assert torch.equal(got["dpost"], total[0]), seed


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
def test_rows_of_zeros_and_at_the_ends(dtype, T, H):
    """Rows of zeros (a masked block's) beside others, and with eps = 0 rows whose squares are
    past fp32's ends."""
    s = inputs(T * H, T, H, dtype, "channel")
    for k in ("y", "sum"):
        s[k][1::3] = 0
    s["y"][2::7] = 0
    got = run_join_backward(s, dtype, "channel")
    check_backward(s, got, dtype, 1.0, 1.0, 1e-5, True, True, True, f"zeros T={T} H={H}")
    assert all(v.isfinite().all() for v in got.values())
    s = inputs(T * H + 1, T, H, dtype, "channel")
    for k in ("y", "sum"):
        s[k][1::3] *= 2.0 ** -60   # (gradients of two such norms are 2^120 times dout)
        s[k][2::3] *= 2.0 ** 100
    got = run_join_backward(s, dtype, "channel", eps=0.0, stream_grad=False, sums=False)
    check_backward(s, {k: got[k] for k in ("dy", "dresidual")}, dtype, 1.0, 1.0, 0.0, True, True,
                   False, f"ends T={T} H={H}")
