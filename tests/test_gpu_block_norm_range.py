"""Block norm's gradients where dout and the stream are of very different sizes, rows of
zeros, and rows near fp32's ends in every form of the kernel (one, two and four pieces a
thread), against 64 bits with the bounds of the other tests."""
import pytest
import torch

from block_norm_helpers import inputs, run_join_backward
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
