"""The 8-bit product and its gradient on the exact cases of linear8_cases: each
kernel of the forward on whole sums far past 2^24, and the gradient against
differences of the forward, element by element."""
import pytest
import torch

import linear8_cases as cases
import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_rows8 import say

pytestmark = pytest.mark.gpu


# forwards of few tokens, of tiles, gradients of few tokens and of tiles
@pytest.mark.parametrize("size,dtype", [
    ((40, 60, 50), torch.float16), ((64, 227, 33), torch.float16), ((100, 33, 70), torch.float16),
    ((130, 200, 300), torch.float16), ((300, 40, 1700), torch.float16), ((1, 28, 40), torch.bfloat16),
    ((70, 28, 90), torch.bfloat16), ((260, 24, 2100), torch.bfloat16)], ids=str)
def test_gradient_is_the_forwards_differences(size, dtype):
    """The sums of both are exact: the gradient is off by its rounding alone."""
    t, k, n = size
    say("linear8 exact differences %s %s" % (size, dtype))
    x8, xs, w8, ws, dy = cases.small(t, k, n, "cuda", seed=t)
    y = torch.empty(t, n, dtype=dtype, device="cuda")
    dx, dw = torch.empty(t, k, dtype=dtype, device="cuda"), torch.empty(n, k, dtype=dtype, device="cuda")
    ws_ = torch.empty(Z.zero_linear8_workspace_bytes(t, k, n), dtype=torch.uint8, device="cuda")
    args = Z.Linear8Args(x8, xs, w8, ws, dim=k, workspace=ws_, y=y, dy=dy.to(dtype), dx=dx, dw=dw)
    Z.zero_linear8_backward(args)

    def forward():
        Z.zero_linear8_forward(args)
        return y.clone()
    for got, want, what in zip((dx, dw), cases.differences(forward, x8, xs, w8, ws, dy, k), ("dx", "dw")):
        ref.within(got.double(), want, ref.half_step(want, dtype), what)


# of 4090 x 4090 the tiles are 256 x 256
@pytest.mark.parametrize("tokens,out", [(t, n) for t in (1, 2, 20, 50, 200, 2049) for n in (20, 1040, 2050)] + [(4090, 4090)])
def test_whole_sums(tokens, out):
    """Past 10^9 and back to an odd number below 2^10, and 2^31 - 16384."""
    say("linear8 whole sums %d x %d" % (tokens, out))
    x8, xs, w8, ws, want = cases.whole(tokens, out, "cuda", seed=tokens + out)
    y = torch.empty(tokens, out, dtype=torch.float16, device="cuda")
    room = torch.empty(Z.zero_linear8_workspace_bytes(tokens, cases.LONGEST, out, backward=False), dtype=torch.uint8,
                       device="cuda")
    Z.zero_linear8_forward(Z.Linear8Args(x8, xs, w8, ws, dim=cases.LONGEST, workspace=room, y=y))
    assert torch.equal(y[:-1, :-1].double(), want[:-1, :-1])
    # of the rows of -128 the sum has up to 31 bits: fp32 and then fp16 round it
    ref.within(y.double(), want, 3 * ref.U * want.abs() + ref.half_step(want, torch.float16), "y")
    assert float(y[-1, -1]) == 32.0
