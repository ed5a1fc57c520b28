"""The 8-bit product where its buffers lie at the edge of what it takes: bias
and scales next to their alignment, and the largest strides."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_linear8 import Call
from test_gpu_rows8 import say

pytestmark = pytest.mark.gpu


def moved(t, by):
    """The same values `by` elements into memory of their own."""
    room = torch.empty(t.numel() + by + 8, dtype=t.dtype, device="cuda")
    view = room[by:by + t.numel()]
    view.copy_(t)
    return view


# forwards of few tokens, small tiles, large ones and slices; gradients of few tokens and of both tiles
SIZES = [(1, 700, 300), (40, 100, 77), (64, 2048, 1024), (300, 64, 1501), (2300, 272, 2050), (260, 8208, 515)]


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_bias_and_scales_next_to_their_alignment(size, by):
    say("linear8 bias and scales %s %d" % (size, by))
    c = Call(*size, torch.float16, any_codes=True)
    c.xs, c.ws, c.bias, c.db = moved(c.xs, by), moved(c.ws, by), moved(c.bias, by), moved(c.db, by)
    c.args.x_scale, c.args.w_scale, c.args.bias, c.args.db = c.xs, c.ws, c.bias, c.db
    c.check()


def far_rows(rows, cols, stride, dtype):
    return torch.empty(rows * stride, dtype=dtype, device="cuda").view(rows, stride)[:, :cols]


@pytest.mark.parametrize("size", [(3, 600, 130), (64, 600, 300), (257, 600, 300)], ids=str)
def test_the_largest_strides_of_codes(size):
    """4 MB from row to row: of a tile's 256 rows 1 GB."""
    t, k, n = size
    say("linear8 strides of 4 MB %s" % (size,))
    c = Call(*size, torch.bfloat16)
    for name, rows in (("x8", t), ("w8", n)):
        far = far_rows(rows, ref.stride(k), 1 << 22, torch.int8)
        far.copy_(getattr(c, name))
        setattr(c, name, far)
        setattr(c.args, name, far)
    c.check()


@pytest.mark.parametrize("size", [(3, 40, 20), (5, 600, 8), (66, 40, 24)], ids=str)
def test_rows_of_16_bits_past_32_bits(size):
    """2^30 elements and more from row to row: offsets past 2^32 bytes."""
    t, k, n = size
    say("linear8 strides of 2^27 and more %s" % (size,))
    c = Call(*size, torch.bfloat16)
    stride = (1 << 30) + 8 if t < 10 else (1 << 27) + 3
    room = torch.empty(t * stride, dtype=torch.bfloat16, device="cuda").view(t, stride)
    dy, y, dx = room[:, :n], room[:, 64:64 + n], room[:, 128:128 + k]
    dy.copy_(c.dy)
    c.args.y, c.args.dy, c.args.dx = y, dy, dx
    c.y, c.dy, c.dx = y, dy, dx
    Z.zero_linear8_forward(c.args)
    c.check_forward()
    Z.zero_linear8_backward(c.args)
    c.check_backward()
