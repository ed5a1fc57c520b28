"""The 8-bit product in a workspace of a larger batch, of the forward alone,
and of a gradient without a copy of dy: the results are those of a workspace
of its own, and nothing past its end is written."""
import re

import pytest
import torch

import zero_sharded_optimizer_step_amd as Z
from test_gpu_linear8 import Call
from test_gpu_rows8 import say

pytestmark = pytest.mark.gpu


def room(size):
    """A workspace of NaN with a margin behind it."""
    whole = torch.full((size // 4 + 64,), float("nan"), device="cuda").view(torch.uint8)
    return whole, whole[:size]


def margin_untouched(whole, size):
    assert bool(torch.isnan(whole[size:].view(torch.float32)).all()), "the workspace was written past its end"


@pytest.mark.parametrize("dim,out", [(512, 1024), (300, 1500), (8000, 130), (2048, 2048)], ids=str)
def test_one_workspace_for_all_batches(dim, out):
    most = 1100
    size = Z.zero_linear8_workspace_bytes(most, dim, out)
    whole, ws = room(size)
    for tokens in (most, 1025, 1024, 640, 513, 129, 128, 65, 64, 33, 17, 16, 1):
        say("linear8 shared workspace %s" % ((tokens, dim, out),))
        c = Call(tokens, dim, out, torch.bfloat16, pad=tokens % 2)
        c.args.workspace = ws
        c.check()
        margin_untouched(whole, size)
        got = [m.clone() for m in (c.y, c.dx, c.dw, c.db)]
        own = Call(tokens, dim, out, torch.bfloat16, pad=tokens % 2)
        Z.zero_linear8_forward(own.args)
        Z.zero_linear8_backward(own.args)
        assert all(torch.equal(a, b) for a, b in zip(got, (own.y, own.dx, own.dw, own.db)))


@pytest.mark.parametrize("size", [(1, 700, 300), (65, 4096, 1024), (256, 4096, 520), (700, 3000, 1504), (2048, 1024, 4200)],
                         ids=str)
def test_each_use_alone(size):
    t, k, n = size
    say("linear8 workspace of one use %s" % (size,))
    c = Call(*size, torch.float16)
    for uses, call, check in ((dict(backward=False), Z.zero_linear8_forward, c.check_forward),
                              (dict(forward=False, any_dy=n % 8 != 0), Z.zero_linear8_backward, c.check_backward)):
        size = Z.zero_linear8_workspace_bytes(t, k, n, **uses)
        whole, c.args.workspace = room(size)
        call(c.args)
        check()
        margin_untouched(whole, size)
    assert n % 8 or t <= 64 or size < Z.zero_linear8_workspace_bytes(t, k, n)


def test_what_a_call_does_not_use_is_not_asked_for():
    """dy's rows off their alignment need the copy, column sums alone do not."""
    t, k, n = 300, 512, 264
    say("linear8 workspace without a copy")
    less = Z.zero_linear8_workspace_bytes(t, k, n, forward=False, any_dy=False)
    c = Call(t, k, n, torch.bfloat16, pad=1)
    whole, c.args.workspace = room(less)
    with pytest.raises(Z.ZeroError, match="workspace_bytes"):
        Z.zero_linear8_backward(c.args)
    c.args.dx = c.args.dw = None
    Z.zero_linear8_backward(c.args)
    want = Call(t, k, n, torch.bfloat16, pad=1)
    Z.zero_linear8_backward(want.args)
    assert torch.equal(c.db, want.db)
    margin_untouched(whole, less)


@pytest.mark.parametrize("wanted", [("dx",), ("dw",), ("db",), ("dx", "dw"), ("dx", "db"), ("dw", "db")], ids="+".join)
def test_a_part_of_the_gradient_in_its_own_room(wanted):
    """Each gradient needs its own operand's room alone."""
    for size in ((20, 300, 500), (64, 2048, 1100), (300, 512, 264), (700, 1000, 333), (2100, 520, 2304)):
        for pad in (0, 1):
            say("linear8 workspace of %s %s %d" % (wanted, size, pad))
            c = Call(*size, torch.bfloat16, pad=pad)
            Z.zero_linear8_backward(c.args)
            want = {name: getattr(c, name).clone() for name in wanted}
            for name in ("dx", "dw", "db"):
                getattr(c, name).fill_(-7)
                if name not in wanted:
                    setattr(c.args, name, None)
            with pytest.raises(Z.ZeroError, match="workspace_bytes") as refused:
                c.args.workspace = c.room[:1]
                Z.zero_linear8_backward(c.args)
            size_needed = int(re.search(r"< (\d+) needed", str(refused.value)).group(1))
            whole, c.args.workspace = room(size_needed)
            Z.zero_linear8_backward(c.args)
            for name in ("dx", "dw", "db"):
                assert torch.equal(getattr(c, name), want[name]) if name in wanted else bool((getattr(c, name) == -7).all())
            margin_untouched(whole, size_needed)
            c.clean()


def test_nothing_of_rows_far_apart():
    """No output channel, or no token, of a dy of any stride: zeros."""
    for t, k, n in ((3, 40, 0), (200, 300, 0), (0, 40, 30)):
        for stride in (1 << 25, (1 << 25) + 8, (1 << 20) + 1):
            say("linear8 nothing of %s, %d apart" % ((t, k, n), stride))
            c = Call(t, k, n, torch.bfloat16)
            rows = torch.empty(min(t, 3) * stride, dtype=torch.bfloat16, device="cuda")
            # no element of a row exists, so three rows' memory does for all
            c.args.dy = rows.as_strided((t, n), (stride, 1)) if n == 0 else c.dy
            Z.zero_linear8_backward(c.args)
            assert not bool(c.dx.any()) and not bool(c.dw.any()) and not bool(c.db.any())
            c.clean()
