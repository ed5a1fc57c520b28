"""What the 8-bit product's calls ask of their workspace and what its size
query says of it: a buffer sized for a batch serves every smaller one, the
forward asks for its own needs alone, and a gradient whose rows are read where
they lie for no copy of them.  On the CPU: a call that is refused names what
it needs before anything is launched."""
import ctypes
import re
import time

import pytest

import zero_sharded_optimizer_step_amd as Z
from test_train8_host import A, linear_args
from zero_sharded_optimizer_step_amd._train_abi import train_lib

SIZE = Z.zero_linear8_workspace_bytes


def needs(way, tokens, dim, out, whole=True, **kw):
    """Bytes that a call of these sizes refuses to do without."""
    stride = out if whole else out + 3
    a = linear_args(tokens=tokens, dim=dim, out=out, x8_stride=(dim + 15) // 16 * 16, w8_stride=(dim + 15) // 16 * 16,
                    y_stride=out, dy_stride=stride, dx_stride=dim, dw_stride=dim, workspace_bytes=0, **kw)
    assert getattr(train_lib(), "zero_linear8_" + way)(ctypes.byref(a), None) == Z.ZERO_ESIZE
    return int(re.search(r"workspace_bytes 0 < (\d+) needed", Z.zero_last_error()).group(1))


# layers of the training example and the measured cases, thin and long ones, and rows that come in pieces of columns
LAYERS = [(4096, 4096), (4096, 16384), (1000, 2053), (512, 4096), (100, 30), (16384, 1024), (40001, 70), (8, 5),
          (2048, 1000), (4096, 60000), (1500, 300000)]


@pytest.mark.parametrize("dim,out", LAYERS, ids=str)
def test_a_larger_batchs_workspace_serves_smaller_ones(dim, out):
    most, last = 4100, 0
    for tokens in list(range(1, 200)) + list(range(200, most, 7)) + [1023, 1024, 1025, 4095, 4096, 4097]:
        size = SIZE(tokens, dim, out)
        if tokens > 1 and tokens <= 4097 and tokens not in (1023, 1024, 1025, 4095, 4096):
            assert size >= last, tokens
            last = size
        assert size <= SIZE(most, dim, out)
    sizes = {uses: SIZE(most, dim, out, **dict(uses)) for uses in (
        (), (("backward", False),), (("forward", False), ("any_dy", False)), (("forward", False),))}
    forward, whole, anywhere = (sizes[u] for u in list(sizes)[1:])
    assert sizes[()] == max(forward, anywhere) and whole <= anywhere
    for tokens in range(1, most + 1):
        assert needs("forward", tokens, dim, out) <= forward
        assert needs("backward", tokens, dim, out, whole=out % 8 == 0) <= (whole if out % 8 == 0 else anywhere)
        assert needs("backward", tokens, dim, out, whole=False) <= anywhere


@pytest.mark.parametrize("dim,out", [(300, 260000), (131071, 1 << 20), (200, 1000)], ids=str)
def test_pieces_of_columns_of_many_tokens(dim, out):
    """Where one more token makes the pieces of columns narrower, the token before needs more."""
    most = 1 << 20
    size = SIZE(most, dim, out)
    for width in range(256, (dim + 255) // 256 * 256 + 1, 256):
        last = (1 << 28) // width - out
        for tokens in (last - 1, last, last + 1):
            if 1 <= tokens <= most:
                assert needs("backward", tokens, dim, out, whole=False) <= size
                assert needs("backward", tokens, dim, out, whole=False) <= SIZE(tokens, dim, out)
    for tokens in (1, 2, 63, 64, 65, 127, 128, 129, 511, 512, 513, 99999, most - 1, most):
        assert needs("backward", tokens, dim, out, whole=False) <= SIZE(tokens, dim, out) <= size


def test_what_is_not_needed_is_not_asked_for():
    # the forward of a batch that inference may have: a few slices' sums, or nothing
    assert needs("forward", 65, 4096, 16384) <= 1 << 20
    assert SIZE(65, 4096, 16384, backward=False) <= 1 << 23
    assert needs("forward", 8192, 4096, 16384) <= 256
    # a gradient of 8192 tokens whose rows are whole 16-byte pieces: no copy of them
    copy = 8192 * 16384 * 2
    whole, anywhere = (needs("backward", 8192, 4096, 16384, whole=w) for w in (True, False))
    assert anywhere - whole == copy
    assert SIZE(8192, 4096, 16384) - SIZE(8192, 4096, 16384, any_dy=False) == copy
    # rows off their alignment, as columns of a wider matrix
    assert needs("backward", 8192, 4096, 16384, dy=A + 2) == anywhere
    # the column sums alone read dy where it lies and need 16 shares of them; each product its own operand
    assert needs("backward", 8192, 4096, 16384, whole=False, dx=None, dw=None) == 16 * 16384 * 4
    dx, dw = (needs("backward", 8192, 4096, 16384, **{other: None, "db": None}) for other in ("dw", "dx"))
    assert (dx, dw) == (16384 * 4096 * 2, 8192 * 4096 * 2) and whole == dx + dw + 16 * 16384 * 4


def test_the_query_is_quick_where_nothing_is_needed():
    start = time.perf_counter()
    for sizes in ((1 << 20, 131071, 0), (1 << 20, 0, 1 << 20), (1 << 20, 131071, 1), (0, 131071, 1 << 20)):
        assert SIZE(*sizes) >= 256
    assert time.perf_counter() - start < 1


def test_uses():
    of = train_lib().zero_linear8_workspace_bytes_for
    assert of(100, 100, 100, 0) == 0 and of(100, 100, 100, 8) == 0 and of(100, 100, 100, -1) == 0
    assert of(100, 131072, 100, 1) == 0 and of(-1, 100, 100, 1) == 0 and of(100, 100, (1 << 20) + 1, 2) == 0
    for sizes in ((0, 0, 0), (1, 1, 1), (100, 100, 100), (700, 8000, 1500)):
        each = [of(*sizes, uses) for uses in (1, 2, 4)]
        assert all(e >= 256 and e % 256 == 0 for e in each)
        assert of(*sizes, 7) == max(each) == SIZE(*sizes)
        named = (Z.ZERO_LINEAR8_FORWARD, Z.ZERO_LINEAR8_BACKWARD, Z.ZERO_LINEAR8_BACKWARD_ANY_DY)
        assert [Z.zero_linear8_workspace_bytes_for(*sizes, uses) for uses in named] == each
    with pytest.raises(ValueError):
        SIZE(100, 100, 100, forward=False, backward=False)
