"""The loss's workspace query: a buffer sized for a batch serves every smaller
one.  On the CPU: a refused call names what it needs before any launch."""
import ctypes
import re

import pytest

import zero_sharded_optimizer_step_amd as Z
from test_train_host import xent_args
from zero_sharded_optimizer_step_amd._train_abi import train_lib

SIZE = Z.zero_xent_workspace_bytes


def needs(tokens, dim, vocab):
    a = xent_args(tokens=tokens, dim=dim, vocab=vocab, x_stride=dim, w_stride=dim, dx_stride=dim, dw_stride=dim,
                  workspace_bytes=0)
    found = set()
    for call in (train_lib().zero_xent_forward, train_lib().zero_xent_backward):
        assert call(ctypes.byref(a), None) == Z.ZERO_ESIZE
        found.add(int(re.search(r"workspace_bytes 0 < (\d+) needed", Z.zero_last_error()).group(1)))
    return max(found)


@pytest.mark.parametrize("dim,vocab", [(4096, 32000), (512, 10007), (1000, 10007), (4096, 128000), (64, 300), (33, 700),
                                       (8192, 50000)], ids=str)
def test_a_larger_batchs_workspace_serves_smaller_ones(dim, vocab):
    most = 5000
    size, last = SIZE(most, dim, vocab), 0
    for tokens in range(1, most + 1):
        need = needs(tokens, dim, vocab)
        assert need <= size, tokens
        if tokens < 300 or tokens % 64 in (0, 1, 63):
            own = SIZE(tokens, dim, vocab)
            assert max(need, last) <= own <= size, tokens
            last = own


@pytest.mark.parametrize("dim,vocab", [(64, 1 << 24), (100000, 3000), (513, 500000)], ids=str)
def test_pieces_of_the_vocabulary_of_many_tokens(dim, vocab):
    """Where one more token makes the pieces narrower, the token before needs more."""
    most = 1 << 20
    size = SIZE(most, dim, vocab)
    for width in list(range(256, 20000, 256)) + list(range(20224, vocab, 65536)):
        for room in (1 << 27, 1 << 26):
            last = room // width
            for tokens in (last - 1, last, last + 1):
                if 1 <= tokens <= most:
                    assert needs(tokens, dim, vocab) <= SIZE(tokens, dim, vocab) <= size
