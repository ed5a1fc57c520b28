"""The loss in a workspace of a larger batch: the results are those of one of
its own, and nothing past its end is written."""
import pytest
import torch

import zero_sharded_optimizer_step_amd as Z
from test_gpu_xent import Call, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,vocab", [(1000, 3001), (512, 10007), (72, 20000)], ids=str)
def test_one_workspace_for_all_batches(dim, vocab):
    most = 1100
    size = Z.zero_xent_workspace_bytes(most, dim, vocab)
    room = torch.full((size // 4 + 64,), float("nan"), device="cuda").view(torch.uint8)
    for tokens in (most, 1025, 1024, 513, 129, 128, 65, 9, 8, 1):
        say("xent shared workspace %s" % ((tokens, dim, vocab),))
        shared, own = (Call(tokens, dim, vocab, torch.bfloat16) for _ in range(2))
        shared.args.workspace = room[:size]
        shared.run()
        own.run()
        for name in ("d_dx", "d_dw"):
            assert torch.equal(getattr(shared, name), getattr(own, name)), name
        for name in ("loss", "lse", "result"):
            assert torch.equal(getattr(shared.args, name), getattr(own.args, name)), name
        if tokens in (8, 129, 1024):
            shared.check()
        assert bool(torch.isnan(room[size:].view(torch.float32)).all()), "written past the workspace's end"
