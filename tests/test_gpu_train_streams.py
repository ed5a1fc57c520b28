"""A tensor list stepped on another stream than the one it was made on."""
import pytest
import torch

import zero_sharded_optimizer_step_amd as Z
from test_gpu_train_tensors import GROUPS, List

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("give", ["object", "handle", "current"])
def test_its_buffers_are_not_reused_while_the_step_waits(give):
    q = List([3000, 70], 32)
    ts = q.set()
    sizes = [(t.data_ptr(), t.numel()) for t in (ts.table, ts.workspace, ts.result)]
    big = torch.ones(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(1500):                             # some 0.5 s
            big.mul_(1.0)
        done = torch.cuda.Event()
        Z.zero_tensors_step(ts, GROUPS, step=1, max_grad_norm=0.0,
                            stream={"object": side, "handle": side.cuda_stream, "current": None}[give])
        done.record(side)
    del ts
    taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in sizes for _ in range(4)]
    if done.query():
        pytest.skip("the step ran before its buffers' memory was asked for")
    assert not {t.data_ptr() for t in taken} & {p for p, _ in sizes}
    torch.cuda.synchronize()
    want = List([3000, 70], 32)
    Z.zero_tensors_step(want.set(), GROUPS, step=1, max_grad_norm=0.0)
    for name in want.flat:
        assert torch.equal(q.flat[name], want.flat[name]), name
