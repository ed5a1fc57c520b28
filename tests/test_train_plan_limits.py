"""CPU test: a step refuses plans that no list can have (nothing is launched)."""
import ctypes

import pytest

import zero_sharded_optimizer_step_amd as Z
from test_train_host import step_args
from zero_sharded_optimizer_step_amd._train_abi import train_lib

I64 = 2**63 - 1
TOP = (2**31 - 1) * 1024                     # elements of the longest list


@pytest.mark.parametrize("numel,n_chunks,n_tensors", [
    (I64, 5, 1), (I64 - 1022, 5, 1), (TOP + 1, 2**31 - 1, 1),       # the chunk count of these wraps or is short
    (5 << 10, 5, 0), (0, 5, 5)])                                    # chunks of no tensor, of no element
def test_step_refuses_impossible_plans(numel, n_chunks, n_tensors):
    room = 64 * n_tensors + 4 * n_chunks
    a = step_args(plan_numel=numel, plan_n_chunks=n_chunks, plan_n_tensors=n_tensors,
                  plan_table_bytes=-(-room // 16) * 16)
    # a NULL workspace: what passes the plan's check is refused with another text
    a.workspace = None
    assert train_lib().zero_tensors_step(ctypes.byref(a), None, None) == Z.ZERO_EINVAL
    assert "plan is not one" in Z.zero_last_error()
