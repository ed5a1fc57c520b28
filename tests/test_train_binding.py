"""CPU tests of the training operators' binding: what a TensorSet keeps, and
the buffers that its calls refuse.  No call here reaches the HIP runtime."""
import gc
import weakref

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_step_amd as Z
from zero_sharded_optimizer_step_amd import train


@pytest.fixture
def anywhere(monkeypatch):
    """Host tensors pass for device ones; nothing is launched."""
    monkeypatch.setattr(train, "_on_device", lambda **tensors: None)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_set_keeps_the_memory_that_its_table_points_at(anywhere, bits):
    # numpy arrays behind the tensors: they live as long as the memory is held
    alive = {}

    def fresh(name, n, dtype):
        a = np.zeros(n, dtype)
        alive[name] = weakref.ref(a)
        return torch.from_numpy(a)
    n, k = 300, Z.state8_blocks(300)
    lists = {"master": [fresh("master", n, np.float32)], "grad": [fresh("grad", n, np.float16)],
             "param": [fresh("param", n, np.float16)]}
    if bits == 32:
        lists.update(exp_avg=[fresh("m", n, np.float32)], exp_avg_sq=[fresh("v", n, np.float32)])
    else:
        # 16-byte aligned codes
        lists.update(state8=[fresh("s", 512 * k + 16, np.uint8)], scale8=[fresh("e", 2 * k, np.uint8)])
        lists["state8"][0] = lists["state8"][0][-lists["state8"][0].data_ptr() % 16:][:512 * k]
    ts = Z.TensorSet(**lists)
    # the caller puts other tensors in their places, in the lists and behind the tensors
    lists["param"][0].data = torch.zeros(n, dtype=torch.float16)
    for seq in lists.values():
        seq[0] = None
    lists["grad"].clear()
    gc.collect()
    assert all(r() is not None for r in alive.values()), [x for x, r in alive.items() if r() is None]
    del ts
    gc.collect()
    assert all(r() is None for r in alive.values())


def a_set():
    m, g = torch.zeros(300), torch.zeros(300, dtype=torch.bfloat16)
    return Z.TensorSet(master=[m], grad=[g], exp_avg=[m.clone()], exp_avg_sq=[m.clone()])


def test_norm_and_apply_refuse_host_tensors(monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(train, "_on_device", lambda **tensors: None)
        ts = a_set()
    groups = [Z.AdamGroup()]
    table = torch.zeros(Z.zero_partials_bytes(2), dtype=torch.uint8)
    # a stream's number, so that no call asks torch for the current one
    with pytest.raises(ValueError, match="partials is on cpu"):
        Z.zero_tensors_norm(ts, groups, 1, 0, table, stream=0)
    with pytest.raises(ValueError, match="global_buf is on cpu"):
        Z.zero_tensors_apply(ts, groups, 1, torch.zeros(32, dtype=torch.uint8), stream=0)


def strided(n, dtype):
    return torch.zeros(2 * n, dtype=dtype)[::2]


def test_calls_refuse_buffers_that_are_not_contiguous(anywhere):
    # the library gets an address only: a strided view would be read at the wrong
    # elements, an expanded one past its memory
    m, v = torch.zeros(300), torch.zeros(300)
    s8, e8 = torch.zeros(1024, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    one, byte = torch.zeros(1), torch.zeros(1, dtype=torch.uint8)
    good = {"exp_avg": m, "exp_avg_sq": v, "state8": s8, "scale8": e8}
    for name, bad in (("exp_avg", strided(300, torch.float32)), ("exp_avg_sq", one.expand(300)),
                      ("state8", byte.expand(1024)), ("scale8", strided(4, torch.uint8))):
        kw = {**good, name: bad}
        with pytest.raises(ValueError, match="%s is not contiguous" % name):
            Z.zero_state8_encode(kw["exp_avg"], kw["exp_avg_sq"], kw["state8"], kw["scale8"], stream=0)
        with pytest.raises(ValueError, match="%s is not contiguous" % name):
            Z.zero_state8_decode(kw["state8"], kw["scale8"], kw["exp_avg"], kw["exp_avg_sq"], stream=0)
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16)
    f, t = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    args = dict(x=x, w=w, target=t, loss=f, lse=f, result=torch.zeros(32, dtype=torch.uint8),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8), dx=x, dw=w)
    for name, bad in (("result", byte.expand(32)), ("workspace", byte.expand(1 << 20))):
        for backward in (False, True):
            with pytest.raises(ValueError, match="%s is not contiguous" % name):
                Z.XentArgs(**{**args, name: bad}).c_args(backward)
    ts, groups = a_set(), [Z.AdamGroup()]
    with pytest.raises(ValueError, match="partials is not contiguous"):
        Z.zero_tensors_norm(ts, groups, 1, 0, byte.expand(Z.zero_partials_bytes(1)), stream=0)
    with pytest.raises(ValueError, match="global_buf is not contiguous"):
        Z.zero_tensors_apply(ts, groups, 1, strided(32, torch.uint8), stream=0)
    with pytest.raises(ValueError, match="scalars is not contiguous"):
        Z.zero_tensors_scalars(ts, groups, 1, scalars=byte.expand(288))


class Elsewhere:
    """What a check of devices sees of a tensor."""
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_calls_refuse_tensors_of_two_devices(monkeypatch):
    train._on_device(a=Elsewhere(1), b=None, c=Elsewhere(1))
    with pytest.raises(ValueError, match="b is on cuda:1, a on cuda:0"):
        train._on_device(a=Elsewhere(0), b=Elsewhere(1))
    # a set's tensors are checked against the first one's device
    seen = []
    monkeypatch.setattr(train, "_on_device", lambda **tensors: seen.append(tensors))
    m, g = torch.zeros(300), torch.zeros(300, dtype=torch.bfloat16)
    away = torch.zeros(300, dtype=torch.bfloat16, device="meta")
    with pytest.raises(Z.ZeroError):                     # it has no address
        Z.TensorSet(master=[m, m.clone()], grad=[g, away], exp_avg=[m, m], exp_avg_sq=[m, m])
    assert [list(t) for t in seen] == [["master[0]", "grad[1]"], ["master[0]"]]
    assert seen[0]["grad[1]"] is away


class Recorded:
    """A buffer that says which streams it was told of."""

    def __init__(self, t):
        self.t, self.streams = t, []

    def __getattr__(self, name):
        return getattr(self.t, name)

    def record_stream(self, stream):
        self.streams.append(stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_a_sets_own_buffers_outlive_their_use_on_another_stream(anywhere, monkeypatch):
    ts, groups = a_set(), [Z.AdamGroup()]
    own = [Recorded(t) for t in (ts.table, ts.workspace, ts.result)]
    ts.table, ts.workspace, ts.result = own
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a[-1])) or 0
    monkeypatch.setattr(train, "train_lib", Lib)
    table = torch.zeros(Z.zero_partials_bytes(1), dtype=torch.uint8)
    a, b, c = Stream(5), Stream(6), Stream(7)
    Z.zero_tensors_step(ts, groups, 1, stream=a)
    Z.zero_tensors_step(ts, groups, 2, stream=a)
    Z.zero_tensors_norm(ts, groups, 1, 0, table, stream=b)
    Z.zero_tensors_apply(ts, groups, 1, torch.zeros(32, dtype=torch.uint8), stream=c)
    assert [h for _, h in calls] == [5, 5, 6, 7]
    assert all(q.streams == [a, b, c] for q in own)


def test_calls_refuse_another_device_than_the_current_one(anywhere, monkeypatch):
    # a call launches on the current device, with that device's stream
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ts, groups = a_set(), [Z.AdamGroup()]
    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0
    monkeypatch.setattr(train, "train_lib", Lib)
    table = torch.zeros(Z.zero_partials_bytes(1), dtype=torch.uint8)
    own = [Recorded(t) for t in (ts.table, ts.workspace, ts.result)]
    ts.table, ts.workspace, ts.result = own
    monkeypatch.setattr(train.XentArgs, "c_args", lambda self, backward: train.zero_xent_args())
    xent = Z.XentArgs(*[own[2]] * 7)
    m, s8, e8 = torch.zeros(300), torch.zeros(1024, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    state = Recorded(m)
    calls = [lambda: Z.zero_tensors_step(ts, groups, 1, stream=0),
             lambda: Z.zero_tensors_norm(ts, groups, 1, 0, table, stream=0),
             lambda: Z.zero_tensors_apply(ts, groups, 1, torch.zeros(32, dtype=torch.uint8), stream=0),
             lambda: Z.zero_xent_forward(xent, stream=0), lambda: Z.zero_xent_backward(xent, stream=0),
             lambda: Z.zero_state8_encode(state, m, s8, e8, stream=0),
             lambda: Z.zero_state8_decode(s8, e8, state, m, stream=0)]
    for t in (own[2], state):
        t.is_cuda, t.device = True, torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle))
    for call in calls:
        with pytest.raises(ValueError, match="on cuda:1; the current device is cuda:0"):
            call()
    assert not launched
    for t in (own[2], state):
        t.device = torch.device("cuda", 0)
    for call in calls:
        call()
    assert len(launched) == len(calls)
