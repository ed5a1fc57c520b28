"""CPU tests of libzero_train_mi355x.so: it exports what include/zero/train.h
declares, plans lists and refuses bad arguments before any work.  No call
here reaches the HIP runtime."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import train_ref
import zero_sharded_optimizer_step_amd as Z
from zero_sharded_optimizer_step_amd import _abi, _train_abi
from zero_sharded_optimizer_step_amd._train_abi import (train_lib, zero_tensor_t, zero_tensors_args,
                                                        zero_xent_args)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                                  # stands for a device address; never read


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "zero", "train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(zero_[a-z0-9_]+)\s*\(", text))
    assert names == set(_train_abi._PROTOTYPES)
    L = ctypes.CDLL(_train_abi.TRAIN_LIB_PATH)
    for n in names:
        assert hasattr(L, n) and callable(getattr(Z, n)), n


def rec(n, at=A, group=0, param=A, **kw):
    f = dict(grad=at, master=at, exp_avg=at, exp_avg_sq=at, param=param, numel=n, group=group, reserved=0)
    f.update(kw)
    return zero_tensor_t(**f)


def test_plan_counts_and_table():
    sizes = [1, 0, 1024, 1025, 300000]
    plan, table = Z.zero_tensors_plan([rec(n, group=t % 3) for t, n in enumerate(sizes)], 8,
                                      torch.bfloat16, torch.bfloat16)
    chunks = [-(-n // 1024) for n in sizes]
    assert plan.numel == sum(sizes) and plan.n_chunks == sum(chunks) and plan.n_groups == 3
    assert len(table) == plan.table_bytes
    recs = np.frombuffer(table, dtype=np.int64, count=8 * len(sizes)).reshape(-1, 8)
    assert list(recs[:, 5]) == sizes
    assert list(recs[:, 6]) == list(np.cumsum([0] + chunks[:-1]))
    blocks = [-(-n // 256) for n in sizes]
    assert list(recs[:, 7] & 0xFFFFFFFF) == list(np.cumsum([0] + blocks[:-1]))
    owner = np.frombuffer(table, dtype=np.uint32, offset=64 * len(sizes), count=plan.n_chunks)
    assert list(owner) == [t for t, c in enumerate(chunks) for _ in range(c)]


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), "EINVAL"), (dict(n=5, group=8), "EINVAL"), (dict(n=5, group=-1), "EINVAL"),
    (dict(n=5, param=None), "EINVAL"), (dict(n=5, grad=None), "EINVAL"), (dict(n=5, exp_avg=None), "EINVAL"),
    (dict(n=5, reserved=1), "EINVAL"), (dict(n=5, grad=A + 1), "EALIGN"), (dict(n=5, master=A + 2), "EALIGN"),
    (dict(n=5, exp_avg=A + 4), "EALIGN"), (dict(n=5, exp_avg_sq=A + 1), "EALIGN"),
    (dict(n=1 << 42), "EINVAL")])
def test_plan_refuses(kw, code):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_tensors_plan([rec(kw.pop("n"), **kw)], 8, torch.bfloat16, torch.bfloat16, want_table=False)
    assert e.value.code == getattr(Z, "ZERO_" + code)


def test_plan_refuses_types_and_room():
    for args in ((16, Z.ZERO_BF16, 0), (32, 9, 0), (32, Z.ZERO_BF16, Z.ZERO_FP32)):
        with pytest.raises(Z.ZeroError):
            Z.zero_tensors_plan([rec(5)], *args, want_table=False)
    plan = _train_abi.zero_tensors_plan_t()
    room = ctypes.create_string_buffer(16)
    arr = (zero_tensor_t * 1)(rec(5))
    rc = train_lib().zero_tensors_plan(arr, 1, 32, Z.ZERO_BF16, Z.ZERO_BF16, ctypes.addressof(room), 16,
                                       ctypes.byref(plan))
    assert rc == Z.ZERO_ESIZE
    assert train_lib().zero_tensors_plan(None, 1, 32, 2, 2, None, 0, ctypes.byref(plan)) == Z.ZERO_EINVAL
    assert train_lib().zero_tensors_plan(arr, 1, 32, 2, 2, None, 0, None) == Z.ZERO_EINVAL


def step_args(**kw):
    a = zero_tensors_args()
    a.plan, _ = Z.zero_tensors_plan([rec(5000, group=1)], 32, torch.bfloat16, torch.bfloat16, want_table=False)
    groups = (_train_abi.zero_adam_group_t * 2)(*[(1e-3, 0.9, 0.999, 1e-8, 0.01)] * 2)
    a._groups = groups
    a.groups = groups
    a.n_groups, a.step, a.loss_scale, a.grad_predivide, a.max_grad_norm = 2, 1, 1.0, 1.0, 1.0
    a.table, a.workspace, a.result, a.workspace_bytes = A, A, A, 1 << 16
    for k, v in kw.items():
        if k.startswith("plan_"):
            setattr(a.plan, k[5:], v)
        elif k.startswith("g_"):
            setattr(groups[1], k[2:], v)
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(step=0), "EINVAL"), (dict(loss_scale=0.0), "EINVAL"), (dict(loss_scale=float("inf")), "EINVAL"),
    (dict(grad_predivide=-1.0), "EINVAL"), (dict(max_grad_norm=float("nan")), "EINVAL"),
    (dict(n_groups=1), "EINVAL"), (dict(n_groups=9), "EINVAL"), (dict(g_lr=-1.0), "EINVAL"),
    (dict(g_beta1=1.0), "EINVAL"), (dict(g_beta2=float("nan")), "EINVAL"), (dict(g_eps=0.0), "EINVAL"),
    (dict(g_weight_decay=float("inf")), "EINVAL"), (dict(peer_sumsq=-1.0), "EINVAL"),
    (dict(table=None), "EINVAL"), (dict(table=A + 8), "EALIGN"), (dict(workspace=None), "EINVAL"),
    (dict(result=None), "EINVAL"), (dict(result=A + 4), "EALIGN"), (dict(workspace_bytes=8), "ESIZE"),
    (dict(scalars=A + 4), "EALIGN"), (dict(plan_state_bits=16), "EINVAL"), (dict(plan_n_chunks=1), "EINVAL"),
    (dict(plan_n_chunks=99), "EINVAL"), (dict(plan_numel=-1), "EINVAL"), (dict(plan_n_groups=0), "EINVAL"),
    (dict(plan_table_bytes=16), "EINVAL")])
def test_step_refuses_before_any_work(kw, code):
    a = step_args(**kw)
    assert train_lib().zero_tensors_step(ctypes.byref(a), None, None) == getattr(Z, "ZERO_" + code)
    assert Z.zero_last_error()


def test_norm_and_apply_refuse():
    a = step_args()
    L = train_lib()
    assert L.zero_tensors_norm(ctypes.byref(a), -1, A, None) == Z.ZERO_EINVAL
    assert L.zero_tensors_norm(ctypes.byref(a), 0, None, None) == Z.ZERO_EINVAL
    assert L.zero_tensors_norm(ctypes.byref(a), 0, A + 8, None) == Z.ZERO_EALIGN
    assert L.zero_tensors_apply(ctypes.byref(a), None, None) == Z.ZERO_EINVAL
    assert L.zero_tensors_apply(ctypes.byref(a), A + 8, None) == Z.ZERO_EALIGN
    assert L.zero_tensors_step(None, None, None) == Z.ZERO_EINVAL


def test_scalars_are_the_step_constants():
    a = step_args(step=3, loss_scale=4.0, seed=(5 << 32) | 77)
    out = _train_abi.zero_tensors_scalars_t()
    assert train_lib().zero_tensors_scalars(ctypes.byref(a), ctypes.byref(out)) == Z.ZERO_OK
    f = np.float32
    g = out.group[1]
    assert out.inv_scale == f(0.25) and g.decay == f(1 - 1e-3 * 0.01) and g.step_size == f(1e-3 / (1 - 0.9**3))
    assert g.inv_sqrt_bc2 == f(1 / np.sqrt(1 - 0.999**3)) and g.one_minus_beta2 == f(1 - 0.999)
    assert out.key == 77 ^ int(train_ref._fmix(np.array([5], dtype=np.uint64))[0])


@pytest.mark.parametrize("call,code", [
    (lambda L: L.zero_state8_encode(A, A, -1, A, A, None), "EINVAL"),
    (lambda L: L.zero_state8_encode(None, A, 5, A, A, None), "EINVAL"),
    (lambda L: L.zero_state8_encode(A + 4, A, 5, A, A, None), "EALIGN"),
    (lambda L: L.zero_state8_encode(A, A, 5, A + 8, A, None), "EALIGN"),
    (lambda L: L.zero_state8_encode(A, A, 5, A, A + 1, None), "EALIGN"),
    (lambda L: L.zero_state8_decode(A, A, 5, A, None, 3, None), "EINVAL"),
    (lambda L: L.zero_state8_decode(A, A, 5, A, A, 4, None), "EINVAL"),
    (lambda L: L.zero_state8_decode(A, A, 0, None, None, 2, None), "OK")])
def test_state8_refuses(call, code):
    assert call(train_lib()) == getattr(Z, "ZERO_" + code)


def xent_args(**kw):
    a = zero_xent_args()
    a.tokens, a.dim, a.vocab = 10, 64, 100
    a.x_stride = a.w_stride = a.dx_stride = a.dw_stride = 64
    a.dtype, a.grad_scale = Z.ZERO_BF16, 1.0
    for n in ("x", "w", "target", "loss", "lse", "result", "dx", "dw", "workspace"):
        setattr(a, n, A)
    a.workspace_bytes = 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), "EINVAL"), (dict(dim=0), "EINVAL"), (dict(vocab=0), "EINVAL"), (dict(tokens=1 << 30), "EINVAL"),
    (dict(dtype=Z.ZERO_FP32), "EINVAL"), (dict(reserved=1), "EINVAL"), (dict(x=None), "EINVAL"),
    (dict(w=None), "EINVAL"), (dict(target=None), "EINVAL"), (dict(lse=None), "EINVAL"),
    (dict(result=None), "EINVAL"), (dict(result=A + 8), "EALIGN"), (dict(x=A + 1), "EALIGN"),
    (dict(target=A + 4), "EALIGN"), (dict(lse=A + 2), "EALIGN"), (dict(x_stride=63), "EINVAL"),
    (dict(w_stride=(1 << 31) + 1), "EINVAL"), (dict(workspace=None), "EINVAL"), (dict(workspace=A + 16), "EALIGN"),
    (dict(workspace_bytes=100), "ESIZE")])
def test_xent_refuses_before_any_work(kw, code):
    for call in (train_lib().zero_xent_forward, train_lib().zero_xent_backward):
        assert call(ctypes.byref(xent_args(**kw)), None) == getattr(Z, "ZERO_" + code)
        assert call(None, None) == Z.ZERO_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(dx=None), "EINVAL"), (dict(dw=None), "EINVAL"), (dict(dx=A + 1), "EALIGN"),
    (dict(dw_stride=10), "EINVAL"), (dict(grad_scale=float("nan")), "EINVAL")])
def test_xent_backward_refuses(kw, code):
    assert train_lib().zero_xent_backward(ctypes.byref(xent_args(**kw)), None) == getattr(Z, "ZERO_" + code)
    assert train_lib().zero_xent_forward(ctypes.byref(xent_args(loss=None)), None) == Z.ZERO_EINVAL


def test_xent_workspace_sizes():
    size = Z.zero_xent_workspace_bytes
    assert size(-1, 64, 100) == 0 and size(1, 0, 100) == 0 and size(1, 64, 0) == 0
    assert size(0, 0, 0) > 0 and size(1, 64, 100) % 256 == 0
    # far less than the logits of a large head in fp32
    assert size(8192, 4096, 128000) < 8192 * 128000 * 4 / 4


def test_binding_refuses_buffers_shorter_than_the_call_touches():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16)
    f, t = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    good = dict(x=x, w=w, target=t, loss=f, lse=f, result=torch.zeros(32, dtype=torch.uint8),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8), dx=x, dw=w)
    for kw in (dict(loss=f[:3]), dict(target=t[:3]), dict(w=w[:, :7]), dict(target=t.int()),
               dict(result=torch.zeros(31, dtype=torch.uint8)), dict(lse=f.double()), dict(x=x.t()),
               dict(w=w.half())):
        with pytest.raises(ValueError):
            Z.XentArgs(**{**good, **kw}).c_args(False)
    for kw in (dict(dx=None), dict(dw=w[:8]), dict(dx=x.float())):
        with pytest.raises(ValueError):
            Z.XentArgs(**{**good, **kw}).c_args(True)
    m, g = torch.zeros(300), torch.zeros(300, dtype=torch.bfloat16)
    s8, e8 = torch.zeros(1024, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        Z.TensorSet(master=[m], grad=[g[:299]], exp_avg=[m], exp_avg_sq=[m])
    with pytest.raises(ValueError):
        Z.TensorSet(master=[m], grad=[g], state8=[s8[:512]], scale8=[e8])
    with pytest.raises(ValueError):
        Z.TensorSet(master=[m], grad=[g], exp_avg=[m])
    with pytest.raises(ValueError):
        Z.TensorSet(master=[m], grad=[g], exp_avg=[m], exp_avg_sq=[m], group=[0, 1])
    with pytest.raises(ValueError):
        Z.TensorSet(master=[torch.zeros(30, 20).t()], grad=[g], exp_avg=[m], exp_avg_sq=[m])
    with pytest.raises(ValueError):
        Z.zero_state8_encode(m, m, s8[:512], e8)
    with pytest.raises(ValueError):
        Z.zero_state8_decode(s8, e8, m, g)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16)
    f, t = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    args = Z.XentArgs(x=x, w=w, target=t, loss=f, lse=f, result=torch.zeros(32, dtype=torch.uint8),
                      workspace=torch.zeros(1 << 16, dtype=torch.uint8), dx=x, dw=w)
    m, g = torch.zeros(300), torch.zeros(300, dtype=torch.bfloat16)
    s8, e8 = torch.zeros(1024, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8)
    for call in (lambda: Z.zero_xent_forward(args), lambda: Z.zero_xent_backward(args),
                 lambda: Z.TensorSet(master=[m], grad=[g], exp_avg=[m], exp_avg_sq=[m]),
                 lambda: Z.zero_state8_encode(m, m, s8, e8), lambda: Z.zero_state8_decode(s8, e8, m, m)):
        with pytest.raises(ValueError, match="device memory"):
            call()
