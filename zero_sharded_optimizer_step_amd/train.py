"""Binding of the training operators (include/zero/train.h): AdamW over a
list of tensors with 32-bit or 8-bit states, the conversion between the two,
the softmax cross entropy of a large vocabulary with its gradient, rows of
8-bit codes, and the gated activation and the product that read them, each
with its gradient.

As in the package's other calls, torch tensors become device pointers, the
current torch stream becomes the hipStream_t, negative status codes become
``ZeroError``, and a buffer too short for what a call touches is refused.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

# imported at the end of the package's own module, which defines these
from . import _dptr, _need, _stream, _torch, dtype_code
from ._abi import check, lib, zero_global_t
from ._train_abi import (ZERO_GLU_GELU, ZERO_GLU_SILU, ZERO_LINEAR8_BACKWARD, ZERO_LINEAR8_BACKWARD_ANY_DY,
                         ZERO_LINEAR8_FORWARD, ZERO_MAX_GROUPS, ZERO_STATE8_BLOCK, train_lib, zero_adam_group_t,
                         zero_glu8_args, zero_linear8_args, zero_tensor_t, zero_tensors_args, zero_tensors_plan_t,
                         zero_tensors_scalars_t, zero_xent_args, zero_xent_result_t)


def _on_device(**tensors) -> None:
    """Refuse host tensors and tensors of two devices: an address that the
    launching GPU does not hold would fault it (see _launching)."""
    first = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("%s is on %s; expected device memory" % (name, t.device))
        if first is None:
            first = name
        elif t.device != tensors[first].device:
            raise ValueError("%s is on %s, %s on %s" % (name, t.device, first, tensors[first].device))


def _launching(t) -> None:
    """Refuse tensors of another device than the current one, on which a call
    launches its kernels."""
    if t.is_cuda and t.device.index != _torch().cuda.current_device():
        raise ValueError("the tensors are on %s; the current device is cuda:%d"
                         % (t.device, _torch().cuda.current_device()))


def _contiguous(**tensors) -> None:
    """Refuse strided and expanded tensors where the library goes by the
    address alone."""
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError("%s is not contiguous" % name)


# ------------------------------------------------------------------ 8-bit states
def state8_blocks(n: int) -> int:
    """Blocks of ZERO_STATE8_BLOCK elements that n elements take: 512 bytes
    of state8 and 2 of scale8 each."""
    return -(-n // ZERO_STATE8_BLOCK)


def _need_state8(state8, scale8, n: int) -> None:
    _need(state8, 512 * state8_blocks(n), "state8")
    _need(scale8, 2 * state8_blocks(n), "scale8")


def zero_state8_encode(exp_avg, exp_avg_sq, state8, scale8, n: Optional[int] = None,
                       stream=None) -> None:
    """fp32 moments into the 8-bit state; n defaults to exp_avg.numel()."""
    n = exp_avg.numel() if n is None else n
    if exp_avg.dtype != _torch().float32 or exp_avg_sq.dtype != _torch().float32:
        raise ValueError("exp_avg and exp_avg_sq must be float32")
    _need(exp_avg, 4 * n, "exp_avg")
    _need(exp_avg_sq, 4 * n, "exp_avg_sq")
    _need_state8(state8, scale8, n)
    _contiguous(exp_avg=exp_avg, exp_avg_sq=exp_avg_sq, state8=state8, scale8=scale8)
    _on_device(exp_avg=exp_avg, exp_avg_sq=exp_avg_sq, state8=state8, scale8=scale8)
    _launching(exp_avg)
    check(train_lib().zero_state8_encode(_dptr(exp_avg), _dptr(exp_avg_sq), n, _dptr(state8),
                                         _dptr(scale8), _stream(stream)), "zero_state8_encode")


def zero_state8_decode(state8, scale8, exp_avg, exp_avg_sq, n: Optional[int] = None,
                       stream=None) -> None:
    """The 8-bit state into exp_avg and exp_avg_sq (fp32, bf16 or fp16, both
    the same); n defaults to exp_avg.numel()."""
    n = exp_avg.numel() if n is None else n
    if exp_avg.dtype != exp_avg_sq.dtype:
        raise ValueError("exp_avg is %s, exp_avg_sq is %s" % (exp_avg.dtype, exp_avg_sq.dtype))
    _need(exp_avg, exp_avg.element_size() * n, "exp_avg")
    _need(exp_avg_sq, exp_avg_sq.element_size() * n, "exp_avg_sq")
    _need_state8(state8, scale8, n)
    _contiguous(exp_avg=exp_avg, exp_avg_sq=exp_avg_sq, state8=state8, scale8=scale8)
    _on_device(exp_avg=exp_avg, exp_avg_sq=exp_avg_sq, state8=state8, scale8=scale8)
    _launching(exp_avg)
    check(train_lib().zero_state8_decode(_dptr(state8), _dptr(scale8), n, _dptr(exp_avg),
                                         _dptr(exp_avg_sq), dtype_code(exp_avg.dtype), _stream(stream)),
          "zero_state8_decode")


# ---------------------------------------------------------------- tensor lists
@dataclass
class AdamGroup:
    """Hyper-parameters of one group of a TensorSet."""
    lr: float = 6e-5
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01


def zero_tensors_plan(tensors: Sequence[zero_tensor_t], state_bits: int, grad_dtype, param_dtype=0,
                      want_table: bool = True):
    """(plan, table): the plan of a list and its table as host bytes (None
    without want_table)."""
    n = len(tensors)
    arr = (zero_tensor_t * max(n, 1))(*tensors)
    plan = zero_tensors_plan_t()
    call = train_lib().zero_tensors_plan
    check(call(arr, n, state_bits, dtype_code(grad_dtype), dtype_code(param_dtype), None, 0, ctypes.byref(plan)),
          "zero_tensors_plan")
    if not want_table:
        return plan, None
    table = bytearray(max(plan.table_bytes, 1))
    buf = (ctypes.c_char * len(table)).from_buffer(table)
    check(call(arr, n, state_bits, dtype_code(grad_dtype), dtype_code(param_dtype), ctypes.addressof(buf),
               len(table), ctypes.byref(plan)), "zero_tensors_plan")
    return plan, table


class TensorSet:
    """A list of tensors with their optimizer state, planned once.

    `master` (fp32) and `grad` are lists of contiguous device tensors; the
    state is `exp_avg` and `exp_avg_sq` (fp32) or `state8` and `scale8`
    (uint8, 512 and 2 bytes per block of 256 elements); `param` is the list of
    16-bit parameters to write, or None; `group[t]` is tensor t's group.
    The table holds their addresses: the set keeps that memory alive,
    whatever becomes of the lists and tensors given here, and a tensor that
    moves or is replaced (a gradient in new memory, say) needs a new set.
    It owns the table, the workspace and `result`, the device zero_global_t
    of the last step (32 bytes); calls on any stream may use them, one call
    after another.  All of a set's calls share these and one argument record:
    steps of one set that overlap, on two streams or from two threads,
    overwrite each other's partials and constants."""

    def __init__(self, master, grad, exp_avg=None, exp_avg_sq=None, state8=None, scale8=None,
                 param=None, group: Optional[Sequence[int]] = None):
        torch = _torch()
        if (exp_avg is None) != (exp_avg_sq is None) or (state8 is None) != (scale8 is None) or \
                (exp_avg is None) == (state8 is None):
            raise ValueError("give exp_avg and exp_avg_sq, or state8 and scale8")
        bits = 32 if state8 is None else 8
        first, second = (exp_avg, exp_avg_sq) if bits == 32 else (state8, scale8)
        n = len(master)
        group = [0] * n if group is None else list(group)
        for what, seq in (("grad", grad), ("first state", first), ("second state", second),
                          ("param", param), ("group", group)):
            if seq is not None and len(seq) != n:
                raise ValueError("%s has %d entries for %d masters" % (what, len(seq), n))
        grad_dtype = grad[0].dtype if n else torch.float32
        param_dtype = param[0].dtype if param is not None and n else None
        state_dtype = torch.float32 if bits == 32 else torch.uint8
        recs = []
        device = master[0].device if n else torch.device("cuda")
        for t in range(n):
            numel = master[t].numel()
            for what, x, dtype in (("master", master[t], torch.float32), ("grad", grad[t], grad_dtype),
                                   ("state", first[t], state_dtype), ("state", second[t], state_dtype),
                                   ("param", param[t] if param is not None else None, param_dtype)):
                if x is None:
                    continue
                if x.dtype != dtype:
                    raise ValueError("tensor %d: %s is %s, expected %s" % (t, what, x.dtype, dtype))
                if not x.is_contiguous():
                    raise ValueError("tensor %d: %s is not contiguous" % (t, what))
                if x.device != device:
                    _on_device(**{"master[0]": master[0], "%s[%d]" % (what, t): x})
            _need(grad[t], grad[t].element_size() * numel, "grad[%d]" % t)
            if bits == 32:
                _need(first[t], 4 * numel, "exp_avg[%d]" % t)
                _need(second[t], 4 * numel, "exp_avg_sq[%d]" % t)
            else:
                _need_state8(first[t], second[t], numel)
            if param is not None:
                _need(param[t], 2 * numel, "param[%d]" % t)
            recs.append(zero_tensor_t(_dptr(grad[t]), _dptr(master[t]), _dptr(first[t]), _dptr(second[t]),
                                      _dptr(param[t]) if param is not None else None, numel, group[t], 0))
        if n:
            _on_device(**{"master[0]": master[0]})       # and with it all others
        # the memory itself: the caller's lists may change, and what lies behind a tensor
        self._keep = [x.untyped_storage() for seq in (master, grad, first, second, param) if seq is not None
                      for x in seq if x is not None]
        self.state_bits = bits
        self.plan, table = zero_tensors_plan(recs, bits, grad_dtype,
                                             0 if param_dtype is None else dtype_code(param_dtype))
        self.table = torch.frombuffer(table, dtype=torch.uint8).to(device)
        self.workspace = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device=device)
        self.result = torch.zeros(32, dtype=torch.uint8, device=device)
        self._streams = set()                            # handles that may use the three at once
        if device.type == "cuda":
            # ready for a step on any stream: the fill is done, and so is what
            # used this memory before on the stream that it was allocated on
            torch.cuda.current_stream(device).synchronize()
            self._streams.add(torch.cuda.current_stream(device).cuda_stream)
        self._group_values = None
        a = self._c = zero_tensors_args()
        a.plan = self.plan
        a.table = _dptr(self.table)
        a.workspace = _dptr(self.workspace)
        a.workspace_bytes = self.workspace.numel()
        a.result = _dptr(self.result)

    def args(self, groups: Sequence[AdamGroup], step: int, loss_scale: float = 1.0,
             max_grad_norm: float = 1.0, seed: int = 0, grad_predivide: float = 1.0,
             peer_sumsq: float = 0.0, peer_overflow: bool = False, scalars=None) -> zero_tensors_args:
        """The zero_tensors_args of a call, the set's one record: it holds
        until the next call.  `scalars` is a device copy of a
        zero_tensors_scalars_t (288 bytes) or None."""
        a = self._c
        values = [(g.lr, g.beta1, g.beta2, g.eps, g.weight_decay) for g in groups]
        if values != self._group_values:
            self._groups = (zero_adam_group_t * max(len(values), 1))(*values)
            a.groups = self._groups
            a.n_groups = len(values)
            self._group_values = values
        a.step = step
        a.loss_scale = loss_scale
        a.grad_predivide = grad_predivide
        a.max_grad_norm = max_grad_norm
        a.peer_sumsq = peer_sumsq
        a.peer_overflow = 1 if peer_overflow else 0
        a.seed = seed & 0xFFFFFFFFFFFFFFFF
        if scalars is not None:
            _need(scalars, ctypes.sizeof(zero_tensors_scalars_t), "scalars")
            _contiguous(scalars=scalars)
            _on_device(**{"scalars": scalars, "the set": self.result})
        a.scalars = _dptr(scalars)
        return a

    def queue(self, stream=None) -> Optional[int]:
        """The handle of `stream` (default: the current one); the set's own
        buffers outlive what a call queues there."""
        _launching(self.result)
        handle = _stream(stream)
        if handle not in self._streams:
            torch = _torch()
            if stream is None:
                stream = torch.cuda.current_stream()
            elif isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream)
            for t in (self.table, self.workspace, self.result):
                t.record_stream(stream)
            self._streams.add(handle)
        return handle


def zero_tensors_step(tensors: TensorSet, groups: Sequence[AdamGroup], step: int,
                      want_info: bool = False, stream=None, **hyper) -> Optional[zero_global_t]:
    """One AdamW step over the set; hyper as TensorSet.args (loss_scale,
    max_grad_norm, seed, grad_predivide, peer_sumsq, peer_overflow, scalars).
    With want_info the call waits for the stream and returns the result."""
    a = tensors.args(groups, step, **hyper)
    info = zero_global_t() if want_info else None
    check(train_lib().zero_tensors_step(ctypes.byref(a), ctypes.byref(info) if want_info else None,
                                        tensors.queue(stream)), "zero_tensors_step")
    return info


def zero_tensors_norm(tensors: TensorSet, groups: Sequence[AdamGroup], step: int, slot: int, partials,
                      stream=None, **hyper) -> None:
    """The set's partial sums into slot `slot` of a zero_partials_bytes
    table, for zero_shard_combine."""
    _need(partials, (slot + 1) * lib().zero_partials_bytes(1), "partials")
    _contiguous(partials=partials)
    _on_device(**{"partials": partials, "the set": tensors.result})
    check(train_lib().zero_tensors_norm(ctypes.byref(tensors.args(groups, step, **hyper)), slot,
                                        _dptr(partials), tensors.queue(stream)), "zero_tensors_norm")


def zero_tensors_apply(tensors: TensorSet, groups: Sequence[AdamGroup], step: int, global_buf,
                       stream=None, **hyper) -> None:
    """The update by a zero_global_t in device memory."""
    _need(global_buf, ctypes.sizeof(zero_global_t), "global_buf")
    _contiguous(global_buf=global_buf)
    _on_device(**{"global_buf": global_buf, "the set": tensors.result})
    check(train_lib().zero_tensors_apply(ctypes.byref(tensors.args(groups, step, **hyper)),
                                         _dptr(global_buf), tensors.queue(stream)), "zero_tensors_apply")


def zero_tensors_scalars(tensors: TensorSet, groups: Sequence[AdamGroup], step: int,
                         **hyper) -> zero_tensors_scalars_t:
    """The step's constants as the kernels take them (host)."""
    out = zero_tensors_scalars_t()
    check(train_lib().zero_tensors_scalars(ctypes.byref(tensors.args(groups, step, **hyper)),
                                           ctypes.byref(out)), "zero_tensors_scalars")
    return out


# --------------------------------------------------------------- cross entropy
def zero_xent_workspace_bytes(tokens: int, dim: int, vocab: int) -> int:
    return train_lib().zero_xent_workspace_bytes(tokens, dim, vocab)


@dataclass
class XentArgs:
    """Builds a zero_xent_args from torch tensors: x [tokens, dim] and w
    [vocab, dim] (fp16 or bf16, rows contiguous, any row stride), target
    int64[tokens], loss and lse fp32[tokens], result uint8[32], and for the
    backward dx and dw like x and w."""
    x: object
    w: object
    target: object
    loss: object
    lse: object
    result: object
    workspace: object
    dx: object = None
    dw: object = None
    grad_scale: float = 1.0

    def c_args(self, backward: bool) -> zero_xent_args:
        torch = _torch()
        a = zero_xent_args()
        x, w = self.x, self.w
        if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
            raise ValueError("x is %s and w is %s; expected [tokens, dim] and [vocab, dim]"
                             % (tuple(x.shape), tuple(w.shape)))
        t, d, v = x.shape[0], x.shape[1], w.shape[0]
        a.tokens, a.dim, a.vocab = t, d, v
        a.dtype = dtype_code(x.dtype)
        mats = [("x", x, (t, d)), ("w", w, (v, d))]
        if backward:
            if self.dx is None or self.dw is None:
                raise ValueError("the backward needs dx and dw")
            mats += [("dx", self.dx, (t, d)), ("dw", self.dw, (v, d))]
        for name, m, shape in mats:
            if m.dtype != x.dtype:
                raise ValueError("%s is %s, x is %s" % (name, m.dtype, x.dtype))
            if tuple(m.shape) != shape:
                raise ValueError("%s is %s, expected %s" % (name, tuple(m.shape), shape))
            if shape[1] > 1 and shape[0] > 0 and m.stride(1) != 1:
                raise ValueError("%s's rows are not contiguous" % name)
            setattr(a, name, _dptr(m))
            # a single row may carry any stride; the library wants dim or more
            setattr(a, name + "_stride", m.stride(0) if shape[0] > 1 else max(m.stride(0), d))
        if self.target.dtype != torch.int64 or not self.target.is_contiguous():
            raise ValueError("target must be a contiguous int64 tensor")
        for name, m in (("loss", self.loss), ("lse", self.lse)):
            if m.dtype != torch.float32 or not m.is_contiguous():
                raise ValueError("%s must be a contiguous float32 tensor" % name)
            _need(m, 4 * t, name)
        _need(self.target, 8 * t, "target")
        _need(self.result, ctypes.sizeof(zero_xent_result_t), "result")
        _contiguous(result=self.result, workspace=self.workspace)
        _on_device(x=x, w=w, target=self.target, loss=self.loss, lse=self.lse, result=self.result,
                   workspace=self.workspace, dx=self.dx if backward else None, dw=self.dw if backward else None)
        a.target, a.loss, a.lse = _dptr(self.target), _dptr(self.loss), _dptr(self.lse)
        a.result = _dptr(self.result)
        a.grad_scale = self.grad_scale
        a.workspace = _dptr(self.workspace)
        a.workspace_bytes = self.workspace.numel() * self.workspace.element_size()
        return a


def zero_xent_forward(args: XentArgs, stream=None) -> None:
    """loss, lse and result of args."""
    a = args.c_args(False)
    _launching(args.x)
    check(train_lib().zero_xent_forward(ctypes.byref(a), _stream(stream)),
          "zero_xent_forward")


def zero_xent_backward(args: XentArgs, stream=None) -> None:
    """dx and dw of args, after zero_xent_forward of the same args."""
    a = args.c_args(True)
    _launching(args.x)
    check(train_lib().zero_xent_backward(ctypes.byref(a), _stream(stream)),
          "zero_xent_backward")


# ----------------------------------------------------------- rows of 8-bit codes
def rows8_stride(dim: int) -> int:
    """Bytes that a row of dim codes takes: dim rounded up to a multiple of
    16, zeros from dim on."""
    return (dim + 15) // 16 * 16


def _rows(name: str, t, rows: int, cols: int, dtype) -> int:
    """The row stride of a matrix [rows, cols] of any row stride."""
    if t.dtype != dtype:
        raise ValueError("%s is %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != (rows, cols):
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), (rows, cols)))
    stride, along = t.stride()
    if along != 1 and cols > 1 and rows > 0:
        raise ValueError("%s's rows are not contiguous" % name)
    # a single row may carry any stride; the library wants cols or more
    return stride if rows > 1 else max(stride, cols)


def _codes(name: str, t, scale, rows: int, dim: int) -> int:
    """The row stride of codes int8 [rows, rows8_stride(dim) or more]."""
    torch = _torch()
    if scale is None or t is None:
        raise ValueError("%s and its scale are given together" % name)
    if t.dtype != torch.int8:
        raise ValueError("%s is %s, expected torch.int8" % (name, t.dtype))
    wide = (dim + 15) // 16 * 16
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < wide:
        raise ValueError("%s is %s, expected [%d, %d or more]" % (name, tuple(shape), rows, wide))
    stride, along = t.stride()
    if along != 1 and wide > 0 and rows > 0:
        raise ValueError("%s's rows are not contiguous" % name)
    if scale.dtype != torch.float32 or scale.numel() != rows or not scale.is_contiguous():
        raise ValueError("%s's scale must be %d contiguous float32 values" % (name, rows))
    # one row, or rows of nothing, may carry any stride, also none that is a multiple of 16
    return stride if rows > 1 and wide > 0 else wide


_DTYPE_CODES = {}


def _dtype(dtype) -> int:
    """dtype_code, looked up."""
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        code = _DTYPE_CODES[dtype] = dtype_code(dtype)
    return code


def _one_device(given: dict) -> None:
    """As _on_device; where all tensors say the same device's number, without
    building what an error would show."""
    first = None
    for t in given.values():
        if first is None:
            first = t.get_device()
            if first < 0:
                break
        elif t.get_device() != first:
            break
    else:
        return
    _on_device(**given)


def _queue(t, stream):
    """The handle of the stream that a call on t's device launches on; as
    _launching and _stream."""
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and t.is_cuda:
            device = torch.cuda.current_device()
            if t.get_device() == device:
                return raw(device)
    _launching(t)
    return _stream(stream)


def zero_rows8_encode(x, codes, scale, stream=None) -> None:
    """Rows of x [rows, dim] (fp32, bf16 or fp16, any row stride) into codes
    int8 [rows, rows8_stride(dim) or more] and scale fp32 [rows]."""
    if x.dim() != 2:
        raise ValueError("x is %s; expected [rows, dim]" % (tuple(x.shape),))
    rows, dim = x.shape
    xs, cs = _rows("x", x, rows, dim, x.dtype), _codes("codes", codes, scale, rows, dim)
    _one_device({"x": x, "codes": codes, "scale": scale})
    check(train_lib().zero_rows8_encode(x.data_ptr(), xs, _dtype(x.dtype), rows, dim, codes.data_ptr(), cs,
                                        scale.data_ptr(), _queue(x, stream)), "zero_rows8_encode")


def zero_rows8_decode(codes, scale, y, stream=None) -> None:
    """The rows that codes and scale stand for into y [rows, dim] (fp32, bf16
    or fp16, any row stride)."""
    if y.dim() != 2:
        raise ValueError("y is %s; expected [rows, dim]" % (tuple(y.shape),))
    rows, dim = y.shape
    ys, cs = _rows("y", y, rows, dim, y.dtype), _codes("codes", codes, scale, rows, dim)
    _one_device({"y": y, "codes": codes, "scale": scale})
    check(train_lib().zero_rows8_decode(codes.data_ptr(), cs, scale.data_ptr(), rows, dim, y.data_ptr(), ys,
                                        _dtype(y.dtype), _queue(y, stream)), "zero_rows8_decode")


# ------------------------------------------------------------- gated activation
_GLU_KINDS = {"silu": ZERO_GLU_SILU, "gelu": ZERO_GLU_GELU}


@dataclass
class Glu8Args:
    """Builds a zero_glu8_args from torch tensors: gate, up, h, dh, dgate and
    dup [tokens, width] (fp16 or bf16, any row stride), gate8, up8 and h8 int8
    [tokens, rows8_stride(width) or more] with scales fp32 [tokens].  Without
    up the activation is not gated (then no up8 and dup either).  The forward
    takes gate and up and writes h, h8 or both, and, where gate8 is given,
    the checkpoint gate8 and up8; the backward takes dh and the checkpoint
    alone."""
    kind: str = "silu"
    gate: object = None
    up: object = None
    gate8: object = None
    gate_scale: object = None
    up8: object = None
    up_scale: object = None
    h: object = None
    h8: object = None
    h_scale: object = None
    dh: object = None
    dgate: object = None
    dup: object = None

    def c_args(self, backward: bool) -> zero_glu8_args:
        a = zero_glu8_args()
        first = self.dh if backward else self.gate
        if first is None or first.dim() != 2:
            raise ValueError("%s must be a tensor [tokens, width]" % ("dh" if backward else "gate"))
        if self.kind not in _GLU_KINDS:
            raise ValueError("kind is %r, expected one of %s" % (self.kind, sorted(_GLU_KINDS)))
        (t, w), dtype = first.shape, first.dtype
        a.tokens, a.width = t, w
        a.dtype, a.kind = _dtype(dtype), _GLU_KINDS[self.kind]
        given = {}
        if backward:
            if self.dgate is None or self.gate8 is None:
                raise ValueError("the backward needs gate8 and dgate")
            given["dh"], a.dh, a.dh_stride = first, first.data_ptr(), _rows("dh", first, t, w, dtype)
            m = given["dgate"] = self.dgate
            a.dgate, a.dgate_stride = m.data_ptr(), _rows("dgate", m, t, w, dtype)
            m = self.dup
            if m is not None:
                given["dup"], a.dup, a.dup_stride = m, m.data_ptr(), _rows("dup", m, t, w, dtype)
        else:
            given["gate"], a.gate, a.gate_stride = first, first.data_ptr(), _rows("gate", first, t, w, dtype)
            m = self.up
            if m is not None:
                given["up"], a.up, a.up_stride = m, m.data_ptr(), _rows("up", m, t, w, dtype)
            m = self.h
            if m is not None:
                given["h"], a.h, a.h_stride = m, m.data_ptr(), _rows("h", m, t, w, dtype)
            q, m = self.h8, self.h_scale
            if q is not None or m is not None:
                a.h8_stride = _codes("h8", q, m, t, w)
                given["h8"], given["h_scale"], a.h8, a.h_scale = q, m, q.data_ptr(), m.data_ptr()
        q, m = self.gate8, self.gate_scale
        if q is not None or m is not None:
            a.gate8_stride = _codes("gate8", q, m, t, w)
            given["gate8"], given["gate_scale"], a.gate8, a.gate_scale = q, m, q.data_ptr(), m.data_ptr()
        q, m = self.up8, self.up_scale
        if q is not None or m is not None:
            a.up8_stride = _codes("up8", q, m, t, w)
            given["up8"], given["up_scale"], a.up8, a.up_scale = q, m, q.data_ptr(), m.data_ptr()
        _one_device(given)
        return a


def zero_glu8_forward(args: Glu8Args, stream=None) -> None:
    """h, h8 and the checkpoint of args, as far as they are given."""
    a = args.c_args(False)
    check(train_lib().zero_glu8_forward(ctypes.byref(a), _queue(args.gate, stream)), "zero_glu8_forward")


def zero_glu8_backward(args: Glu8Args, stream=None) -> None:
    """dgate and dup of args from dh and the checkpoint."""
    a = args.c_args(True)
    check(train_lib().zero_glu8_backward(ctypes.byref(a), _queue(args.dh, stream)), "zero_glu8_backward")


# ---------------------------------------------------------------- 8-bit products
def zero_linear8_workspace_bytes_for(tokens: int, dim: int, out: int, uses: int) -> int:
    """Bytes of workspace for calls of up to `tokens` tokens, of the uses named:
    ZERO_LINEAR8_FORWARD, ZERO_LINEAR8_BACKWARD, ZERO_LINEAR8_BACKWARD_ANY_DY."""
    return train_lib().zero_linear8_workspace_bytes_for(tokens, dim, out, uses)


def zero_linear8_workspace_bytes(tokens: int, dim: int, out: int, forward: bool = True, backward: bool = True,
                                 any_dy: bool = True) -> int:
    """Bytes of workspace for calls of up to `tokens` tokens: of the forward,
    of the backward, or of both.  Without any_dy the backward's dy has rows of
    whole 16-byte pieces (16-byte aligned, out and the stride multiples of 8),
    which it reads where they lie."""
    uses = (ZERO_LINEAR8_FORWARD if forward else 0) | \
        ((ZERO_LINEAR8_BACKWARD_ANY_DY if any_dy else ZERO_LINEAR8_BACKWARD) if backward else 0)
    if not uses:
        raise ValueError("a workspace for neither the forward nor the backward")
    return zero_linear8_workspace_bytes_for(tokens, dim, out, uses)


@dataclass
class Linear8Args:
    """Builds a zero_linear8_args from torch tensors: x8 int8 [tokens,
    rows8_stride(dim) or more] and w8 int8 [out, the same] with scales fp32
    [tokens] and [out]; bias [out] or None and y [tokens, out] for the
    forward; dy [tokens, out] and those of dx [tokens, dim], dw [out, dim]
    and db [out] that are wanted for the backward (fp16 or bf16, matrices of
    any row stride).  A backward without dx needs no w8, one without dw no
    x8."""
    x8: object
    x_scale: object
    w8: object
    w_scale: object
    dim: int
    workspace: object
    bias: object = None
    y: object = None
    dy: object = None
    dx: object = None
    dw: object = None
    db: object = None

    def c_args(self, backward: bool) -> zero_linear8_args:
        a = zero_linear8_args()
        first = self.dy if backward else self.y
        if first is None or first.dim() != 2:
            raise ValueError("%s must be a tensor [tokens, out]" % ("dy" if backward else "y"))
        (t, n), k, dtype = first.shape, self.dim, first.dtype
        a.tokens, a.dim, a.out, a.dtype = t, k, n, _dtype(dtype)
        m = self.workspace
        if not m.is_contiguous():
            raise ValueError("workspace is not contiguous")
        a.workspace, a.workspace_bytes = m.data_ptr(), m.numel() * m.element_size()
        given = {"workspace": m}
        if backward:
            given["dy"], a.dy, a.dy_stride = first, first.data_ptr(), _rows("dy", first, t, n, dtype)
            dx, dw = self.dx, self.dw
            if dx is not None:
                given["dx"], a.dx, a.dx_stride = dx, dx.data_ptr(), _rows("dx", dx, t, k, dtype)
            if dw is not None:
                given["dw"], a.dw, a.dw_stride = dw, dw.data_ptr(), _rows("dw", dw, n, k, dtype)
            v, name = self.db, "db"
        else:
            given["y"], a.y, a.y_stride = first, first.data_ptr(), _rows("y", first, t, n, dtype)
            v, name = self.bias, "bias"
        if v is not None:
            if v.dtype != dtype or v.numel() != n or not v.is_contiguous():
                raise ValueError("%s must be %d contiguous %s values" % (name, n, dtype))
            given[name] = v
            if backward:
                a.db = v.data_ptr()
            else:
                a.bias = v.data_ptr()
        if not backward or dw is not None:
            q, m = self.x8, self.x_scale
            a.x8_stride = _codes("x8", q, m, t, k)
            given["x8"], given["x_scale"], a.x8, a.x_scale = q, m, q.data_ptr(), m.data_ptr()
        if not backward or dx is not None:
            q, m = self.w8, self.w_scale
            a.w8_stride = _codes("w8", q, m, n, k)
            given["w8"], given["w_scale"], a.w8, a.w_scale = q, m, q.data_ptr(), m.data_ptr()
        _one_device(given)
        return a


def zero_linear8_forward(args: Linear8Args, stream=None) -> None:
    """y of args."""
    a = args.c_args(False)
    check(train_lib().zero_linear8_forward(ctypes.byref(a), _queue(args.y, stream)), "zero_linear8_forward")


def zero_linear8_backward(args: Linear8Args, stream=None) -> None:
    """Those of dx, dw and db of args that are given."""
    a = args.c_args(True)
    check(train_lib().zero_linear8_backward(ctypes.byref(a), _queue(args.dy, stream)), "zero_linear8_backward")
