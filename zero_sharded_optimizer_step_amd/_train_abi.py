"""ctypes mirror of include/zero/train.h and the loader of
libzero_train_mi355x.so, which lies next to libzero_mi355x.so and uses it.
Marshalling only; there is no fallback path."""
from __future__ import annotations

import ctypes
import os

from . import _abi
from ._abi import f32, f64, i32, i64, sz, vp, zero_global_t

TRAIN_LIB_PATH = os.path.join(_abi.PKG, "libzero_train_mi355x.so")

ZERO_STATE8_BLOCK = 256
ZERO_MAX_GROUPS = 8
ZERO_ROWS8_MAX_DIM = 131071
ZERO_GLU_SILU, ZERO_GLU_GELU = 0, 1
ZERO_LINEAR8_FORWARD, ZERO_LINEAR8_BACKWARD, ZERO_LINEAR8_BACKWARD_ANY_DY = 1, 2, 4
u32, u64 = ctypes.c_uint32, ctypes.c_uint64


class zero_tensor_t(ctypes.Structure):
    _fields_ = [("grad", vp), ("master", vp), ("exp_avg", vp), ("exp_avg_sq", vp), ("param", vp),
                ("numel", i64), ("group", i32), ("reserved", i32)]


class zero_tensors_plan_t(ctypes.Structure):
    _fields_ = [("numel", i64), ("n_chunks", i64), ("n_tensors", i32), ("n_groups", i32),
                ("state_bits", i32), ("grad_dtype", i32), ("param_dtype", i32), ("reserved", i32),
                ("table_bytes", u64), ("workspace_bytes", u64)]


class zero_adam_group_t(ctypes.Structure):
    _fields_ = [("lr", f64), ("beta1", f64), ("beta2", f64), ("eps", f64), ("weight_decay", f64)]


class zero_group_scalars_t(ctypes.Structure):
    _fields_ = [(n, f32) for n in ("decay", "beta1", "one_minus_beta1", "beta2", "one_minus_beta2",
                                   "step_size", "inv_sqrt_bc2", "eps")]


class zero_tensors_scalars_t(ctypes.Structure):
    _fields_ = [("inv_scale", f32), ("peer_overflow", i32), ("key", u32), ("reserved", u32),
                ("max_grad_norm", f64), ("peer_sumsq", f64),
                ("group", zero_group_scalars_t * ZERO_MAX_GROUPS)]


assert ctypes.sizeof(zero_tensors_scalars_t) == 288


class zero_tensors_args(ctypes.Structure):
    _fields_ = [("plan", zero_tensors_plan_t), ("table", vp), ("workspace", vp),
                ("workspace_bytes", sz), ("groups", ctypes.POINTER(zero_adam_group_t)),
                ("n_groups", i32), ("peer_overflow", i32), ("step", i64), ("loss_scale", f64),
                ("grad_predivide", f64), ("max_grad_norm", f64), ("peer_sumsq", f64), ("seed", u64),
                ("result", vp), ("scalars", vp)]


class zero_xent_result_t(ctypes.Structure):
    _fields_ = [("loss_sum", f64), ("count", i64), ("out_of_range", i32), ("reserved", i32),
                ("mean", f32), ("inv_count", f32)]


assert ctypes.sizeof(zero_xent_result_t) == 32


class zero_xent_args(ctypes.Structure):
    _fields_ = [("tokens", i64), ("dim", i64), ("vocab", i64), ("x_stride", i64), ("w_stride", i64),
                ("dx_stride", i64), ("dw_stride", i64), ("dtype", i32), ("reserved", i32),
                ("x", vp), ("w", vp), ("target", vp), ("loss", vp), ("lse", vp), ("result", vp),
                ("dx", vp), ("dw", vp), ("grad_scale", f64), ("workspace", vp),
                ("workspace_bytes", sz)]


class zero_glu8_args(ctypes.Structure):
    _fields_ = [("tokens", i64), ("width", i64), ("gate_stride", i64), ("up_stride", i64),
                ("h_stride", i64), ("dh_stride", i64), ("dgate_stride", i64), ("dup_stride", i64),
                ("gate8_stride", i64), ("up8_stride", i64), ("h8_stride", i64), ("dtype", i32),
                ("kind", i32), ("gate", vp), ("up", vp), ("gate8", vp), ("gate_scale", vp),
                ("up8", vp), ("up_scale", vp), ("h", vp), ("h8", vp), ("h_scale", vp), ("dh", vp),
                ("dgate", vp), ("dup", vp)]


class zero_linear8_args(ctypes.Structure):
    _fields_ = [("tokens", i64), ("dim", i64), ("out", i64), ("x8_stride", i64), ("w8_stride", i64),
                ("y_stride", i64), ("dy_stride", i64), ("dx_stride", i64), ("dw_stride", i64),
                ("dtype", i32), ("reserved", i32), ("x8", vp), ("x_scale", vp), ("w8", vp),
                ("w_scale", vp), ("bias", vp), ("y", vp), ("dy", vp), ("dx", vp), ("dw", vp),
                ("db", vp), ("workspace", vp), ("workspace_bytes", sz)]


_P = ctypes.POINTER
_PROTOTYPES = {
    "zero_state8_encode": (ctypes.c_int, [vp, vp, i64, vp, vp, vp]),
    "zero_state8_decode": (ctypes.c_int, [vp, vp, i64, vp, vp, i32, vp]),
    "zero_tensors_plan": (ctypes.c_int, [_P(zero_tensor_t), i32, i32, i32, i32, vp, sz,
                                         _P(zero_tensors_plan_t)]),
    "zero_tensors_step": (ctypes.c_int, [_P(zero_tensors_args), _P(zero_global_t), vp]),
    "zero_tensors_norm": (ctypes.c_int, [_P(zero_tensors_args), i32, vp, vp]),
    "zero_tensors_apply": (ctypes.c_int, [_P(zero_tensors_args), vp, vp]),
    "zero_tensors_scalars": (ctypes.c_int, [_P(zero_tensors_args), _P(zero_tensors_scalars_t)]),
    "zero_xent_workspace_bytes": (sz, [i64, i64, i64]),
    "zero_xent_forward": (ctypes.c_int, [_P(zero_xent_args), vp]),
    "zero_xent_backward": (ctypes.c_int, [_P(zero_xent_args), vp]),
    "zero_rows8_encode": (ctypes.c_int, [vp, i64, i32, i64, i64, vp, i64, vp, vp]),
    "zero_rows8_decode": (ctypes.c_int, [vp, i64, vp, i64, i64, vp, i64, i32, vp]),
    "zero_glu8_forward": (ctypes.c_int, [_P(zero_glu8_args), vp]),
    "zero_glu8_backward": (ctypes.c_int, [_P(zero_glu8_args), vp]),
    "zero_linear8_workspace_bytes": (sz, [i64, i64, i64]),
    "zero_linear8_workspace_bytes_for": (sz, [i64, i64, i64, i32]),
    "zero_linear8_forward": (ctypes.c_int, [_P(zero_linear8_args), vp]),
    "zero_linear8_backward": (ctypes.c_int, [_P(zero_linear8_args), vp]),
}

_lib = None


def train_lib() -> ctypes.CDLL:
    """The loaded HIP library of the training operators; raises if it has
    not been built."""
    global _lib
    if _lib is None:
        _abi.lib()
        if not os.path.exists(TRAIN_LIB_PATH):
            raise ImportError(
                "libzero_train_mi355x.so is not built (expected at %s); run "
                "`python -m zero_sharded_optimizer_step_amd.build`" % TRAIN_LIB_PATH)
        L = ctypes.CDLL(TRAIN_LIB_PATH)
        for name, (res, args) in _PROTOTYPES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib
