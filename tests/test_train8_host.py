"""CPU tests of the 8-bit training operators: what the library and its binding
refuse before any work, and the definitions that the GPU tests compare with.
No call here reaches the HIP runtime."""
import ctypes

import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from zero_sharded_optimizer_step_amd import train
from zero_sharded_optimizer_step_amd._train_abi import train_lib, zero_glu8_args, zero_linear8_args

A = 1 << 20                                  # stands for a device address; never read
TOP = 1 << 31


def rows8(x=A, x_stride=100, dtype=Z.ZERO_BF16, rows=10, dim=100, codes=A, codes_stride=112, scale=A):
    L = train_lib()
    return (L.zero_rows8_encode(x, x_stride, dtype, rows, dim, codes, codes_stride, scale, None),
            L.zero_rows8_decode(codes, codes_stride, scale, rows, dim, x, x_stride, dtype, None))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "EINVAL"), (dict(rows=TOP), "EINVAL"), (dict(dim=-1), "EINVAL"), (dict(dim=131072), "EINVAL"),
    (dict(dtype=0), "EINVAL"), (dict(dtype=4), "EINVAL"), (dict(x=None), "EINVAL"), (dict(codes=None), "EINVAL"),
    (dict(scale=None), "EINVAL"), (dict(x_stride=99), "EINVAL"), (dict(x_stride=TOP + 1), "EINVAL"),
    (dict(codes_stride=96), "EINVAL"), (dict(codes_stride=TOP + 16), "EINVAL"), (dict(codes_stride=120), "EALIGN"),
    (dict(codes=A + 8), "EALIGN"), (dict(x=A + 1), "EALIGN"), (dict(x=A + 2, dtype=Z.ZERO_FP32), "EALIGN"),
    (dict(scale=A + 2), "EALIGN"), (dict(rows=0, x=None, codes=None, scale=None), "OK")])
def test_rows8_refuses(kw, code):
    assert rows8(**kw) == (getattr(Z, "ZERO_" + code),) * 2


def glu_args(**kw):
    a = zero_glu8_args()
    a.tokens, a.width, a.dtype, a.kind = 10, 100, Z.ZERO_BF16, Z.ZERO_GLU_SILU
    for n in ("gate", "up", "h", "dh", "dgate", "dup"):
        setattr(a, n, A)
        setattr(a, n + "_stride", 100)
    for n in ("gate8", "up8", "h8"):
        setattr(a, n, A)
        setattr(a, n + "_stride", 112)
        setattr(a, n[:-1] + "_scale", A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BOTH = [(dict(tokens=-1), "EINVAL"), (dict(tokens=TOP), "EINVAL"), (dict(width=-1), "EINVAL"),
        (dict(width=131072), "EINVAL"), (dict(dtype=Z.ZERO_FP32), "EINVAL"), (dict(kind=2), "EINVAL"),
        (dict(kind=-1), "EINVAL"), (dict(gate_scale=None), "EINVAL"), (dict(up_scale=None), "EINVAL"),
        (dict(gate8_stride=96), "EINVAL"), (dict(gate8_stride=120), "EALIGN"), (dict(gate8=A + 4), "EALIGN"),
        (dict(up8=None), "EINVAL"), (dict(up8=A + 8), "EALIGN"), (dict(up8_stride=96), "EINVAL"),
        (dict(gate8=None), "EINVAL"), (dict(up_scale=A + 1), "EALIGN")]
FORWARD = [(dict(gate=None), "EINVAL"), (dict(gate_stride=99), "EINVAL"), (dict(up_stride=99), "EINVAL"),
           (dict(gate=A + 1), "EALIGN"), (dict(up=A + 1), "EALIGN"), (dict(up=None), "EINVAL"),
           (dict(h=None, h8=None), "EINVAL"), (dict(h=A + 1), "EALIGN"), (dict(h_stride=99), "EINVAL"),
           (dict(h8_stride=96), "EINVAL"), (dict(h_scale=None), "EINVAL"), (dict(h8=A + 8), "EALIGN"),
           (dict(h_stride=TOP + 1), "EINVAL"), (dict(tokens=0), "OK"), (dict(width=0), "OK")]
BACKWARD = [(dict(dh=None), "EINVAL"), (dict(dgate=None), "EINVAL"), (dict(dup=None), "EINVAL"),
            (dict(dh=A + 1), "EALIGN"), (dict(dup=A + 1), "EALIGN"), (dict(dh_stride=99), "EINVAL"),
            (dict(dgate_stride=99), "EINVAL"), (dict(dup_stride=TOP + 1), "EINVAL"), (dict(tokens=0), "OK"),
            (dict(width=0), "OK")]


@pytest.mark.parametrize("kw,code", BOTH)
def test_glu8_refuses(kw, code):
    for call in (train_lib().zero_glu8_forward, train_lib().zero_glu8_backward):
        assert call(ctypes.byref(glu_args(**kw)), None) == getattr(Z, "ZERO_" + code)
        assert call(None, None) == Z.ZERO_EINVAL


@pytest.mark.parametrize("way,kw,code", [("forward", *c) for c in FORWARD] + [("backward", *c) for c in BACKWARD])
def test_glu8_refuses_each_way(way, kw, code):
    call = getattr(train_lib(), "zero_glu8_" + way)
    assert call(ctypes.byref(glu_args(**kw)), None) == getattr(Z, "ZERO_" + code)


@pytest.mark.parametrize("kw,why", [
    (dict(), "dgate and dup"), (dict(dh=2 * A), "dgate and dup"),
    (dict(dup=2 * A, dgate_stride=104), "another stride"), (dict(dgate=2 * A, dup_stride=104), "another stride"),
    (dict(dup=2 * A, dh_stride=104), "another stride")])
def test_glu8_gradients_in_one_memory(kw, why):
    """dgate or dup may be dh's memory, with its stride, and neither the other's."""
    call = train_lib().zero_glu8_backward
    assert call(ctypes.byref(glu_args(**kw)), None) == Z.ZERO_EINVAL
    assert why in Z.zero_last_error()
    # where there is nothing to write it does not matter
    for none in (dict(tokens=0), dict(width=0)):
        assert call(ctypes.byref(glu_args(**{**kw, **none})), None) == Z.ZERO_OK


def linear_args(**kw):
    a = zero_linear8_args()
    a.tokens, a.dim, a.out, a.dtype = 10, 100, 70, Z.ZERO_FP16
    a.x8_stride = a.w8_stride = 112
    a.y_stride = a.dy_stride = 70
    a.dx_stride = a.dw_stride = 100
    for n in ("x8", "x_scale", "w8", "w_scale", "bias", "y", "dy", "dx", "dw", "db", "workspace"):
        setattr(a, n, A)
    a.workspace_bytes = 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), "EINVAL"), (dict(dim=-1), "EINVAL"), (dict(out=-1), "EINVAL"), (dict(tokens=(1 << 20) + 1), "EINVAL"),
    (dict(dim=131072), "EINVAL"), (dict(out=(1 << 20) + 1), "EINVAL"), (dict(dtype=Z.ZERO_FP32), "EINVAL"),
    (dict(reserved=1), "EINVAL"), (dict(x8=None), "EINVAL"), (dict(w8=None), "EINVAL"), (dict(x_scale=None), "EINVAL"),
    (dict(w_scale=None), "EINVAL"), (dict(x8_stride=96), "EINVAL"), (dict(w8_stride=(1 << 22) + 16), "EINVAL"),
    (dict(x8_stride=120), "EALIGN"), (dict(w8=A + 8), "EALIGN"), (dict(x_scale=A + 2), "EALIGN"),
    (dict(workspace=None), "EINVAL"), (dict(workspace=A + 16), "EALIGN"), (dict(workspace_bytes=100), "ESIZE")])
def test_linear8_refuses(kw, code):
    for call in (train_lib().zero_linear8_forward, train_lib().zero_linear8_backward):
        assert call(ctypes.byref(linear_args(**kw)), None) == getattr(Z, "ZERO_" + code)
        assert call(None, None) == Z.ZERO_EINVAL


@pytest.mark.parametrize("way,kw,code", [
    ("forward", dict(y=None), "EINVAL"), ("forward", dict(y=A + 1), "EALIGN"), ("forward", dict(y_stride=69), "EINVAL"),
    ("forward", dict(bias=A + 1), "EALIGN"), ("forward", dict(tokens=0), "OK"), ("forward", dict(out=0), "OK"),
    ("backward", dict(dy=None), "EINVAL"), ("backward", dict(dy=A + 1), "EALIGN"), ("backward", dict(dy_stride=69), "EINVAL"),
    ("backward", dict(dx=A + 1), "EALIGN"), ("backward", dict(dw_stride=99), "EINVAL"), ("backward", dict(db=A + 1), "EALIGN"),
    ("backward", dict(dx=None, dw=None, db=None), "EINVAL"), ("backward", dict(tokens=0, out=0), "OK"),
    # what an unwanted gradient would read is not looked at
    ("backward", dict(dx=None, w8=None, w_scale=None, dy=A + 1), "EALIGN"),
    ("backward", dict(dw=None, x8=A + 1, x8_stride=0, dy=None), "EINVAL")])
def test_linear8_refuses_each_way(way, kw, code):
    call = getattr(train_lib(), "zero_linear8_" + way)
    assert call(ctypes.byref(linear_args(**kw)), None) == getattr(Z, "ZERO_" + code)


def test_linear8_workspace_sizes():
    size = Z.zero_linear8_workspace_bytes
    assert size(-1, 64, 64) == 0 and size(1, 131072, 64) == 0 and size(1, 64, (1 << 20) + 1) == 0
    assert size(0, 0, 0) > 0 and size(1, 1, 1) % 256 == 0
    # few tokens: parts of dx's sums alone
    assert size(1, 4096, 16384) <= 1 << 20 and size(64, 4096, 16384) <= 1 << 24
    # the largest: dy's rows made whole, and beside it not much more than what 256 columns of both operands take
    assert size(1 << 20, 131071, 1 << 20) < 2 * (1 << 40) + (1 << 31)


def test_binding_refuses(monkeypatch):
    # host tensors pass for device ones, and nothing is launched
    monkeypatch.setattr(train, "_on_device", lambda **tensors: None)
    monkeypatch.setattr(train, "_launching", lambda t: None)
    b, i8, f = torch.bfloat16, torch.int8, torch.float32
    x, codes, scale = torch.zeros(4, 40, dtype=b), torch.zeros(4, 48, dtype=i8), torch.zeros(4)
    for bad in ((x[0], codes, scale), (x, codes[:, :40], scale), (x, codes[:3], scale), (x, codes.to(torch.uint8), scale),
                (x, codes, scale[:3]), (x, codes, scale.double()), (x.t(), codes, scale), (x.double(), codes, scale),
                (x, codes, torch.zeros(8)[::2]), (x, torch.zeros(48, 4, dtype=i8).t(), scale), (x, codes, None)):
        with pytest.raises(ValueError):
            Z.zero_rows8_encode(*bad, stream=0)
        with pytest.raises(ValueError):
            Z.zero_rows8_decode(bad[1], bad[2], bad[0], stream=0)
    # rows that the library refuses: expanded, and codes off their alignment
    room = torch.zeros(4 * 48 + 32, dtype=i8)
    off = room[(-room.data_ptr()) % 16 + 1:]
    for bad in ((x[:1].expand(4, 40), codes), (x, codes[:1].expand(4, 48)), (x, off[:192].view(4, 48)),
                (x, torch.zeros(4, 56, dtype=i8)[:, :48])):
        with pytest.raises(Z.ZeroError):
            Z.zero_rows8_encode(bad[0], bad[1], scale, stream=0)
    good = dict(gate=x, up=x, gate8=codes, gate_scale=scale, up8=codes, up_scale=scale, h=x, h8=codes, h_scale=scale,
                dh=x, dgate=x, dup=x)
    Z.Glu8Args(**good).c_args(False)
    Z.Glu8Args(**good).c_args(True)
    Z.Glu8Args(**{**good, "gate": None, "up": None, "h": None, "h8": None, "h_scale": None}).c_args(True)
    for kw in (dict(gate=None), dict(up=x[:, :39]), dict(h=x.half()), dict(kind="relu"), dict(gate_scale=None),
               dict(h8=codes[:, :32]), dict(gate=x[0]), dict(h_scale=scale[:2]), dict(up8=None)):
        with pytest.raises(ValueError):
            Z.Glu8Args(**{**good, **kw}).c_args(False)
    for kw in (dict(dh=None), dict(dgate=None), dict(dup=x[:3]), dict(gate8=None, gate_scale=None), dict(dgate=x.float()),
               dict(up_scale=scale.half())):
        with pytest.raises(ValueError):
            Z.Glu8Args(**{**good, **kw}).c_args(True)
    w8, ws, y = torch.zeros(9, 48, dtype=i8), torch.zeros(9), torch.zeros(4, 9, dtype=b)
    good = dict(x8=codes, x_scale=scale, w8=w8, w_scale=ws, dim=40, workspace=torch.zeros(1 << 16, dtype=torch.uint8),
                bias=torch.zeros(9, dtype=b), y=y, dy=y, dx=x, dw=torch.zeros(9, 40, dtype=b), db=torch.zeros(9, dtype=b))
    Z.Linear8Args(**good).c_args(False)
    Z.Linear8Args(**good).c_args(True)
    for kw in (dict(y=None), dict(y=y[:3]), dict(x8=codes[:, :32]), dict(w8=w8[:8]), dict(bias=torch.zeros(9)),
               dict(bias=torch.zeros(8, dtype=b)), dict(dim=49), dict(x_scale=None), dict(w_scale=ws[:8]),
               dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 16)), dict(y=y.t())):
        with pytest.raises(ValueError):
            Z.Linear8Args(**{**good, **kw}).c_args(False)
    for kw in (dict(dy=None), dict(dx=x[:, :39]), dict(dw=x), dict(db=torch.zeros(9)), dict(dy=y.half()),
               dict(db=torch.zeros(18, dtype=b)[::2])):
        with pytest.raises(ValueError):
            Z.Linear8Args(**{**good, **kw}).c_args(True)
    # what an unwanted gradient would read need not be there
    Z.Linear8Args(**{**good, "dx": None, "w8": None, "w_scale": None}).c_args(True)
    Z.Linear8Args(**{**good, "dw": None, "x8": None, "x_scale": None}).c_args(True)


class Elsewhere:
    """A tensor on another device than the current one."""

    def __init__(self, t):
        self.t, self.is_cuda, self.device = t, True, torch.device("cuda", 1)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_host_tensors_and_other_devices(monkeypatch):
    b, i8 = torch.bfloat16, torch.int8
    x, codes, scale = torch.zeros(4, 40, dtype=b), torch.zeros(4, 48, dtype=i8), torch.zeros(4)
    w8, ws, y = torch.zeros(9, 48, dtype=i8), torch.zeros(9), torch.zeros(4, 9, dtype=b)
    room = torch.zeros(1 << 16, dtype=torch.uint8)

    def calls(x, codes, scale, w8, ws, y, room):
        glu = Z.Glu8Args(gate=x, up=x, gate8=codes, gate_scale=scale, up8=codes, up_scale=scale, h=x, dh=x, dgate=x, dup=x)
        lin = Z.Linear8Args(codes, scale, w8, ws, dim=40, workspace=room, y=y, dy=y, dx=x)
        return [lambda: Z.zero_rows8_encode(x, codes, scale), lambda: Z.zero_rows8_decode(codes, scale, x),
                lambda: Z.zero_glu8_forward(glu), lambda: Z.zero_glu8_backward(glu),
                lambda: Z.zero_linear8_forward(lin), lambda: Z.zero_linear8_backward(lin)]
    for call in calls(x, codes, scale, w8, ws, y, room):
        with pytest.raises(ValueError, match="device memory"):
            call()
    launched = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: launched.append(name) or 0
    monkeypatch.setattr(train, "train_lib", Lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in calls(*(Elsewhere(t) for t in (x, codes, scale, w8, ws, y, room))):
        with pytest.raises(ValueError, match="on cuda:1; the current device is cuda:0"):
            call()
    assert not launched


# -------------------------------------------------- the definitions themselves
def test_held_rows_by_hand():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5], [127.5, 1.0, 3.0, -127.0], [0.0, 0.0, -0.0, 0.0], [1.0, -1.0, 1 / 128, 0.0]])
    q, s = ref.hold(x)
    assert s.tolist() == [1.0, 2.0, 2.0**-126, 2.0**-6]
    assert q[:, :4].tolist() == [[127, 0, 2, -2], [64, 0, 2, -64], [0, 0, 0, 0], [64, -64, 0, 0]]
    assert q.shape == (4, 16) and not q[:, 4:].any()
    q, s = ref.hold(torch.tensor([[65504.0, 2.0**-24], [2.0**-24, 0.0]], dtype=torch.float16))
    assert s.tolist() == [512.0, 2.0**-24] and q[:, :2].tolist() == [[127, 0], [1, 0]]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_held_value_is_one_of_the_type(dtype):
    lo, hi = ref.RANGE[dtype]
    q = torch.arange(-127, 128, dtype=torch.float64)
    for e in {lo, lo + 1, -3, 0, hi - 1, hi}:
        v = q * 2.0**e
        assert torch.equal(v.to(dtype).double(), v) and bool(torch.isfinite(v.to(dtype)).all())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_is_torchs_and_its_slope_the_differences(kind):
    x = torch.linspace(-9, 9, 4001, dtype=torch.float64)
    p, h, d = ref.act(x, kind)
    want = torch.nn.functional.silu(x) if kind == "silu" else torch.nn.functional.gelu(x, approximate="tanh")
    assert float((h - want).abs().max()) < 1e-14
    step = 1e-5
    near = (ref.act(x + step, kind)[1] - ref.act(x - step, kind)[1]) / (2 * step)
    # step^2 / 6 of a third derivative below 3, and 2^-52 of values up to 9 over the step
    assert float((near - d).abs().max()) < 3 * step**2 + 9 * 2.0**-52 / step
