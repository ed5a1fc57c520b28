"""Plain definitions of the 8-bit training operators (include/zero/train.h)
for their tests, in torch float64 on the tensors' own device, with the bounds
of the kernels' roundings.  Nothing here uses the library.

Bounds.  A rounding to a type is off by half a step, eps / 2 relative to the
value (or half the least subnormal).  u = 2^-24 is fp32's."""
import math

import torch

RANGE = {torch.float16: (-24, 9), torch.bfloat16: (-126, 121), torch.float32: (-126, 121)}
LEAST = {torch.float16: 2.0**-24, torch.bfloat16: 2.0**-133, torch.float32: 2.0**-149}
U = 2.0**-24


def half_step(value, dtype):
    return value.abs() * (torch.finfo(dtype).eps / 2) + LEAST[dtype] / 2


def stride(dim):
    return -(-dim // 16) * 16


# ------------------------------------------------------------------------ rows
def hold(x):
    """(codes int64 [rows, stride(dim)], scale fp64 [rows]) of rows x of their own type."""
    lo, hi = RANGE[x.dtype]
    rows, dim = x.shape
    bad = ~torch.isfinite(x).all(1)
    v = torch.where(bad.view(-1, 1), torch.zeros_like(x), x).double()
    top = v.abs().amax(1) if dim else torch.zeros(rows, dtype=torch.float64, device=x.device)
    e = torch.frexp(top).exponent.double() - 7            # top = f 2^(e + 7), f in [0.5, 1)
    e = e + (torch.round(top * torch.exp2(-e)) > 127).double()
    e = torch.where(top > 0, e, torch.full_like(e, lo)).clamp(lo, hi)
    scale = torch.exp2(e)
    q = torch.zeros(rows, stride(dim), dtype=torch.int64, device=x.device)
    q[:, :dim] = torch.round(v / scale.view(-1, 1)).clamp(-127, 127).long()
    return q, torch.where(bad, torch.full_like(scale, math.nan), scale)


def values(codes, scale, dim):
    """What codes and scales stand for, fp64."""
    return codes[:, :dim].double() * scale.double().view(-1, 1)


# ------------------------------------------------------------ gated activation
GELU, CUBIC = 2 * math.sqrt(2 / math.pi), 0.044715


def act(x, kind):
    """(p, act, act') of fp64 x."""
    z = x if kind == "silu" else GELU * (x + CUBIC * x**3)
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    slope = torch.ones_like(x) if kind == "silu" else GELU * (1 + 3 * CUBIC * x * x)
    # p and q fall faster than any power of x rises
    far = x.abs() > 1e4
    return p, x * p, p + torch.where(far, torch.zeros_like(x), x * p * q * slope)


def act_bounds(x, kind):
    """(relative error of p, error of act') of the kernel's fp32 arithmetic:
    z has at most 5 roundings, its product with log2 e and the constants 3
    more, so exp(-z) is off by 8 u |z| and an instruction's 2 u, 1 + exp and
    the reciprocal add 4 u.  1 - p is then off by that times p and u.  The
    factor 2 covers what is of second order.  |z| stops where p is 0 or 1."""
    z = x if kind == "silu" else GELU * (x + CUBIC * x**3)
    rel = 2 * U * (8 * z.abs().clamp(max=130) + 6)
    p, _, d = act(x, kind)
    g = torch.ones_like(x) if kind == "silu" else GELU * (1 + 3 * CUBIC * x.clamp(-16, 16)**2)
    xg = x.abs() * g
    return rel, rel * d.abs() + 2 * p * xg * (rel * p + 2 * U) + 12 * U * (p + xg * p * (1 - p))


def glu(gate, up, kind):
    """(h in fp64, its bound before the rounding)."""
    x = gate.double()
    p, h, _ = act(x, kind)
    rel, _ = act_bounds(x, kind)
    w = torch.ones_like(h) if up is None else up.double()
    # a p below fp32's least normal may be 0
    return h * w, (rel + 4 * U) * (h * w).abs() + (x * w).abs() * 2.0**-124


def glu_grad(dh, gate, up, kind):
    """(dgate, bound, dup, bound) in fp64 from the held values; dup None without up."""
    dh, w = dh.double(), torch.ones_like(dh, dtype=torch.float64) if up is None else up
    _, h, d = act(gate, kind)
    rel, off = act_bounds(gate, kind)
    dgate = dh * w * d
    bound = (dh * w).abs() * (off + 2.0**-124 * (1 + gate.abs())) + 4 * U * dgate.abs()
    if up is None:
        return dgate, bound, None, None
    return dgate, bound, dh * h, (rel + 4 * U) * (dh * h).abs() + (dh * gate).abs() * 2.0**-124


# --------------------------------------------------------------------- products
def linear(x8, xs, w8, ws, dim, bias):
    """(y in fp64, its bound before the rounding): the whole sum is exact, then
    fp32 rounds it, its product with one scale and the last multiply-add."""
    s = x8[:, :dim].double() @ w8[:, :dim].double().t()
    y = s * xs.double().view(-1, 1) * ws.double()
    b = 0.0 if bias is None else bias.double()
    return y + b, 3 * U * y.abs() + 2 * U * (y + b).abs()


def product(a, b, k):
    """(a b in fp64, the bound of its fp32 sum): the products of 16-bit values
    are exact in fp32; a chain of k / 32 sums of 32, each sum a tree of 5, up
    to 64 slices joined, every rounding at most 2 u of the magnitudes' sum (the
    matrix cores may cut off instead of rounding)."""
    return a @ b, (k / 32 + 5 + 64) * 2 * U * (a.abs() @ b.abs())


def column_sum(dy, rows):
    """(sums, bound): a thread adds at most rows / 8 values, 8 threads and 1024
    shares at most are joined; shares of fewer than 64 rows are not made."""
    dy = dy.double()
    return dy.sum(0), (rows / 8 + 8 + min(1024, rows / 64 + 1)) * U * dy.abs().sum(0)


def within(got, want, bound, what="", dtype=None):
    """Every element of got (fp64 of an output) within its bound of want, and
    NaN exactly where want is.  With a dtype, what it rounds to infinity
    (half a step past its largest number) may be infinite, of want's sign."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), "%s: NaN in other places" % what
    same = got == want
    if dtype is not None:
        info = torch.finfo(dtype)
        past = want.abs() + bound >= info.max * (1 + info.eps / 4)
        same |= past & torch.isinf(got) & (torch.sign(got) == torch.sign(want))
    off = torch.where(nan | same, torch.zeros_like(want), (got - want).abs())
    bad = ~nan & ~(off <= bound)
    assert not bool(bad.any()), "%s: %d of %d elements outside, first %s: %s, expected %s within %s" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(),
        bound[bad][0].item())
