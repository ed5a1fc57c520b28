"""The gated activation where its p is below fp32's least normal number: there
x p is still a normal bf16 for a while, and has to be what the definition says.

Bounds: those of rows8_ref with its allowance for a p that becomes 0 (2^-124)
replaced by what fp32 itself can hold.  p is off by half of fp32's least step
where it is held, or by itself where it is not: 2^-150 each way.  The products
that follow are rounded to fp32, half of its least step (2^-150) or u, and the
next factor multiplies that: (p, x p), then up; (p, slope), then dh, then up."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_glu8 import Call
from test_gpu_rows8 import say

pytestmark = pytest.mark.gpu
LEAST = 2.0**-149                              # twice the half step of fp32's least numbers

# silu's p is 2^-126 at -87.3 and 2^-150 at -104; gelu's at -9.86 and -10.5
GATES = {"silu": torch.linspace(-106, -80, 209), "gelu": torch.linspace(-10.75, -9.5, 201)}


def call(kind, dtype, gated, up):
    """A row of one gate each, so that the held gate is near it too."""
    v = GATES[kind].to(dtype)
    c = Call(len(v), 24, dtype, kind, gated, sigma=1.0)
    c.gate.copy_(v.view(-1, 1).expand(-1, 24))
    if gated:
        c.up.copy_(torch.linspace(up / 2, up, 24).to(dtype).expand(len(v), 24))
        c.dh.copy_(torch.ones(24, dtype=dtype).expand(len(v), 24))
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("gated,up", [(False, 1.0), (True, 1.0), (True, 30000.0)], ids=["plain", "gated", "gated far"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_below_the_least_normal_p(kind, gated, up, dtype):
    say("glu8 low end %s %s %s %s" % (kind, gated, up, dtype))
    c = call(kind, dtype, gated, up)
    Z.zero_glu8_forward(c.args)
    Z.zero_glu8_backward(c.args)

    x = c.gate.double()
    w = torch.ones_like(x) if c.up is None else c.up.double()
    p, h, _ = ref.act(x, kind)
    rel, _ = ref.act_bounds(x, kind)
    off = (rel + 4 * ref.U) * (h * w).abs() + (x.abs() + 1) * w.abs() * LEAST + LEAST
    want = h * w
    ref.within(c.h.double(), want, off + ref.half_step(want, dtype), "h", dtype)

    x = ref.values(c.gate8, c.gate_scale, c.w)
    w = torch.ones_like(x) if c.up is None else ref.values(c.up8, c.up_scale, c.w)
    dh = c.dh.double()
    _, h, d = ref.act(x, kind)
    rel, off = ref.act_bounds(x, kind)
    # p's error through the slope's factors: 1 + |x| of silu, 1 + |x| g of gelu with g below 27 here
    factor = 1 + 27 * x.abs()
    want = dh * w * d
    off = (dh * w).abs() * (off + factor * LEAST) + 4 * ref.U * want.abs() + (w.abs() + 1) * LEAST
    ref.within(c.dgate.double(), want, off + ref.half_step(want, dtype), "dgate", dtype)
    if gated:
        want = dh * h
        off = (rel + 4 * ref.U) * want.abs() + (x.abs() + 1) * dh.abs() * LEAST + LEAST
        ref.within(c.dup.double(), want, off + ref.half_step(want, dtype), "dup", dtype)
    if dtype == torch.bfloat16:
        # the cases are there: normal numbers of the type from a p below fp32's least normal
        low = (p < 2.0**-126) & ((p * c.gate.double()).abs() > 2.0**-126)
        assert int(low.sum()) >= 24 * 8 and bool((c.h[low] != 0).all())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("width", [24, 3000, 17000, 40000])
def test_beside_a_nan_and_in_rows_read_twice(kind, width):
    """One such gate in a row of ordinary ones, also where the row holds a NaN;
    the others are what they are without it."""
    say("glu8 low end beside %s %d" % (kind, width))
    c = Call(4, width, torch.bfloat16, kind, True, sigma=1.0)
    Z.zero_glu8_forward(c.args)
    plain = c.h.clone()
    at = width // 2
    c.gate[1, at] = c.gate[2, at] = {"silu": -88.0, "gelu": -10.0625}[kind]
    c.gate[2, at + 1] = float("nan")
    c.up[:, at] = 1.0
    Z.zero_glu8_forward(c.args)
    p, h, _ = ref.act(c.gate[1, at].double(), kind)
    rel, _ = ref.act_bounds(c.gate[1, at].double(), kind)
    off = (rel + 4 * ref.U) * h.abs() + (GATES[kind].abs().max().item() + 2) * LEAST
    assert float(p) < 2.0**-126 < float(h.abs())
    for row in (1, 2):
        assert abs(float(c.h[row, at]) - float(h)) <= float(off + ref.half_step(h, torch.bfloat16))
    assert bool(torch.isnan(c.h[2, at + 1]))
    rest = torch.ones(width, dtype=torch.bool, device="cuda")
    rest[at:at + 2] = False
    assert torch.equal(c.h[:, rest], plain[:, rest])
    c.same_codes(c.h8[:2], c.h_scale[:2], c.h[:2], "h8")
    assert bool(torch.isnan(c.h_scale[2]))


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_a_scale_may_be_negative(kind, gated):
    """Codes and scales of the other sign stand for the same gates."""
    say("glu8 low end, negative scales %s %s" % (kind, gated))
    c = call(kind, torch.bfloat16, gated, 1.0)
    Z.zero_glu8_forward(c.args)
    Z.zero_glu8_backward(c.args)
    want = [m.clone() for m in (c.dgate, c.dup) if m is not None]
    assert int((want[0] != 0).sum()) > 24 * 100
    c.gate8.neg_()
    c.gate_scale.neg_()
    Z.zero_glu8_backward(c.args)
    for got, w in zip((c.dgate, c.dup), want):
        assert torch.equal(got, w)
