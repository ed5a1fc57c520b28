"""Finite logits far from zero, as rows of a padded vocabulary give that hold
the type's lowest value, or one column far above the rest: the loss and its
gradient are finite and the definition's, in both tiles and with few tokens."""
import pytest
import torch

import train_ref
from test_gpu_xent import Call, say

pytestmark = pytest.mark.gpu

# few tokens; tiles of 128 x 128; tiles of 256 x 256
SIZES = [(5, 64, 900), (40, 64, 900), (3900, 64, 3900)]
SPAN = slice(256, 768)                       # whole waves' columns of either tile


def outputs(c):
    return {"loss": c.args.loss, "lse": c.args.lse, "dx": c.d_dx, "dw": c.d_dw}


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype,value,factor", [
    (torch.bfloat16, -3.1e9, 1.0), (torch.bfloat16, -1e30, 1.0),
    (torch.bfloat16, torch.finfo(torch.bfloat16).min, 1.0),
    (torch.float16, torch.finfo(torch.float16).min, 65504.0)])
def test_masked_columns_of_lowest_values(size, dtype, value, factor):
    say("%s %s %g" % (size, dtype, value))
    c = Call(*size, dtype, seed=1)
    # column 0 is the mask: `factor` in every token, `value` in the masked rows of w, else 0
    c.x[:, 0] = factor
    c.w[:, 0] = 0.0
    c.w[SPAN] = 0.0
    c.w[SPAN, 0] = value
    hidden = torch.zeros(size[2], dtype=torch.bool)
    hidden[SPAN] = True
    c.target[(c.target >= 0) & hidden[c.target.clamp(min=0)]] = 3
    for name in ("x", "w"):
        getattr(c, "d_" + name).copy_(getattr(c, name))
    c.args.target.copy_(c.target)
    c.run()
    x, w, target = c.x.cuda(), c.w.cuda(), c.args.target
    r = train_ref.xent(x, w, target)
    # P is 0 in the masked columns, so neither their logits' nor their w's size is in any error
    r["size"][:, SPAN] = 0.0
    seen = w.clone()
    seen[SPAN] = 0.0
    b = train_ref.xent_bounds(r, x, seen, dtype)
    for name, got in outputs(c).items():
        err = (got.double() - r[name]).abs()
        say("  %-4s worst error %.3g of its bound" % (name, (err / b[name].clamp(min=1e-300)).max().item()))
        assert bool((err <= b[name]).all()), name
    assert not bool(c.d_dw[SPAN].any())
    assert abs(c.result().loss_sum - float(r["sum"])) <= float(b["loss"].sum())


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("value", [2e10, 1e30, 3e38])
def test_one_column_far_above(size, value):
    # its logit is the row's maximum and lse at once, its probability 1, all others' 0
    say("%s %g" % (size, value))
    c = Call(*size, torch.bfloat16, ignored=0.0, seed=2)
    top = 300
    c.x[:, 0] = 1.0
    c.w[:, 0] = 0.0
    c.w[top] = 0.0
    c.w[top, 0] = value
    c.target[0] = top
    for name in ("x", "w"):
        getattr(c, "d_" + name).copy_(getattr(c, name))
    c.args.target.copy_(c.target)
    c.run()
    x, w, target = c.x.cuda().double(), c.w.cuda().double(), c.args.target
    at = w[top, 0]                                     # value as the type has it; the logit is exact
    assert bool((c.args.lse.double() == at).all())
    rows = torch.arange(size[0], device="cuda")
    hit = x @ w.t()
    hit = hit[rows, target]
    # a logit's own fp32 sums (at most 64 of 2^-23 of the magnitudes), then one subtraction
    near = torch.where(target == top, torch.zeros_like(hit), 64 * 2.0**-23 * (x.abs() @ w.abs().t())[rows, target])
    assert bool(((c.args.loss.double() - (at - hit)).abs() <= near + 2.0**-24 * (at - hit).abs()).all())
    # P is exactly 1 at the top and -1 at the target: what is left are fp32 sums and one rounding
    n = 1.0 / size[0]
    p = torch.zeros(size[0], size[2], dtype=torch.float64, device="cuda")
    p[:, top] = 1.0
    p[rows, target] -= 1.0
    u = torch.finfo(torch.bfloat16).eps / 2
    for name, got, a, k in (("dx", c.d_dx, (p, w), size[2]), ("dw", c.d_dw, (p.t().contiguous(), x), size[0])):
        want = n * (a[0] @ a[1])
        sums = n * (a[0].abs() @ a[1].abs()) * (k + 2) * 2.0**-23
        assert bool(((got.double() - want).abs() <= u * want.abs() + sums * (1 + u) + 2.0**-134).all()), name
