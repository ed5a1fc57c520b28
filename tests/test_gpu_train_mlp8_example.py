"""examples/train_mlp8.py runs, and its gradients are the definition's, stage
by stage on what the stage before left."""
import math
import os
import sys

import pytest
import torch

import rows8_ref as ref
import train_ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_it_runs(kind):
    import train_mlp8
    losses = train_mlp8.main(["--steps", "5", "--vocab", "300", "--dim", "72", "--width", "100", "--tokens", "200",
                              "--kind", kind])
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)


def test_its_gradients_are_the_definitions():
    import train_mlp8
    m = train_mlp8.GatedBigram(300, 72, 100, 130, 1e-2, seed=2)
    token, target = m.batch()
    m.gradients(token, target)
    torch.cuda.synchronize()
    bf16 = torch.bfloat16

    def near(got, want, off, what):
        ref.within(got.double(), want, off + ref.half_step(want, bf16), what)
    r = train_ref.xent(m.z.cpu(), m.param[3].cpu(), target.cpu())
    b = train_ref.xent_bounds(r, m.z.cpu(), m.param[3].cpu(), bf16)
    assert bool(((m.dz.cpu().double() - r["dx"]).abs() <= b["dx"]).all())
    assert bool(((m.grad[3].cpu().double() - r["dw"]).abs() <= b["dw"]).all())
    dz, w = m.dz.double(), [ref.values(*m.w8[0], 72), ref.values(*m.w8[1], 100)]
    near(m.dh, *ref.product(dz, w[1], 72), "dh")
    near(m.grad[2], *ref.product(dz.t(), ref.values(*m.h8, 100), 130), "down")
    dgate, og, dup, ou = ref.glu_grad(m.dh, ref.values(*m.gate8, 100), ref.values(*m.up8, 100), "silu")
    near(m.dboth[:, :100], dgate, og, "dgate")
    near(m.dboth[:, 100:], dup, ou, "dup")
    d = m.dboth.double()
    near(m.grad[1], *ref.product(d.t(), ref.values(*m.x8, 72), 130), "gate and up")
    # dx is rounded, dz added and the sum rounded again
    want, off = ref.product(d, w[0], 200)
    near(m.dx, want + dz, off + ref.half_step(want, bf16) * 1.01, "dx")
    kept, sixteen = m.kept_bytes()
    assert kept < 0.7 * sixteen
