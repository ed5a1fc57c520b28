"""The training operators run together: examples/train_bigram.py learns, and
its first step is the definition's."""
import math
import os
import sys

import pytest
import torch

import train_ref
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_it_learns_and_its_state_survives_a_checkpoint():
    import train_bigram
    # 400 tokens, each seen about 5 times a step: far from uniform (5.99) after 60 steps of Adam
    losses, same = train_bigram.main(["--steps", "60", "--vocab", "400", "--dim", "64", "--tokens", "2048",
                                      "--lr", "0.02"])
    assert same and all(math.isfinite(x) for x in losses)
    assert losses[0] > 5.0 and losses[-1] < 3.0


def test_first_step_is_the_definition():
    import train_bigram
    m = train_bigram.Bigram(300, 64, 100, 1e-2, seed=3)
    token, target = m.batch()
    x = m.param[0][token].cpu()
    w = m.param[1].cpu()
    before = [p.cpu().double() for p in m.master]
    m.train_step(token, target)
    r = train_ref.xent(x, w, target.cpu())
    b = train_ref.xent_bounds(r, x, w, torch.bfloat16)
    assert bool(((m.dx.cpu().double() - r["dx"]).abs() <= b["dx"]).all())
    assert bool(((m.grad[1].cpu().double() - r["dw"]).abs() <= b["dw"]).all())
    # AdamW's first step from zero moments on these gradients: lr against the
    # sign of g where |g'| is far above eps, and the decay of the head's group
    coef = m.set.result.view(torch.float32)[4].item()
    for p0, p1, g, wd in zip(before, m.master, m.grad, (0.0, 0.01)):
        g = g.cpu().double() * coef
        want = p0 * (1 - 1e-2 * wd) - 1e-2 * g / (g.abs() + 1e-8)
        # fp32: about ten roundings of numbers of the size of p and of the step
        assert bool(((p1.cpu().double() - want).abs() <= 2.0**-20 * (p0.abs() + 1e-2)).all())
