"""The training operators together: a bigram language model (an embedding and
a large head) trained in bf16 with fp32 masters and 8-bit AdamW moments.

    python examples/train_bigram.py [--steps 200] [--vocab 32000] [--dim 512] [--tokens 4096]

A step is the loss of the head with its gradient (zero_xent_forward,
zero_xent_backward: the logits are never kept), the embedding's gradient by
torch, and one zero_tensors_step over both tensors, which takes the norm over
the two, clips, updates and casts.  At the end the moments are read back in
fp32 (what a checkpoint holds) and encoded again (what a resume does).
The data is synthetic: token t is followed by one of four tokens that depend
on t, and every tenth target is masked."""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_optimizer_step_amd as Z  # noqa: E402

MASKED = -100


class Bigram:
    def __init__(self, vocab, dim, tokens, lr, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.generator, self.vocab, self.step = g, vocab, 0
        self.master = [torch.randn(vocab, dim, generator=g, device="cuda"),
                       torch.randn(vocab, dim, generator=g, device="cuda").mul_(dim**-0.5)]
        self.param = [m.to(torch.bfloat16) for m in self.master]
        self.grad = [torch.zeros_like(p) for p in self.param]
        k = Z.state8_blocks(vocab * dim)
        self.state8 = [torch.zeros(512 * k, dtype=torch.uint8, device="cuda") for _ in self.master]
        # zero moments: every code 0 under any exponent from 1 on
        self.scale8 = [torch.ones(2 * k, dtype=torch.uint8, device="cuda") for _ in self.master]
        self.set = Z.TensorSet(master=self.master, grad=self.grad, state8=self.state8, scale8=self.scale8,
                               param=self.param, group=[1, 0])
        self.groups = [Z.AdamGroup(lr=lr), Z.AdamGroup(lr=lr, weight_decay=0.0)]
        self.x = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
        self.dx = torch.empty_like(self.x)
        self.target = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.xent = Z.XentArgs(
            x=self.x, w=self.param[1], target=self.target, dx=self.dx, dw=self.grad[1],
            loss=torch.empty(tokens, device="cuda"), lse=torch.empty(tokens, device="cuda"),
            result=torch.zeros(32, dtype=torch.uint8, device="cuda"),
            workspace=torch.empty(Z.zero_xent_workspace_bytes(tokens, dim, vocab), dtype=torch.uint8,
                                  device="cuda"))

    def batch(self):
        n = self.target.numel()
        token = torch.randint(0, self.vocab, (n,), generator=self.generator, device="cuda")
        choice = torch.randint(0, 4, (n,), generator=self.generator, device="cuda")
        target = (token * 7 + choice * 13 + 1) % self.vocab
        target[torch.rand(n, generator=self.generator, device="cuda") < 0.1] = MASKED
        return token, target

    def train_step(self, token, target):
        """Queues one step; the mean loss is a device tensor, read when needed."""
        self.step += 1
        self.target.copy_(target)
        torch.index_select(self.param[0], 0, token, out=self.x)
        Z.zero_xent_forward(self.xent)
        Z.zero_xent_backward(self.xent)
        self.grad[0].zero_().index_add_(0, token, self.dx)
        Z.zero_tensors_step(self.set, self.groups, step=self.step, max_grad_norm=1.0, seed=self.step)
        return self.xent.result.view(torch.float32)[6].clone()

    def moments(self):
        """The moments of each tensor in fp32, as a checkpoint holds them."""
        out = []
        for m, s, e in zip(self.master, self.state8, self.scale8):
            pair = [torch.empty(m.numel(), device="cuda") for _ in range(2)]
            Z.zero_state8_decode(s, e, pair[0], pair[1])
            out.append(pair)
        return out

    def resume(self, moments):
        for (m, v), s, e in zip(moments, self.state8, self.scale8):
            Z.zero_state8_encode(m, v, s, e)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--dim", type=int, default=512)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--lr", type=float, default=3e-3)
    a = p.parse_args(argv)
    model = Bigram(a.vocab, a.dim, a.tokens, a.lr)
    losses = []
    for t in range(a.steps):
        losses.append(model.train_step(*model.batch()))
        if t % 20 == 0 or t == a.steps - 1:
            print("step %4d  loss %.4f  (uniform %.4f, best %.4f)"
                  % (t + 1, losses[-1].item(), math.log(a.vocab), math.log(4)), flush=True)
    held = model.moments()
    model.resume(held)
    same = all(torch.equal(x, y) for p, q in zip(held, model.moments()) for x, y in zip(p, q))
    print("moments read back and encoded again are the same: %s" % same, flush=True)
    return [float(x) for x in losses], same


if __name__ == "__main__":
    main()
