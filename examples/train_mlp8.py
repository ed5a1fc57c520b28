"""A gated layer trained on 8-bit rows: a bigram language model of an
embedding, one gated feed-forward layer and a large head, in bf16 with fp32
masters and 8-bit AdamW moments.

    python examples/train_mlp8.py [--steps 200] [--vocab 32000] [--dim 512] [--width 2048] [--tokens 4096]

The layer's products take 8-bit rows and 8-bit weights (zero_linear8_forward);
what the backward needs of its activations stays in 8 bits: its input, gate
and up, and the activation's result, one byte an element and a scale a token
(printed, beside the 16-bit bytes).  A step holds the parameters in 8 bits
again after each update, and ends with one zero_tensors_step over all tensors.
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


def rows8(rows, dim):
    """Room for rows of codes and their scales."""
    return (torch.empty(rows, Z.rows8_stride(dim), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda"))


class GatedBigram:
    """x = embedding; z = x + W2 (silu(Wg x) * Wu x); logits = head z."""

    def __init__(self, vocab, dim, width, tokens, lr, kind="silu", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.generator, self.vocab, self.width, self.step = g, vocab, width, 0

        def normal(rows, cols, sigma):
            return torch.randn(rows, cols, generator=g, device="cuda").mul_(sigma)

        def sixteen(rows, cols):
            return torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        # embedding, gate and up, down, head
        self.master = [normal(vocab, dim, 1.0), normal(2 * width, dim, dim**-0.5), normal(dim, width, width**-0.5),
                       normal(vocab, dim, dim**-0.5)]
        self.param = [m.to(torch.bfloat16) for m in self.master]
        self.grad = [torch.zeros_like(p) for p in self.param]
        blocks = [Z.state8_blocks(m.numel()) for m in self.master]
        self.state8 = [torch.zeros(512 * k, dtype=torch.uint8, device="cuda") for k in blocks]
        self.scale8 = [torch.ones(2 * k, dtype=torch.uint8, device="cuda") for k in blocks]
        self.set = Z.TensorSet(master=self.master, grad=self.grad, state8=self.state8, scale8=self.scale8,
                               param=self.param, group=[1, 0, 0, 0])
        self.groups = [Z.AdamGroup(lr=lr), Z.AdamGroup(lr=lr, weight_decay=0.0)]
        # the layer: weights and what the backward keeps, in 8 bits
        self.w8 = [rows8(2 * width, dim), rows8(dim, width)]
        self.x8, self.gate8, self.up8, self.h8 = rows8(tokens, dim), rows8(tokens, width), rows8(tokens, width), rows8(tokens, width)
        self.x, self.y, self.z, self.dz, self.dx = (sixteen(tokens, dim) for _ in range(5))
        both, self.dboth, self.dh = sixteen(tokens, 2 * width), sixteen(tokens, 2 * width), sixteen(tokens, width)
        room = torch.empty(max(Z.zero_linear8_workspace_bytes(tokens, dim, 2 * width),
                               Z.zero_linear8_workspace_bytes(tokens, width, dim)), dtype=torch.uint8, device="cuda")
        self.first = Z.Linear8Args(*self.x8, *self.w8[0], dim=dim, workspace=room, y=both, dy=self.dboth, dx=self.dx,
                                   dw=self.grad[1])
        self.second = Z.Linear8Args(*self.h8, *self.w8[1], dim=width, workspace=room, y=self.y, dy=self.dz, dx=self.dh,
                                    dw=self.grad[2])
        self.glu = Z.Glu8Args(kind=kind, gate=both[:, :width], up=both[:, width:], gate8=self.gate8[0],
                              gate_scale=self.gate8[1], up8=self.up8[0], up_scale=self.up8[1], h8=self.h8[0],
                              h_scale=self.h8[1], dh=self.dh, dgate=self.dboth[:, :width], dup=self.dboth[:, width:])
        self.target = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.xent = Z.XentArgs(
            x=self.z, w=self.param[3], target=self.target, dx=self.dz, dw=self.grad[3],
            loss=torch.empty(tokens, device="cuda"), lse=torch.empty(tokens, device="cuda"),
            result=torch.zeros(32, dtype=torch.uint8, device="cuda"),
            workspace=torch.empty(Z.zero_xent_workspace_bytes(tokens, dim, vocab), dtype=torch.uint8, device="cuda"))

    def kept_bytes(self):
        """(bytes the backward keeps of the layer's activations, the same in 16 bits)."""
        held = [self.x8, self.gate8, self.up8, self.h8]
        return (sum(q.numel() + 4 * s.numel() for q, s in held),
                2 * (self.x.numel() + 3 * self.dh.numel()))

    def batch(self):
        n = self.target.numel()
        token = torch.randint(0, self.vocab, (n,), generator=self.generator, device="cuda")
        choice = torch.randint(0, 4, (n,), generator=self.generator, device="cuda")
        target = (token * 7 + choice * 13 + 1) % self.vocab
        target[torch.rand(n, generator=self.generator, device="cuda") < 0.1] = MASKED
        return token, target

    def gradients(self, token, target):
        """Queues the forward and the backward."""
        self.target.copy_(target)
        for p, held in zip(self.param[1:3], self.w8):
            Z.zero_rows8_encode(p, *held)
        torch.index_select(self.param[0], 0, token, out=self.x)
        Z.zero_rows8_encode(self.x, *self.x8)
        Z.zero_linear8_forward(self.first)
        Z.zero_glu8_forward(self.glu)
        Z.zero_linear8_forward(self.second)
        torch.add(self.x, self.y, out=self.z)
        Z.zero_xent_forward(self.xent)
        Z.zero_xent_backward(self.xent)
        Z.zero_linear8_backward(self.second)
        Z.zero_glu8_backward(self.glu)
        Z.zero_linear8_backward(self.first)
        self.dx += self.dz
        self.grad[0].zero_().index_add_(0, token, self.dx)

    def train_step(self, token, target):
        """Queues one step; the mean loss is a device tensor, read when needed."""
        self.step += 1
        self.gradients(token, target)
        Z.zero_tensors_step(self.set, self.groups, step=self.step, max_grad_norm=1.0, seed=self.step)
        return self.xent.result.view(torch.float32)[6].clone()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--dim", type=int, default=512)
    p.add_argument("--width", type=int, default=2048)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--kind", choices=("silu", "gelu"), default="silu")
    p.add_argument("--lr", type=float, default=3e-3)
    a = p.parse_args(argv)
    model = GatedBigram(a.vocab, a.dim, a.width, a.tokens, a.lr, a.kind)
    print("the layer keeps %d bytes of activations for its backward, %d in 16 bits" % model.kept_bytes(), flush=True)
    losses = []
    for t in range(a.steps):
        losses.append(model.train_step(*model.batch()))
        if t % 20 == 0 or t == a.steps - 1:
            print("step %4d  loss %.4f  (uniform %.4f, best %.4f)"
                  % (t + 1, losses[-1].item(), math.log(a.vocab), math.log(4)), flush=True)
    return [float(x) for x in losses]


if __name__ == "__main__":
    main()
