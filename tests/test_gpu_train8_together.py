"""The 8-bit operators as a training step uses them: a gated layer's rows
held, its products, activation, gradients and one step of its weights, against
the same in fp64 from the same held values."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_rows8 import say

pytestmark = pytest.mark.gpu


class Layer:
    """y = W2 (silu(Wg x) * Wu x), its weights in fp32 masters and 16-bit
    parameters held in 8 bits, of any sizes."""

    def __init__(self, tokens, dim, width, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.t, self.d, self.f, self.dtype = tokens, dim, width, dtype
        cuda = dict(device="cuda")

        def rows(r, k):
            return torch.empty(r, Z.rows8_stride(k), dtype=torch.int8, **cuda), torch.empty(r, **cuda)
        self.master = [(torch.randn(2 * width, dim, generator=g) / dim**0.5).cuda(),
                       (torch.randn(dim, width, generator=g) / width**0.5).cuda()]
        self.param = [m.to(dtype) for m in self.master]
        self.grad = [torch.empty_like(p) for p in self.param]
        self.w8 = [rows(2 * width, dim), rows(dim, width)]
        self.x = torch.randn(tokens, dim, generator=g).to(dtype).cuda()
        self.dy = torch.randn(tokens, dim, generator=g).to(dtype).cuda()
        self.x8, self.h8 = rows(tokens, dim), rows(tokens, width)
        self.gate8, self.up8 = rows(tokens, width), rows(tokens, width)
        self.both, self.dboth = (torch.empty(tokens, 2 * width, dtype=dtype, **cuda) for _ in range(2))
        self.y, self.dx = (torch.empty(tokens, dim, dtype=dtype, **cuda) for _ in range(2))
        self.dh = torch.empty(tokens, width, dtype=dtype, **cuda)
        need = max(Z.zero_linear8_workspace_bytes(tokens, dim, 2 * width), Z.zero_linear8_workspace_bytes(tokens, width, dim))
        room = torch.empty(need, dtype=torch.uint8, **cuda)
        self.first = Z.Linear8Args(*self.x8, *self.w8[0], dim=dim, workspace=room, y=self.both, dy=self.dboth,
                                   dx=self.dx, dw=self.grad[0])
        self.second = Z.Linear8Args(*self.h8, *self.w8[1], dim=width, workspace=room, y=self.y, dy=self.dy,
                                    dx=self.dh, dw=self.grad[1])
        self.glu = Z.Glu8Args(kind="silu", gate=self.both[:, :width], up=self.both[:, width:], gate8=self.gate8[0],
                              gate_scale=self.gate8[1], up8=self.up8[0], up_scale=self.up8[1], h8=self.h8[0],
                              h_scale=self.h8[1], dh=self.dh, dgate=self.dboth[:, :width], dup=self.dboth[:, width:])
        self.moments = [[torch.zeros_like(m) for m in self.master] for _ in range(2)]
        self.set = Z.TensorSet(master=self.master, grad=self.grad, exp_avg=self.moments[0], exp_avg_sq=self.moments[1],
                               param=self.param)
        self.groups = [Z.AdamGroup(lr=1e-3)]

    def step(self, t):
        for p, (q, s) in zip(self.param, self.w8):
            Z.zero_rows8_encode(p, q, s)
        Z.zero_rows8_encode(self.x, *self.x8)
        Z.zero_linear8_forward(self.first)
        Z.zero_glu8_forward(self.glu)
        Z.zero_linear8_forward(self.second)
        Z.zero_linear8_backward(self.second)
        Z.zero_glu8_backward(self.glu)
        Z.zero_linear8_backward(self.first)
        Z.zero_tensors_step(self.set, self.groups, step=t, max_grad_norm=1.0)

    def check(self, params):
        """Every stage against the definition on that stage's own inputs."""
        def same(held, x, what):
            q, s = ref.hold(x)
            assert torch.equal(held[0].long(), q) and torch.equal(held[1].double(), s), what

        def near(got, want, off, what):
            ref.within(got.double(), want, off + ref.half_step(want, self.dtype), what)
        for held, p in zip(self.w8, params):
            same(held, p, "w8")
        same(self.x8, self.x, "x8")
        near(self.both, *ref.linear(*self.x8, *self.w8[0], self.d, None), "gate and up")
        same(self.gate8, self.both[:, :self.f], "gate8")
        same(self.up8, self.both[:, self.f:], "up8")
        h, off = ref.glu(self.both[:, :self.f], self.both[:, self.f:], "silu")
        off = off + ref.half_step(h, self.dtype) + self.h8[1].double().view(-1, 1) / 2
        ref.within(ref.values(*self.h8, self.f), h, off, "h8")
        near(self.y, *ref.linear(*self.h8, *self.w8[1], self.f, None), "y")
        value = [ref.values(q, s, k) for (q, s), k in zip(self.w8, (self.d, self.f))]
        dy = self.dy.double()
        near(self.dh, *ref.product(dy, value[1], self.d), "dh")
        near(self.grad[1], *ref.product(dy.t(), ref.values(*self.h8, self.f), self.t), "dw2")
        gate, up = ref.values(*self.gate8, self.f), ref.values(*self.up8, self.f)
        dgate, og, dup, ou = ref.glu_grad(self.dh, gate, up, "silu")
        near(self.dboth[:, :self.f], dgate, og, "dgate")
        near(self.dboth[:, self.f:], dup, ou, "dup")
        d = self.dboth.double()
        near(self.dx, *ref.product(d, value[0], 2 * self.f), "dx")
        near(self.grad[0], *ref.product(d.t(), ref.values(*self.x8, self.d), self.t), "dw1")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", [(1, 64, 48), (50, 100, 300), (333, 512, 1001)], ids=str)
def test_training_step(size, dtype):
    say("together %s %s" % (size, dtype))
    m = Layer(*size, dtype)
    for t in (1, 2):
        params = [p.clone() for p in m.param]
        before = [w.clone() for w in m.master]
        m.step(t)
        m.check(params)
        assert all(not torch.equal(a, b) for a, b in zip(before, m.master))


def test_training_step_captured():
    """One graph of the whole step but the update, replayed on other inputs."""
    say("together captured")
    m = Layer(100, 144, 272, torch.bfloat16)
    m.step(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(2)
    for _ in range(3):
        m.x.normal_()
        m.dy.normal_()
        params = [p.clone() for p in m.param]
        graph.replay()
        torch.cuda.synchronize()
        m.check(params)


def test_an_overflow_skips_the_step():
    """A token that is not finite reaches the gradients and the step's flag."""
    say("together overflow")
    m = Layer(60, 96, 112, torch.float16)
    m.step(1)
    before = [w.clone() for w in m.master]
    m.x[17, 5] = float("inf")
    m.step(2)
    assert m.set.result.view(torch.int32)[5].item() != 0
    assert all(torch.equal(a, b) for a, b in zip(before, m.master))
