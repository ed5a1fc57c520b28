"""The gated activation with its 8-bit checkpoint against its definition in
fp64, with the bounds of rows8_ref."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_rows8 import place, say, untouched

pytestmark = pytest.mark.gpu


class Call:
    """A call's buffers, gate and up the halves of one matrix."""

    def __init__(self, tokens, width, dtype, kind, gated, pad=0, shift=0, held=True, out16=True, out8=True, seed=0,
                 sigma=2.0):
        g = torch.Generator().manual_seed(seed)
        self.t, self.w, self.kind, self.dtype = tokens, width, kind, dtype
        self.rooms = []
        parts = 2 if gated else 1

        def both(src):
            room, m = place(tokens, parts * width, dtype, pad, shift, src)
            self.rooms.append((room, m))
            return m[:, :width], m[:, width:] if gated else None

        def held8(wanted):
            if not wanted:
                return None, None
            room, codes = place(tokens, ref.stride(width), torch.int8, 16 if pad else 0)
            scales, s = place(1, tokens, torch.float32)
            self.rooms += [(room, codes), (scales, s)]
            return codes, s[0]
        self.gate, self.up = both((torch.randn(tokens, parts * width, generator=g) * sigma).to(dtype))
        _, self.dh = place(tokens, width, dtype, pad, shift, torch.randn(tokens, width, generator=g).to(dtype))
        self.gate8, self.gate_scale = held8(held)
        self.up8, self.up_scale = held8(held and gated)
        self.h8, self.h_scale = held8(out8)
        self.h = None
        if out16:
            room, self.h = place(tokens, width, dtype, pad, shift)
            self.rooms.append((room, self.h))
        self.dgate, self.dup = both(None)
        self.args = Z.Glu8Args(kind=kind, gate=self.gate, up=self.up, gate8=self.gate8, gate_scale=self.gate_scale,
                               up8=self.up8, up_scale=self.up_scale, h=self.h, h8=self.h8, h_scale=self.h_scale,
                               dh=self.dh, dgate=self.dgate, dup=self.dup)

    def same_codes(self, codes, scale, x, what):
        q, s = ref.hold(x)
        assert torch.equal(scale.double().nan_to_num(-1.0), s.nan_to_num(-1.0)), what
        assert torch.equal(codes.long(), q), what

    def check_forward(self):
        want, bound = ref.glu(self.gate, self.up, self.kind)
        if self.h is not None:
            ref.within(self.h.double(), want, bound + ref.half_step(want, self.dtype), "h", self.dtype)
            if self.h8 is not None:
                self.same_codes(self.h8, self.h_scale, self.h, "h8")
        elif self.h8 is not None:
            # h's rounding, and half of a code's step
            off = bound + ref.half_step(want, self.dtype) + self.h_scale.double().view(-1, 1) / 2
            ref.within(ref.values(self.h8, self.h_scale, self.w), want, off, "h8")
        if self.gate8 is not None:
            self.same_codes(self.gate8, self.gate_scale, self.gate, "gate8")
            if self.up is not None:
                self.same_codes(self.up8, self.up_scale, self.up, "up8")

    def check_backward(self, dh=None):
        dh = self.dh if dh is None else dh
        gate = ref.values(self.gate8, self.gate_scale, self.w)
        up = None if self.up is None else ref.values(self.up8, self.up_scale, self.w)
        dgate, bg, dup, bu = ref.glu_grad(dh, gate, up, self.kind)
        ref.within(self.dgate.double(), dgate, bg + ref.half_step(dgate, self.dtype), "dgate", self.dtype)
        if up is not None:
            ref.within(self.dup.double(), dup, bu + ref.half_step(dup, self.dtype), "dup", self.dtype)

    def check(self):
        Z.zero_glu8_forward(self.args)
        self.check_forward()
        Z.zero_glu8_backward(self.args)
        self.check_backward()
        assert all(untouched(*r) for r in self.rooms)


SIZES = [(1, 1), (37, 7), (5, 64), (130, 128), (9, 129), (6, 512), (5, 513), (9, 2048), (3, 2049), (4, 4097), (2, 8200),
         (3, 16384), (2, 16400), (1, 131071)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_sizes(gated, kind, dtype):
    for size in SIZES:
        say("glu8 %s %s %s %s" % (size, kind, gated, dtype))
        Call(*size, dtype, kind, gated).check()


@pytest.mark.parametrize("pad,shift", [(1, 0), (6, 3), (8, 8)])
def test_strides_and_alignment(pad, shift):
    for gated in (True, False):
        say("glu8 strides %s %s" % ((pad, shift), gated))
        Call(11, 301, torch.float16, "gelu", gated, pad, shift).check()
        Call(3, 5003, torch.bfloat16, "silu", gated, pad, shift).check()


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_only_what_is_wanted(gated):
    """h alone (no checkpoint), h8 alone, and each with the checkpoint."""
    for held, out16, out8 in ((False, True, False), (False, False, True), (True, True, False), (True, False, True)):
        for size in ((20, 100), (3, 3000), (2, 17000)):
            say("glu8 %s %s %s %s" % (size, held, out16, out8))
            c = Call(*size, torch.bfloat16, "silu", gated, held=held, out16=out16, out8=out8)
            Z.zero_glu8_forward(c.args)
            c.check_forward()
            assert all(untouched(*r) for r in c.rooms)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_in_place_of_dh(kind):
    for size in ((7, 90), (5, 5001)):
        for which in ("dgate", "dup"):
            say("glu8 in place %s %s %s" % (size, kind, which))
            c = Call(*size, torch.bfloat16, kind, True, pad=4)
            Z.zero_glu8_forward(c.args)
            dh = c.dh.clone()
            setattr(c, which, c.dh)
            setattr(c.args, which, c.dh)
            Z.zero_glu8_backward(c.args)
            c.check_backward(dh)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_large_and_small_values(kind, dtype):
    """The activation's two ends, values whose powers overflow fp32, zeros of
    both signs and the least numbers: finite wherever the definition's rounding is."""
    say("glu8 values %s %s" % (kind, dtype))
    top = torch.finfo(dtype).max
    # what a row holds shares one scale, so every magnitude has a row of its own
    tops = [0.0, 1e-7, 1e-3, 0.5, 3.0, 10.0, 20.0, 60.0, 88.0, 100.0, 300.0, 5000.0, 60000.0]
    tops += [1e10, 1e13, 1e20, 1e30, top / 2] if dtype == torch.bfloat16 else []
    ramp = torch.linspace(-1, 1, 203, dtype=torch.float64)
    c = Call(len(tops), 203, dtype, kind, True, sigma=1.0)
    c.gate.copy_(torch.stack([ramp * t for t in tops]).to(dtype))
    c.check()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_tokens_that_are_not_finite(kind):
    """A NaN or an infinity stays in its token, in whatever reads the row that holds it."""
    for width in (50, 3001, 16500):
        say("glu8 not finite %s %d" % (kind, width))
        c = Call(9, width, torch.float16, kind, True)
        c.gate[1, 5], c.gate[2, width - 1], c.gate[7, 0] = float("nan"), float("inf"), float("-inf")
        c.up[4, 3], c.up[5, width // 2] = float("inf"), float("nan")
        c.gate[6, 2], c.up[6, 2] = 60000.0, 60000.0        # h overflows: +inf in fp16
        Z.zero_glu8_forward(c.args)
        Z.zero_glu8_backward(c.args)
        c.same_codes(c.gate8, c.gate_scale, c.gate, "gate8")
        c.same_codes(c.up8, c.up_scale, c.up, "up8")
        c.same_codes(c.h8, c.h_scale, c.h, "h8")
        assert bool(torch.isinf(c.h[6, 2])) and bool(torch.isnan(c.h_scale[6]))
        fine = torch.tensor([0, 3, 6, 8], device="cuda")
        assert bool(torch.isfinite(c.h_scale[fine[[0, 1, 3]]]).all())
        for row, dgate, dup in ((1, True, True), (2, True, True), (7, True, True), (4, True, False), (5, True, False),
                                (0, False, False), (3, False, False), (6, False, False), (8, False, False)):
            assert bool(torch.isnan(c.dgate[row]).all()) == dgate, row
            assert bool(torch.isnan(c.dup[row]).all()) == dup, row
        c.check_backward()


def test_formula_against_differences():
    """The kernel's gradient, and the definition's, against differences of the definition."""
    for kind in ("silu", "gelu"):
        say("glu8 differences %s" % kind)
        c = Call(40, 300, torch.float16, kind, True)
        Z.zero_glu8_forward(c.args)
        Z.zero_glu8_backward(c.args)
        gate, up = (ref.values(q, s, 300) for q, s in ((c.gate8, c.gate_scale), (c.up8, c.up_scale)))
        step = 1e-5
        slope = (ref.act(gate + step, kind)[1] - ref.act(gate - step, kind)[1]) / (2 * step)
        # differences: step^2 / 6 of the third derivative (below 3), and 2^-52 of values up to 20 over the step
        near = 3 * step**2 + 20 * 2.0**-52 / step
        want = c.dh.double() * up * slope
        formula, bound, _, _ = ref.glu_grad(c.dh, gate, up, kind)
        far = (c.dh.double() * up).abs() * near
        ref.within(formula, want, far, "formula")
        ref.within(c.dgate.double(), want, far + bound + ref.half_step(formula, torch.float16), "kernel")


def test_no_tokens():
    for t, w in ((0, 40), (0, 0), (3, 0)):
        c = Call(t, w, torch.bfloat16, "silu", True)
        Z.zero_glu8_forward(c.args)
        Z.zero_glu8_backward(c.args)
        torch.cuda.synchronize()
        assert all(untouched(*r) for r in c.rooms if r[1].dtype != torch.float32)


def test_offsets_past_32_bits():
    tokens, width = 17000, 131064
    say("glu8 %d x %d" % (tokens, width))
    g = torch.Generator(device="cuda").manual_seed(0)
    gate, up, h, dh = (torch.zeros(tokens, width, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    codes = [torch.empty(tokens, ref.stride(width), dtype=torch.int8, device="cuda") for _ in range(3)]
    scales = [torch.empty(tokens, device="cuda") for _ in range(3)]
    at = [0, 8191, 16383, 16384, 16385, 16386, tokens - 1]
    for r in at:
        for m in (gate, up, dh):
            m[r].copy_(torch.randn(width, generator=g, device="cuda"))
    a = Z.Glu8Args(kind="silu", gate=gate, up=up, gate8=codes[0], gate_scale=scales[0], up8=codes[1],
                   up_scale=scales[1], h=h, h8=codes[2], h_scale=scales[2], dh=dh)
    Z.zero_glu8_forward(a)
    want, bound = ref.glu(gate[at], up[at], "silu")
    ref.within(h[at].double(), want, bound + ref.half_step(want, torch.bfloat16), "h")
    for q, s, x in ((codes[0], scales[0], gate), (codes[1], scales[1], up), (codes[2], scales[2], h)):
        cq, cs = ref.hold(x[at])
        assert torch.equal(q[at].long(), cq) and torch.equal(s[at].double(), cs)
        assert int(q.view(torch.int32).ne(0).any(1).sum()) == len(at)
    # the gradients take the inputs' memory
    a.dgate, a.dup = gate, up
    Z.zero_glu8_backward(a)
    held = [ref.values(codes[i][at], scales[i][at], width) for i in range(2)]
    dgate, bg, dup, bu = ref.glu_grad(dh[at], *held, "silu")
    ref.within(gate[at].double(), dgate, bg + ref.half_step(dgate, torch.bfloat16), "dgate")
    ref.within(up[at].double(), dup, bu + ref.half_step(dup, torch.bfloat16), "dup")
    assert int(gate.any(1).sum()) == len(at) and int(up.any(1).sum()) == len(at)


def test_captured_and_on_a_side_stream():
    say("glu8 captured")
    c = Call(33, 1001, torch.bfloat16, "silu", True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Z.zero_glu8_forward(c.args)
        Z.zero_glu8_backward(c.args)
    side.synchronize()
    c.check_forward()
    c.check_backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_glu8_forward(c.args)
        Z.zero_glu8_backward(c.args)
    for i in range(4):
        c.gate.normal_(std=1.0 + i)
        c.up.normal_()
        c.dh.normal_()
        graph.replay()
        torch.cuda.synchronize()
        c.check_forward()
        c.check_backward()
