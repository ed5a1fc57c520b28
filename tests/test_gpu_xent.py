"""The cross entropy of a large vocabulary against its definition in fp64, at
sizes where tiles, pieces and slices end oddly, with the bounds of
train_ref.xent_bounds."""
import pytest
import torch

import train_ref
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu


def say(msg):
    print(msg, flush=True)


class Call:
    """A call's buffers; `pad` extra elements between rows, `shift` elements
    off the allocation's start."""

    def __init__(self, tokens, dim, vocab, dtype, ignored=0.2, seed=0, pad=0, shift=0, grad_scale=1.0,
                 spread=3.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        self.x = torch.randn(tokens, dim, generator=g).to(dtype)
        self.w = (torch.randn(vocab, dim, generator=g) * spread / max(1, dim) ** 0.5).to(dtype)
        self.target = torch.randint(0, vocab, (tokens,), generator=g)
        if ignored:
            self.target[torch.rand(tokens, generator=g) < ignored] = -100

        def place(rows, cols, src=None):
            room = torch.full((rows * (cols + pad) + shift + 8,), -7.0, dtype=dtype, device="cuda")
            view = room[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
            if src is not None:
                view.copy_(src)
            return room, view
        self.rooms = {}
        for name, shape, src in (("x", (tokens, dim), self.x), ("w", (vocab, dim), self.w),
                                 ("dx", (tokens, dim), None), ("dw", (vocab, dim), None)):
            self.rooms[name], view = place(*shape, src)
            setattr(self, "d_" + name, view)
        bytes_ = Z.zero_xent_workspace_bytes(tokens, dim, vocab)
        self.ws = torch.full((bytes_ // 4 + 64,), float("nan"), device="cuda").view(torch.uint8)
        self.args = Z.XentArgs(x=self.d_x, w=self.d_w, target=self.target.cuda(),
                               loss=torch.full((tokens,), -1.0, device="cuda"),
                               lse=torch.full((tokens,), -1.0, device="cuda"),
                               result=torch.zeros(32, dtype=torch.uint8, device="cuda"),
                               workspace=self.ws[:bytes_], dx=self.d_dx, dw=self.d_dw, grad_scale=grad_scale)

    def run(self, backward=True):
        Z.zero_xent_forward(self.args)
        if backward:
            Z.zero_xent_backward(self.args)
        torch.cuda.synchronize()

    def result(self):
        from zero_sharded_optimizer_step_amd._train_abi import zero_xent_result_t
        return zero_xent_result_t.from_buffer_copy(bytes(self.args.result.cpu().numpy().tobytes()))

    def check(self, backward=True):
        r = train_ref.xent(self.x, self.w, self.target, self.args.grad_scale)
        b = train_ref.xent_bounds(r, self.x, self.w, self.dtype)
        names = ["loss", "lse"] + (["dx", "dw"] if backward else [])
        for name in names:
            got = (getattr(self, "d_" + name) if name in ("dx", "dw") else getattr(self.args, name)).cpu().double()
            err = (got - r[name]).abs()
            worst = (err / b[name].clamp(min=1e-300)).max().item() if err.numel() else 0.0
            say("  %-4s worst error %.3g of its bound" % (name, worst))
            assert bool((err <= b[name]).all()), name
        q = self.result()
        assert q.count == r["count"] and q.out_of_range == int((self.target >= self.w.shape[0]).sum())
        assert abs(q.loss_sum - float(r["sum"])) <= float(b["loss"].sum()) + 1e-12
        assert abs(q.mean - float(r["mean"])) <= float(b["loss"].sum()) / max(1, r["count"]) + 2.0**-23 * abs(float(r["mean"]))
        for name, room in self.rooms.items():            # nothing outside the rows
            view = getattr(self, "d_" + name)
            keep = torch.ones_like(room, dtype=torch.bool)
            keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
            assert bool((room[keep] == -7.0).all()), name


SIZES = [(1, 64, 100), (1, 4096, 1000), (2, 1, 5), (5, 8, 1), (3, 65, 257), (16, 96, 300), (17, 128, 300),
         (130, 200, 515), (64, 513, 1025), (256, 1000, 1024), (509, 72, 2003), (1025, 33, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes(size, dtype):
    say("%s %s" % (size, dtype))
    c = Call(*size, dtype)
    c.run()
    c.check()


# several pieces of the vocabulary; slices of both gradients; large tiles
@pytest.mark.parametrize("size", [(4096, 64, 9001), (512, 2048, 8200), (70, 256, 40000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_large(size):
    say("%s" % (size,))
    c = Call(*size, torch.bfloat16)
    c.run()
    c.check()


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 8)])
def test_strides_and_alignment(pad, shift):
    c = Call(100, 192, 333, torch.bfloat16, pad=pad, shift=shift)
    c.run()
    c.check()


def test_grad_scale_and_repeat():
    c = Call(77, 128, 400, torch.float16, grad_scale=2.0**10)
    c.run()
    c.check()
    first = [c.d_dx.clone(), c.d_dw.clone(), c.args.loss.clone(), c.args.lse.clone()]
    c.ws.fill_(0xFF)
    c.run()
    for a, b in zip(first, [c.d_dx, c.d_dw, c.args.loss, c.args.lse]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 40])
def test_targets_outside(tokens):
    # none counts: loss 0, mean 0, gradients exactly zero; past the vocabulary is counted
    c = Call(tokens, 64, 300, torch.bfloat16)
    c.args.target.fill_(-1)
    c.target.fill_(-1)
    c.args.target[0] = c.target[0] = 300
    c.run()
    c.check()
    assert c.result().mean == 0.0 and c.result().out_of_range == 1
    assert not bool(c.d_dx.any()) and not bool(c.d_dw.any())


def test_infinite_and_nan_logits():
    c = Call(6, 64, 300, torch.bfloat16, ignored=0.0)
    x = c.d_x
    x.abs_()
    c.d_w[7] = -float("inf")                     # x > 0: column 7 is -inf
    x[2] = float("nan")
    x[3] = 0.0                                   # 0 * inf: NaN
    x[4, 0] = float("inf")
    x[:, 0].clamp_(min=0.5)
    x[0].clamp_(min=0.25)
    x[1].clamp_(min=0.25)
    c.args.target[:] = 9
    c.run(backward=False)
    ref = torch.logsumexp(x.cpu().double() @ c.d_w.cpu().double().t(), 1)
    got = c.args.lse.cpu().double()
    say("%s / %s" % (got.tolist(), ref.tolist()))
    assert torch.isnan(got[2]) and torch.isnan(got[3]) and not torch.isfinite(got[4])
    for i in (0, 1, 5):
        assert torch.isfinite(ref[i]) == torch.isfinite(got[i])
        if torch.isfinite(ref[i]):
            assert abs(got[i] - ref[i]) < 1e-4 * abs(ref[i])
    # every logit -inf
    c.d_w[:] = -float("inf")
    x.fill_(1.0)
    c.run(backward=False)
    assert bool((c.args.lse == -float("inf")).all())


def test_no_tokens():
    c = Call(0, 64, 300, torch.bfloat16)
    c.run()
    assert c.result().count == 0 and c.result().mean == 0.0
    assert not bool(c.d_dw.any())


def test_gradient_against_differences():
    # the forward's mean along random directions of x and w, in fp64 central
    # differences of the definition at the same inputs
    c = Call(12, 32, 90, torch.float16)
    c.run()
    g = torch.Generator().manual_seed(5)
    for name in ("x", "w"):
        at = getattr(c, name).double()
        d = torch.randn(at.shape, generator=g, dtype=torch.float64)
        h = 1e-4
        f = [train_ref.xent(*(((at + s * h * d, c.w) if name == "x" else (c.x, at + s * h * d))), c.target)["mean"]
             for s in (1, -1)]
        slope = float((f[0] - f[1]) / (2 * h))
        got = float((getattr(c, "d_d" + name).cpu().double() * d).sum())
        r = train_ref.xent(c.x, c.w, c.target)
        bound = float((train_ref.xent_bounds(r, c.x, c.w, c.dtype)["d" + name] * d.abs()).sum()) + 1e-6
        say("%s: slope %.8f, gradient %.8f, bound %.2g" % (name, slope, got, bound))
        assert abs(slope - got) <= bound


def test_captured_and_on_a_side_stream():
    c = Call(300, 256, 1500, torch.bfloat16)
    e = Call(300, 256, 1500, torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Z.zero_xent_forward(c.args)
        Z.zero_xent_backward(c.args)
    torch.cuda.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Z.zero_xent_forward(c.args)
        Z.zero_xent_backward(c.args)
    for rep in range(3):
        new = torch.randn(300, 256, generator=torch.Generator().manual_seed(rep)).to(torch.bfloat16)
        for q in (c, e):
            q.x = new
            q.d_x.copy_(new)
        for t in (c.d_dx, c.d_dw, c.args.loss):
            t.fill_(0.0)
        g.replay()
        _ = torch.ones(1000, device="cuda").sum().item()
        e.run()
        for name in ("d_dx", "d_dw"):
            assert torch.equal(getattr(c, name), getattr(e, name)), (rep, name)
        assert torch.equal(c.args.lse, e.args.lse) and torch.equal(c.args.result, e.args.result)


# several pieces of the vocabulary: of 256 MB of P, and of 128 MB where w's rows are repacked
@pytest.mark.parametrize("size", [(16384, 64, 8500), (16384, 61, 4200)], ids=lambda s: "x".join(map(str, s)))
def test_pieces(size):
    say("%s" % (size,))
    c = Call(*size, torch.bfloat16, ignored=0.1)
    c.run()
    x, w = c.x.cuda(), c.w.cuda()
    r = train_ref.xent(x, w, c.args.target)
    b = train_ref.xent_bounds(r, x, w, c.dtype)
    for name in ("loss", "lse", "dx", "dw"):
        got = getattr(c, "d_" + name) if name in ("dx", "dw") else getattr(c.args, name)
        assert bool(((got.double() - r[name]).abs() <= b[name]).all()), name


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("size", [(5, 64, 300), (300, 72, 515), (2100, 64, 700)], ids=lambda s: "x".join(map(str, s)))
def test_masked_rows_reach_no_sum(size, bad):
    # rows of x without a target hold NaN or infinities: the others' loss and
    # all of dx and dw are those of the batch without these rows
    c = Call(*size, torch.bfloat16, ignored=0.0, seed=3)
    masked = torch.arange(size[0]) % 3 == 1
    masked[-1] = True
    c.target[masked] = -100
    c.args.target.copy_(c.target)
    c.d_x[masked.cuda()] = bad
    c.run()
    x = c.x.clone()
    x[masked] = 0.0
    r = train_ref.xent(x, c.w, c.target)
    b = train_ref.xent_bounds(r, x, c.w, c.dtype)
    for name in ("dx", "dw"):
        assert bool(((getattr(c, "d_" + name).cpu().double() - r[name]).abs() <= b[name]).all()), name
    loss = c.args.loss.cpu().double()
    assert bool(((loss - r["loss"]).abs() <= b["loss"]).all()) and c.result().count == int((~masked).sum())
    assert not bool(c.d_dx[masked.cuda()].any())


# where the forward changes its kernel, and k that ends inside a wave's share
@pytest.mark.parametrize("size", [(8, 72, 130), (9, 72, 130), (7, 1096, 100), (1, 2056, 50000), (8, 520, 33),
                                  (33, 4104, 300)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_few_tokens(size, dtype):
    say("%s %s" % (size, dtype))
    c = Call(*size, dtype)
    c.run()
    c.check()


def on_gpu(c):
    """A call's outputs against the definition computed in fp64 on the GPU."""
    x, w = c.d_x.contiguous(), c.d_w.contiguous()
    r = train_ref.xent(x, w, c.args.target, c.args.grad_scale)
    b = train_ref.xent_bounds(r, x, w, c.dtype)
    for name in ("loss", "lse", "dx", "dw"):
        got = getattr(c, "d_" + name) if name in ("dx", "dw") else getattr(c.args, name)
        err = (got.double() - r[name]).abs()
        say("  %-4s worst error %.3g of its bound" % (name, (err / b[name].clamp(min=1e-300)).max().item()))
        assert bool((err <= b[name]).all()), name


# every product in 256 x 256 tiles that end oddly, from the caller's rows and from repacked ones
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", [(4100, 3080, 4104), (4100, 3079, 4099), (4000, 72, 3700), (4000, 65, 3701)], ids=lambda s: "x".join(map(str, s)))
def test_large_tiles(size, dtype):
    say("%s %s" % (size, dtype))
    c = Call(*size, dtype, ignored=0.05)
    c.run()
    on_gpu(c)


# w past 2^31 elements and 2^32 bytes
@pytest.mark.parametrize("tokens", [2, 40])
def test_offsets_past_32_bits(tokens):
    vocab, dim = 300000, 8192
    say("%d tokens" % tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda").normal_(0.0, 3.0 / dim**0.5, generator=g)
    x = torch.randn(tokens, dim, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randint(vocab - 1000, vocab, (tokens,), generator=g, device="cuda")
    a = Z.XentArgs(x=x, w=w, target=target, loss=torch.empty(tokens, device="cuda"),
                   lse=torch.empty(tokens, device="cuda"), result=torch.zeros(32, dtype=torch.uint8, device="cuda"),
                   workspace=torch.empty(Z.zero_xent_workspace_bytes(tokens, dim, vocab), dtype=torch.uint8,
                                         device="cuda"), dx=torch.empty_like(x), dw=torch.full_like(w, 9.0))
    Z.zero_xent_forward(a)
    Z.zero_xent_backward(a)
    logits = torch.empty(tokens, vocab, dtype=torch.float64, device="cuda")
    size = torch.empty_like(logits)
    for v in range(0, vocab, 50000):
        logits[:, v:v + 50000] = x.double() @ w[v:v + 50000].double().t()
        size[:, v:v + 50000] = x.double().abs() @ w[v:v + 50000].double().abs().t()
    lse = torch.logsumexp(logits, 1)
    rows = torch.arange(tokens, device="cuda")
    loss = lse - logits[rows, target]
    soft = (logits - lse[:, None]).exp()
    p = soft.clone()
    p[rows, target] -= 1.0
    r = {"loss": loss, "lse": lse, "p": p, "soft": soft, "kept": torch.ones(tokens, dtype=torch.bool, device="cuda"),
         "at": target, "c": 1.0 / tokens, "size": size}
    # the bounds of slices of w's rows: those of dx add up
    bound_dx, dx = torch.zeros(tokens, dim, dtype=torch.float64, device="cuda"), torch.zeros_like(x, dtype=torch.float64)
    u = torch.finfo(torch.bfloat16).eps / 2
    e_row = (dim * 2.0**-23 * size).amax(1)
    dp = p.abs() * u + soft * (2 * e_row + 2.0**-19)[:, None] + 2.0**-134
    dp[rows, target] += 2.0**-23
    assert bool(((a.lse.double() - lse).abs() <= e_row + 2.0**-20 + 2.0**-22 * lse.abs()).all())
    assert bool(((a.loss.double() - loss).abs() <= 2 * e_row + 2.0**-20 + 2.0**-22 * (lse.abs() + (lse - loss).abs())).all())
    for v in range(0, vocab, 50000):
        part, wv = slice(v, v + 50000), w[v:v + 50000].double()
        dx += r["c"] * (p[:, part] @ wv)
        bound_dx += r["c"] * (dp[:, part] @ wv.abs() + vocab * 2.0**-23 * (p[:, part].abs() @ wv.abs())) * (1 + u)
        dw = r["c"] * (p[:, part].t() @ x.double())
        bound = r["c"] * (dp[:, part].t() @ x.double().abs() +
                          tokens * 2.0**-23 * (p[:, part].abs().t() @ x.double().abs())) * (1 + u) + u * dw.abs() + 2.0**-134
        assert bool(((a.dw[part].double() - dw).abs() <= bound).all()), v
    assert bool(((a.dx.double() - dx).abs() <= bound_dx + u * dx.abs() + 2.0**-134).all())


# the same in tiles of 128 x 128 and of 256 x 256: columns of -inf, rows of NaN, all -inf
@pytest.mark.parametrize("size", [(20, 64, 300), (300, 64, 40000), (3900, 64, 3900)], ids=lambda s: "x".join(map(str, s)))
def test_infinite_logits_in_tiles(size):
    c = Call(*size, torch.bfloat16, ignored=0.0)
    c.d_x.abs_().clamp_(min=0.25)                # x > 0: the columns below are -inf
    c.d_w[7:150] = -float("inf")
    c.d_x[2] = float("nan")
    c.d_w[200, 0] = 2.0
    c.d_x[4, 0] = float("inf")                   # its logits are +-inf and NaN
    c.args.target[:] = 220
    c.run(backward=False)
    x, w = c.d_x.double().contiguous(), c.d_w.double().contiguous()
    rest = torch.ones(size[0], dtype=torch.bool, device="cuda")
    rest[2] = rest[4] = False
    alive = torch.ones(size[2], dtype=torch.bool, device="cuda")
    alive[7:150] = False
    logits = x[rest] @ w[alive].t()
    want = torch.logsumexp(logits, 1)
    # as train_ref.xent_bounds has it
    bound = (64 * 2.0**-23 * (x[rest].abs() @ w[alive].abs().t())).amax(1) + 2.0**-20 + 2.0**-22 * want.abs()
    got = c.args.lse.double()
    assert bool(((got[rest] - want).abs() <= bound).all())
    assert bool(torch.isnan(got[2])) and not bool(torch.isfinite(got[4]))
    # a target on a -inf column: an infinite loss, no NaN
    c.args.target[:] = 10
    c.run(backward=False)
    assert bool((c.args.loss[rest] == float("inf")).all())
    c.d_w[:] = -float("inf")
    c.d_x.fill_(1.0)
    c.run(backward=False)
    assert bool((c.args.lse == -float("inf")).all())
