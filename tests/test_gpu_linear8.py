"""The product of 8-bit rows with 8-bit weights and its gradient against the
definition in fp64, with the bounds of rows8_ref, at sizes where tiles, pieces
and slices end oddly and where another kernel takes over."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z
from test_gpu_rows8 import place, say, untouched

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]


class Call:
    def __init__(self, tokens, dim, out, dtype, bias=True, pad=0, shift=0, code_pad=0, seed=0, any_codes=False):
        g = torch.Generator().manual_seed(seed)
        self.t, self.k, self.n, self.dtype = tokens, dim, out, dtype
        self.rooms = []

        def held(rows):
            if any_codes:
                q = torch.randint(-128, 128, (rows, ref.stride(dim)), generator=g)
                q[:, dim:] = 0
                s = torch.randn(rows, generator=g).exp() / 100
            else:
                x = torch.randn(rows, dim, generator=g) * torch.randn(rows, 1, generator=g).exp()
                q, s = ref.hold(x.to(dtype))
            # codes of other rows lie between and behind these
            _, codes = place(rows, ref.stride(dim), torch.int8, code_pad, 0, q.to(torch.int8), fill=77)
            return codes, s.float().cuda()

        def sixteen(rows, cols, src=None):
            room, view = place(rows, cols, dtype, pad, shift, src)
            if src is None:
                self.rooms.append((room, view))
            return view
        self.x8, self.xs = held(tokens)
        self.w8, self.ws = held(out)
        self.bias = torch.randn(out, generator=g).to(dtype).cuda() if bias else None
        self.y = sixteen(tokens, out)
        self.dy = sixteen(tokens, out, torch.randn(tokens, out, generator=g).to(dtype))
        self.dx, self.dw = sixteen(tokens, dim), sixteen(out, dim)
        self.db = sixteen(1, out)[0]
        need = Z.zero_linear8_workspace_bytes(tokens, dim, out)
        self.room = torch.full((need // 4 + 64,), float("nan"), device="cuda").view(torch.uint8)
        self.args = Z.Linear8Args(x8=self.x8, x_scale=self.xs, w8=self.w8, w_scale=self.ws, dim=dim,
                                  workspace=self.room[:need], bias=self.bias, y=self.y, dy=self.dy, dx=self.dx,
                                  dw=self.dw, db=self.db)
        self.need = need

    def check_forward(self):
        want, bound = ref.linear(self.x8, self.xs, self.w8, self.ws, self.k, self.bias)
        ref.within(self.y.double(), want, bound + ref.half_step(want, self.dtype), "y")

    def sixteen_bits(self, codes, scale):
        return ref.values(codes, scale, self.k).float().to(self.dtype).double()

    def check_backward(self):
        dy = self.dy.double()
        dx, off = ref.product(dy, self.sixteen_bits(self.w8, self.ws), self.n)
        ref.within(self.dx.double(), dx, off + ref.half_step(dx, self.dtype), "dx")
        dw, off = ref.product(dy.t(), self.sixteen_bits(self.x8, self.xs), self.t)
        ref.within(self.dw.double(), dw, off + ref.half_step(dw, self.dtype), "dw")
        if self.db is not None:
            db, off = ref.column_sum(dy, self.t)
            ref.within(self.db.double(), db, off + ref.half_step(db, self.dtype), "db")

    def clean(self):
        assert all(untouched(*r) for r in self.rooms)
        tail = self.room[self.need:].view(torch.float32)
        assert bool(torch.isnan(tail).all()), "the workspace was written past its end"

    def check(self):
        Z.zero_linear8_forward(self.args)
        self.check_forward()
        Z.zero_linear8_backward(self.args)
        self.check_backward()
        self.clean()


# tokens around the changes of kernel, dims and outs around 16, 128 and 256
SIZES = [(1, 1, 1), (1, 16, 16), (2, 17, 33), (15, 100, 130), (16, 128, 128), (17, 144, 40), (32, 300, 65), (33, 129, 257),
         (48, 1000, 100), (64, 4096, 48), (65, 4096, 48), (100, 31, 511), (128, 256, 256), (129, 255, 257), (256, 513, 300),
         (257, 1024, 64), (300, 64, 1500), (509, 1000, 700), (1025, 48, 77), (640, 2064, 640)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype):
    say("linear8 %s %s" % (size, dtype))
    Call(*size, dtype, seed=sum(size)).check()


@pytest.mark.parametrize("size", [(2048, 1024, 4200), (4200, 512, 2304), (2300, 4200, 2050)], ids=str)
def test_large_tiles(size):
    say("linear8 large %s" % (size,))
    Call(*size, torch.bfloat16, bias=False).check()


@pytest.mark.parametrize("size", [(700, 3000, 1501), (130, 5000, 3001), (1500, 4200, 260), (260, 16400, 515), (1100, 2100, 130),
                                  (1, 16400, 1024), (17, 12300, 1001), (50, 9000, 2048), (64, 40000, 70), (3, 100001, 9)],
                         ids=str)
def test_sums_cut_into_slices(size):
    """So few tiles and so long a sum that the forward's is cut too, with odd rows of the parts."""
    say("linear8 slices %s" % (size,))
    Call(*size, torch.bfloat16).check()
    Call(*size, torch.float16, bias=False, pad=3, shift=1, any_codes=True).check()


@pytest.mark.parametrize("pad,shift,code_pad", [(1, 0, 16), (3, 5, 0), (8, 8, 48)])
def test_strides_and_alignment(pad, shift, code_pad):
    for size in ((5, 100, 70), (40, 65, 130), (200, 144, 260), (130, 1001, 140)):
        say("linear8 strides %s %s" % (size, (pad, shift, code_pad)))
        Call(*size, torch.float16, pad=pad, shift=shift, code_pad=code_pad).check()


@pytest.mark.parametrize("size", [(3, 200, 104), (70, 520, 264), (300, 1000, 200), (2048, 1024, 2184)], ids=str)
def test_what_lies_beside_dy_is_not_read(size):
    """dy as columns of a wider matrix, aligned so that it is read where it
    lies; a NaN there times the zeros past the last channel would show."""
    t, k, n = size
    say("linear8 beside dy %s" % (size,))
    for dtype in DTYPES:
        c = Call(t, k, n, dtype)
        wide = torch.full((t + 8, n + 72), float("nan"), dtype=dtype, device="cuda")
        wide[4:4 + t, 8:8 + n] = c.dy
        Z.zero_linear8_backward(c.args)
        want = c.dx.clone(), c.dw.clone(), c.db.clone()
        for out in (c.dx, c.dw, c.db):
            out.fill_(-7)
        c.args.dy = wide[4:4 + t, 8:8 + n]
        Z.zero_linear8_backward(c.args)
        assert all(torch.equal(a, b) for a, b in zip((c.dx, c.dw, c.db), want))
        c.clean()


@pytest.mark.parametrize("size", [(3, 200, 100), (30, 2000, 100), (60, 80, 20), (300, 1000, 200)], ids=str)
def test_any_codes_and_scales(size):
    """Codes down to -128 and scales that are no powers of two, which the gradient rounds once."""
    say("linear8 any codes %s" % (size,))
    for dtype in DTYPES:
        Call(*size, dtype, any_codes=True).check()


@pytest.mark.parametrize("out", [20, 1040])
@pytest.mark.parametrize("tokens", [1, 20, 200])
def test_sums_are_whole(tokens, out):
    """The longest row of the largest codes: past 2^24 no fp32 sum would be exact."""
    dim = 131071
    say("linear8 longest %d x %d" % (tokens, out))
    c = Call(tokens, dim, out, torch.float16, bias=False)
    for codes, scale in ((c.x8, c.xs), (c.w8, c.ws)):
        codes[:, :dim] = -128
        scale.fill_(2.0**-13)
    c.x8[:, 1::2] = 127
    c.x8[:, -1] = 0
    c.w8[0, 2::3] = 127
    c.w8[1] = torch.where(torch.arange(c.w8.shape[1], device="cuda") % 2 == 0, 127, 126).to(torch.int8)
    Z.zero_linear8_forward(c.args)
    c.check_forward()


@pytest.mark.parametrize("size", [(1, 5, 3), (1, 5, 8), (1, 513, 3000), (2, 1000, 4099), (2, 16, 70000), (3, 1027, 1100), (4, 3001, 400),
                                  (5, 4100, 8200), (8, 600, 56000), (1, 131071, 65), (9, 30, 31), (16, 1000, 2053), (17, 129, 9),
                                  (31, 2064, 777), (32, 128, 256), (33, 4096, 520), (48, 300, 9001), (49, 1030, 4100), (64, 127, 20011),
                                  (64, 70000, 33), (64, 2048, 1024)], ids=str)
def test_gradient_of_few_tokens(size):
    """One pass over the weights.  A wave adds 32 rows of dx's sum at a time,
    less than a 32nd of all of them, then eight waves' and up to 512 shares'
    sums are joined, the latter 16 at once: 8 + 32 + 16 roundings, for which
    the tiles' bound has 64.  A thread adds at most 8 pairs of db's sum, and
    its 64 values meet in two more steps."""
    t, k, n = size
    say("linear8 few gradient %s" % (size,))
    for dtype, pad, shift in ((torch.bfloat16, 0, 0), (torch.float16, 3, 1)):
        c = Call(t, k, n, dtype, pad=pad, shift=shift, code_pad=16 * pad, any_codes=pad > 0)
        Z.zero_linear8_backward(c.args)
        c.check_backward()
        c.clean()
        # each alone gives the same
        for name in ("dx", "dw"):
            kept = getattr(c, name).clone()
            for other in {"dx", "dw", "db"} - {name}:
                setattr(c.args, other, None)
            getattr(c, name).fill_(-7)
            Z.zero_linear8_backward(c.args)
            assert torch.equal(getattr(c, name), kept), name
            for other in ("dx", "dw", "db"):
                setattr(c.args, other, getattr(c, other))


@pytest.mark.parametrize("size", [(1, 40, 5), (5, 40, 30), (20, 300, 2001), (64, 2048, 1100), (130, 20, 300)], ids=str)
def test_column_sums_alone(size):
    """db alone, in the workspace that few tokens need little of."""
    say("linear8 db alone %s" % (size,))
    c = Call(*size, torch.float16, pad=1)
    c.args.dx = c.args.dw = c.args.x8 = c.args.x_scale = c.args.w8 = c.args.w_scale = None
    Z.zero_linear8_backward(c.args)
    db, off = ref.column_sum(c.dy, c.t)
    ref.within(c.db.double(), db, off + ref.half_step(db, torch.float16), "db")
    assert bool((c.dx == -7).all()) and bool((c.dw == -7).all())
    c.clean()


@pytest.mark.parametrize("size", [(20, 90, 40), (200, 700, 300)], ids=str)
def test_tokens_and_channels_that_are_not_finite(size):
    """A NaN scale is one token's or one channel's in y, that channel's share of every dx and that token's of every dw."""
    say("linear8 not finite %s" % (size,))
    c = Call(*size, torch.bfloat16)
    c.xs[3] = float("nan")
    c.x8[3] = 0
    Z.zero_linear8_forward(c.args)
    Z.zero_linear8_backward(c.args)
    bad = torch.isnan(c.y)
    assert bool(bad[3].all()) and int(bad.sum()) == c.n
    assert bool(torch.isnan(c.dw).all()) and not bool(torch.isnan(c.dx).any())
    c = Call(*size, torch.bfloat16)
    c.ws[7] = float("nan")
    Z.zero_linear8_forward(c.args)
    Z.zero_linear8_backward(c.args)
    bad = torch.isnan(c.y)
    assert bool(bad[:, 7].all()) and int(bad.sum()) == c.t
    assert bool(torch.isnan(c.dx).all()) and not bool(torch.isnan(c.dw).any())
    # and a gradient that overflowed: its token's dx, its channel's dw and db
    c = Call(*size, torch.bfloat16)
    c.dy[5, 9] = float("inf")
    Z.zero_linear8_backward(c.args)
    fine = torch.isfinite(c.dx).all(1)
    assert not bool(fine[5]) and int((~fine).sum()) == 1
    fine = torch.isfinite(c.dw).all(1)
    assert not bool(fine[9]) and int((~fine).sum()) == 1
    fine = torch.isfinite(c.db)
    assert not bool(fine[9]) and int((~fine).sum()) == 1


def test_only_what_is_wanted():
    for wanted in (("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db")):
        say("linear8 wanted %s" % (wanted,))
        c = Call(150, 200, 170, torch.float16)
        for name in ("dx", "dw", "db"):
            if name not in wanted:
                setattr(c.args, name, None)
        if "dx" not in wanted:
            c.args.w8 = c.args.w_scale = None
        if "dw" not in wanted:
            c.args.x8 = c.args.x_scale = None
        Z.zero_linear8_backward(c.args)
        kept = {name: getattr(c, name).clone() for name in wanted}
        for name in ("dx", "dw", "db"):
            assert name in wanted or bool((getattr(c, name) == -7).all())
        full = Call(150, 200, 170, torch.float16)
        Z.zero_linear8_backward(full.args)
        for name in wanted:
            assert torch.equal(kept[name], getattr(full, name)), name


@pytest.mark.parametrize("size", [(0, 40, 30), (5, 0, 30), (100, 0, 30), (5, 40, 0), (1, 40, 0), (2, 0, 30), (0, 0, 0), (0, 0, 5), (3, 0, 0)], ids=str)
def test_empty_sizes(size):
    say("linear8 empty %s" % (size,))
    c = Call(*size, torch.bfloat16, pad=2)
    Z.zero_linear8_forward(c.args)
    Z.zero_linear8_backward(c.args)
    torch.cuda.synchronize()
    if c.t and c.n:
        assert torch.equal(c.y, c.bias.expand(c.t, c.n))
        c.check_backward()
    else:
        assert not bool(c.dx.any()) and not bool(c.dw.any()) and not bool(c.db.any())
    c.clean()


@pytest.mark.parametrize("size,dim_at", [((96, 600, 1 << 20), 256), ((300, 1100, 500000), 512)], ids=str)
def test_columns_in_pieces(size, dim_at):
    """So many rows that the held values are written out some columns at a time."""
    t, k, n = size
    say("linear8 pieces %s" % (size,))
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(n, k, generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn(t, k, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(t, n, generator=g, device="cuda").to(torch.bfloat16)
    hold = []
    for m in (x, w):
        q, s = torch.empty(m.shape[0], ref.stride(k), dtype=torch.int8, device="cuda"), torch.empty(m.shape[0], device="cuda")
        Z.zero_rows8_encode(m, q, s)
        Z.zero_rows8_decode(q, s, m)
        hold.append((q, s))
    room = torch.empty(Z.zero_linear8_workspace_bytes(t, k, n), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    Z.zero_linear8_backward(Z.Linear8Args(*hold[0], *hold[1], dim=k, workspace=room, dy=dy, dx=dx, dw=dw))
    # columns of every piece, around its ends
    cols = sorted({0, 1, dim_at - 1, dim_at, dim_at + 1, k - 1, k // 2})
    want, off = ref.product(dy.double(), w[:, cols].double(), n)
    ref.within(dx[:, cols].double(), want, off + ref.half_step(want, torch.bfloat16), "dx")
    rows = torch.randint(0, n, (2000,), generator=g, device="cuda")
    want, off = ref.product(dy[:, rows].double().t(), x.double(), t)
    ref.within(dw[rows].double(), want, off + ref.half_step(want, torch.bfloat16), "dw")


def test_more_of_dy_than_the_caches_hold():
    t, k, n = 8209, 48, 16424
    say("linear8 %d x %d x %d" % (t, k, n))
    g = torch.Generator(device="cuda").manual_seed(0)
    dy = torch.randn(t, n + 3, generator=g, device="cuda").to(torch.float16)[:, :n]
    w = torch.randn(n, k, generator=g, device="cuda").to(torch.float16)
    w8, ws = torch.empty(n, 48, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    Z.zero_rows8_encode(w, w8, ws)
    Z.zero_rows8_decode(w8, ws, w)
    dx, db = torch.empty(t, k, dtype=torch.float16, device="cuda"), torch.empty(n, dtype=torch.float16, device="cuda")
    room = torch.empty(Z.zero_linear8_workspace_bytes(t, k, n), dtype=torch.uint8, device="cuda")
    Z.zero_linear8_backward(Z.Linear8Args(None, None, w8, ws, dim=k, workspace=room, dy=dy, dx=dx, db=db))
    want, off = ref.column_sum(dy, t)
    ref.within(db.double(), want, off + ref.half_step(want, torch.float16), "db")
    rows = torch.arange(0, t, 7, device="cuda")
    want, off = ref.product(dy[rows].double(), w.double(), n)
    ref.within(dx[rows].double(), want, off + ref.half_step(want, torch.float16), "dx")


@pytest.mark.parametrize("tokens", [2, 64, 70])
def test_offsets_past_32_bits(tokens):
    """Weights of more than 4 GB."""
    dim, out = 4112, 1 << 20
    say("linear8 %d x %d x %d" % (tokens, dim, out))
    g = torch.Generator(device="cuda").manual_seed(0)
    w8 = torch.randint(-127, 128, (out, dim), generator=g, device="cuda", dtype=torch.int8)
    x8 = torch.randint(-127, 128, (tokens, dim), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = (torch.full((r,), 2.0**-9, device="cuda") for r in (tokens, out))
    y = torch.empty(tokens, out, dtype=torch.bfloat16, device="cuda")
    room = torch.empty(Z.zero_linear8_workspace_bytes(tokens, dim, out), dtype=torch.uint8, device="cuda")
    Z.zero_linear8_forward(Z.Linear8Args(x8, xs, w8, ws, dim=dim, workspace=room, y=y))
    parts = (slice(0, 300), slice((1 << 19) + 5, (1 << 19) + 3000), slice(out - 777, out))
    for rows in parts:
        want, off = ref.linear(x8, xs, w8[rows], ws[rows], dim, None)
        ref.within(y[:, rows].double(), want, off + ref.half_step(want, torch.bfloat16), "y")
    dy = torch.randn(tokens, out, generator=g, device="cuda").to(torch.bfloat16)
    dx = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(out, dim, dtype=torch.bfloat16, device="cuda")
    Z.zero_linear8_backward(Z.Linear8Args(x8, xs, w8, ws, dim=dim, workspace=room, dy=dy, dx=dx, dw=dw))
    cols = [0, 1, 255, 256, 511, 512, 3000, dim - 1]
    want, off = ref.product(dy.double(), w8[:, cols].double() * 2.0**-9, out)
    ref.within(dx[:, cols].double(), want, off + ref.half_step(want, torch.bfloat16), "dx")
    for rows in parts:
        want, off = ref.product(dy[:, rows].double().t(), x8.double() * 2.0**-9, tokens)
        ref.within(dw[rows].double(), want, off + ref.half_step(want, torch.bfloat16), "dw")


def test_gradient_against_differences():
    """d/dx and d/dw of sum(dy y) as the forward itself changes: the product is
    linear, so a change of one code changes the sum by the gradient's element."""
    say("linear8 differences")
    t, k, n = 40, 60, 50
    c = Call(t, k, n, torch.float16, bias=False)
    c.x8.clamp_(-100, 100)
    c.w8.clamp_(-100, 100)
    Z.zero_linear8_backward(c.args)
    dy = c.dy.double()

    def total():
        Z.zero_linear8_forward(c.args)
        return (dy * c.y.double()).sum(), (dy * ref.half_step(c.y.double(), torch.float16) * 2.02).abs().sum()
    base, off0 = total()
    for codes, scale, grad, row, col in ((c.x8, c.xs, c.dx, 7, 59), (c.x8, c.xs, c.dx, 39, 0), (c.w8, c.ws, c.dw, 49, 31),
                                         (c.w8, c.ws, c.dw, 3, 17)):
        old = codes[row, col].clone()
        codes[row, col] = old + 20
        more, off1 = total()
        codes[row, col] = old
        got = grad[row, col].double() * 20 * scale[row].double()
        # both sums are of rounded y (and fp32's few roundings of them), the gradient is rounded once
        assert abs(more - base - got) <= off0 + off1 + abs(got) * 2.0**-10


def test_results_do_not_depend_on_the_run():
    say("linear8 repeated")
    for size in ((30, 900, 200), (509, 1000, 700)):
        c = Call(*size, torch.bfloat16)
        seen = []
        for _ in range(3):
            Z.zero_linear8_forward(c.args)
            Z.zero_linear8_backward(c.args)
            seen.append([m.clone() for m in (c.y, c.dx, c.dw, c.db)])
            c.room[:c.need].fill_(0x7f)                    # nothing of the last call's is read
        assert all(torch.equal(a, b) for other in seen[1:] for a, b in zip(seen[0], other))


@pytest.mark.parametrize("size", [(1, 700, 300), (4, 1000, 2000), (40, 700, 300), (300, 700, 333)], ids=str)
def test_captured_and_on_a_side_stream(size):
    say("linear8 captured %s" % (size,))
    c = Call(*size, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Z.zero_linear8_forward(c.args)
        Z.zero_linear8_backward(c.args)
    side.synchronize()
    c.check_forward()
    c.check_backward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_linear8_forward(c.args)
        Z.zero_linear8_backward(c.args)
    for _ in range(4):
        c.x8[:, :c.k].random_(-127, 128)
        c.dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        c.check_forward()
        c.check_backward()


def test_two_calls_at_once():
    """Calls with workspaces of their own on two streams."""
    say("linear8 two streams")
    calls = [Call(300, 700, 500, torch.bfloat16, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(calls, streams):
            Z.zero_linear8_forward(c.args, stream=s)
            Z.zero_linear8_backward(c.args, stream=s)
    torch.cuda.synchronize()
    for c in calls:
        c.check_forward()
        c.check_backward()
        c.clean()
