"""Rows of 8-bit codes on the GPU: every code, scale and padding byte equals
the definition's, at row lengths around every change of the kernels."""
import pytest
import torch

import rows8_ref as ref
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def say(msg):
    print(msg, flush=True)


def place(rows, cols, dtype, pad=0, shift=0, src=None, fill=-7):
    """(allocation, view [rows, cols]) with `pad` elements between rows,
    `shift` off the start and 64 behind, all filled with `fill`."""
    room = torch.full((shift + rows * (cols + pad) + 64,), fill, dtype=dtype, device="cuda")
    view = room[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    if src is not None:
        view.copy_(src)
    return room, view


def untouched(room, view, fill=-7):
    """What lies around the view still holds `fill`."""
    mask = torch.ones_like(room, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset() - room.storage_offset()).fill_(False)
    return bool((room[mask] == fill).all())


def sample(rows, dim, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, dim, generator=g) * torch.randn(rows, 1, generator=g).mul(2).exp()
    x[torch.rand(rows, dim, generator=g) < 0.01] *= 20
    return x.to(dtype)


def check(x, pad=0, shift=0, code_pad=0):
    rows, dim = x.shape
    _, dx = place(rows, dim, x.dtype, pad, shift, x)
    room, codes = place(rows, ref.stride(dim), torch.int8, code_pad, 0)
    scales = torch.full((rows + 3,), -7.0, device="cuda")
    Z.zero_rows8_encode(dx, codes, scales[:rows])
    q, s = ref.hold(x)
    assert torch.equal(codes.cpu().long(), q)
    assert torch.equal(scales[:rows].cpu().double().nan_to_num(-1.0), s.nan_to_num(-1.0))
    assert untouched(room, codes) and bool((scales[rows:] == -7).all())
    want = ref.values(q, s, dim)
    for dtype in (DTYPES if x.dtype == torch.float32 else [x.dtype, torch.float32]):
        room, y = place(rows, dim, dtype, pad, shift)
        Z.zero_rows8_decode(codes, scales[:rows], y)
        # one rounding to the type, to nearest even; q s itself is exact in fp32
        assert torch.equal(y.cpu().double().nan_to_num(-1.0), want.float().to(dtype).double().nan_to_num(-1.0))
        assert untouched(room, y)


SIZES = [(1, 1), (3, 7), (300, 16), (5, 64), (5, 65), (9, 128), (9, 129), (64, 512), (6, 513), (33, 2048), (33, 2049),
         (7, 4096), (7, 4097), (5, 8192), (5, 8200), (3, 16384), (3, 16385), (2, 40001), (1, 131071)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype):
    say("rows8 %s %s" % (size, dtype))
    check(sample(*size, dtype))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,shift,code_pad", [(1, 0, 0), (8, 1, 16), (3, 5, 48)])
def test_strides_and_alignment(pad, shift, code_pad, dtype):
    say("rows8 strides %s %s" % ((pad, shift, code_pad), dtype))
    for size in ((13, 100), (5, 777), (4, 4099)):
        check(sample(*size, dtype), pad, shift, code_pad)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim", [24, 1000, 20000])
def test_rows_at_the_edges(dim, dtype):
    """Zeros, the largest and smallest numbers, ties, and the top that rounds to 128."""
    say("rows8 edges %d %s" % (dim, dtype))
    info = torch.finfo(dtype)
    base = sample(1, dim, dtype, seed=dim).clamp(-3, 3)[0] / 4
    tops = [0.0, info.max, -info.max, info.tiny, ref.LEAST[dtype], 127.0, 127.5, -127.49, 127.25, 128.0, 1.0,
            63.5, 64.0, 2.0**-14, 65504.0, 32752.0]
    x = torch.stack([base * 0 if t == 0 else (base.double() * t / 4).to(dtype) for t in tops])
    x[:, 0] = torch.tensor(tops, dtype=torch.float64).to(dtype)
    x[7, 1:6] = torch.tensor([0.5, 1.5, -2.5, 63.5, -126.5]).to(dtype)
    x[11, 1:6] = torch.tensor([0.25, 0.75, -1.25, 31.75, -0.0]).to(dtype)
    check(x)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dim", [40, 3000, 17000])
def test_rows_that_are_not_finite(dim, dtype):
    say("rows8 not finite %d %s" % (dim, dtype))
    x = sample(8, dim, dtype, seed=1)
    for row, col, bad in ((1, 0, "inf"), (3, dim - 1, "-inf"), (4, dim // 2, "nan"), (6, 3, "-nan")):
        x[row, col] = float(bad)
    check(x)


def test_no_rows_and_no_elements():
    for rows, dim in ((0, 40), (0, 0), (5, 0)):
        scale = torch.full((rows,), -7.0, device="cuda")
        codes = torch.empty(rows, ref.stride(dim), dtype=torch.int8, device="cuda")
        Z.zero_rows8_encode(torch.empty(rows, dim, dtype=torch.float16, device="cuda"), codes, scale)
        assert bool((scale == 2.0**-24).all())
        Z.zero_rows8_decode(codes, scale, torch.empty(rows, dim, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()


def test_decode_takes_any_scale():
    say("rows8 any scale")
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(-128, 128, (50, 96), generator=g).to(torch.int8)
    scale = torch.randn(50, generator=g).exp()
    for dtype in DTYPES:
        y = torch.empty(50, 90, dtype=dtype, device="cuda")
        Z.zero_rows8_decode(codes.cuda(), scale.cuda(), y)
        want = (codes[:, :90].float() * scale.view(-1, 1)).to(dtype)
        assert torch.equal(y.cpu(), want)


def test_more_rows_than_a_grid_has_blocks():
    """Rows of a few elements, 32 to a block: a block comes round again."""
    rows = (1 << 25) + 77
    say("rows8 %d rows" % rows)
    x = torch.randn(rows, 4, device="cuda").to(torch.bfloat16)
    codes = torch.full((rows, 16), 5, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    y = torch.empty_like(x)
    Z.zero_rows8_encode(x, codes, scale)
    Z.zero_rows8_decode(codes, scale, y)
    for at in range(0, rows, 1 << 23):
        part = slice(at, min(rows, at + (1 << 23)))
        q, s = ref.hold(x[part])
        assert torch.equal(scale[part].double(), s) and torch.equal(codes[part].long(), q), at
        assert torch.equal(y[part].double(), ref.values(q, s, 4)), at


def test_offsets_past_32_bits():
    rows, dim = 34000, 131064
    say("rows8 %d x %d" % (rows, dim))
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(rows, ref.stride(dim), dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    at = [0, 1, 16383, 16384, 32767, 32768, 33000, rows - 1]
    for r in at:
        x[r].copy_(torch.randn(dim, device="cuda") * (r + 1))
    Z.zero_rows8_encode(x, codes, scale)
    q, s = ref.hold(x[at])
    assert torch.equal(codes[at].long(), q) and torch.equal(scale[at].double(), s)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert bool((scale[keep] == 2.0**-126).all())
    assert int(codes.view(torch.int32).ne(0).any(1).sum()) == len(at)
    x.fill_(1.0)
    Z.zero_rows8_decode(codes, scale, x)
    assert torch.equal(x[at].double(), ref.values(q, s, dim))
    assert int(x.any(1).sum()) == len(at)


def test_captured_and_on_a_side_stream():
    say("rows8 captured")
    x, codes, scale, y = (torch.empty(70, 1001, dtype=torch.bfloat16, device="cuda"),
                          torch.empty(70, 1008, dtype=torch.int8, device="cuda"), torch.empty(70, device="cuda"),
                          torch.empty(70, 1001, dtype=torch.bfloat16, device="cuda"))
    x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Z.zero_rows8_encode(x, codes, scale)
        Z.zero_rows8_decode(codes, scale, y)
    side.synchronize()
    q, s = ref.hold(x)
    assert torch.equal(y.double(), ref.values(q, s, 1001))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_rows8_encode(x, codes, scale)
        Z.zero_rows8_decode(codes, scale, y)
    for i in range(4):
        x.normal_(std=2.0**i)
        graph.replay()
        torch.cuda.synchronize()
        q, s = ref.hold(x)
        assert torch.equal(codes.long(), q) and torch.equal(scale.double(), s)
        assert torch.equal(y.double(), ref.values(q, s, 1001))
