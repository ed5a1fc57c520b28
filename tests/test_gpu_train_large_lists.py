"""Lists of more than a few chunks of 1024 elements: where the step joins the
norm in a launch of its own (above 2048 chunks), where a block of the norm has
several runs in flight and goes round again (above 16384), and past 32 bits of
bytes.  Expected values are one rounding per operation in fp32 torch, or the
8-bit codes by their definition, for every element."""
import numpy as np
import pytest
import torch

import train_ref as R
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu

CHUNK, BLOCK = 1024, 256
GROUPS = [Z.AdamGroup(lr=1e-3), Z.AdamGroup(lr=2e-4, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0)]
STEP = 7


def say(msg):
    print(msg, flush=True)


def f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def i32(x):
    x &= 0xFFFFFFFF
    return x - (1 << 32) if x >> 31 else x


# ---------------------------------------------- the 8-bit state, in torch on the GPU
def scaled(x, k):
    """x 2^k in fp64, k whole and within its exponents."""
    return x * ((k.long() + 1023) << 52).view(torch.float64)


def exponents(x):
    """Biased exponents [b, 1] of the largest of x [b, 256] >= 0: one more above mantissa 1.875."""
    big = x.amax(1, keepdim=True)
    f, e = torch.frexp(big.double())                     # big = f 2^e, f in [0.5, 1)
    e = torch.where(big > 0, e - 1 + (f > 0.9375).int(), torch.full_like(e, -127))
    return (e + 127).clamp(1, 254)


def codes(x, e, field, noise):
    """Codes of x >= 0 under e: y in steps of its binade's eighth, plus the noise, down."""
    y = scaled(x.double(), field - e)
    _, k = torch.frexp(y)
    k = (k - 1).clamp(min=-126)
    n = torch.floor(scaled(y, 3 - k) + noise)            # [8, 16], below 8 when subnormal
    up = n >= 16
    k, n = torch.where(up, k + 1, k), torch.where(up, torch.full_like(n, 8.0), n).int()
    return torch.where(n < 8, n, (k + 127) * 8 + n - 8).clamp(0, 8 * field + 7)


def values(c, e, field):
    k = (c >> 3).clamp(min=1)
    n = (c & 7) + torch.where(c >> 3 > 0, 8, 0)
    return scaled(n.double(), k - field + e - 127 - 3).float()


def fmix(x):
    """MurmurHash3's 32-bit finalizer on int32."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * i32(0x85EBCA6B)
    x = x ^ ((x >> 13) & 0x7FFFF)
    x = x * i32(0xC2B2AE35)
    return x ^ ((x >> 16) & 0xFFFF)


def noises(first, blocks, seed):
    key = (seed & 0xFFFFFFFF) ^ int(R._fmix(np.array([seed >> 32], dtype=np.uint64))[0])
    place = torch.arange(blocks * BLOCK, dtype=torch.int64, device="cuda") + first * BLOCK
    h = fmix((place * 0x9E3779B1 + key).to(torch.int32)).view(-1, BLOCK)
    return [(n * 16 + 8).double() / 2**20 for n in (h & 0xFFFF, (h >> 16) & 0xFFFF)]


def unpack(s8, e8):
    s, e = s8.view(-1, 2, BLOCK).int(), e8.view(-1, 2).int()
    m = values(s[:, 0] & 127, e[:, :1], 15)
    return torch.where(s[:, 0] > 127, -m, m).view(-1), values(s[:, 1], e[:, 1:], 31).view(-1)


def pack(m, v, noise):
    m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
    em, ev = exponents(m.abs()), exponents(v)
    cm, cv = codes(m.abs(), em, 15, noise[0]), codes(v, ev, 31, noise[1])
    cv = torch.where(v > 0, cv.clamp(min=1), cv)
    cm = torch.where((m < 0) & (cm > 0), cm + 128, cm)
    return torch.stack([cm, cv], 1).to(torch.uint8).view(-1), torch.cat([em, ev], 1).to(torch.uint8).view(-1)


# --------------------------------------------------------------------- the lists
def blocks_of(n):
    return -(-n // BLOCK)


class Large:
    """Tensors carved out of flat buffers, packed end to end from element 3 on.
    The 8-bit state starts from zero codes and is filled by a first step."""

    def __init__(self, sizes, bits, grad=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.bits = sizes, bits
        self.group = [t % 2 for t in range(len(sizes))]
        self.places = [3 + sum(sizes[:t]) for t in range(len(sizes))]
        total = sum(sizes) + 8
        self.grad = torch.randn(total, generator=g, device="cuda").mul_(1e-3).to(grad)
        self.master = torch.randn(total, generator=g, device="cuda").mul_(0.02)
        self.param = torch.full((total,), 9.0, dtype=torch.bfloat16, device="cuda")
        if bits == 32:
            self.m = torch.randn(total, generator=g, device="cuda").mul_(1e-4)
            self.v = torch.randn(total, generator=g, device="cuda").mul_(1e-3).square_()
        else:
            k = sum(blocks_of(n) for n in sizes)
            m = torch.randn(k * BLOCK, generator=g, device="cuda").mul_(1e-4)
            v = torch.randn(k * BLOCK, generator=g, device="cuda").mul_(1e-3).square_()
            b = 0
            for n in sizes:                               # what pads a last block is zero
                m[b + n:b + blocks_of(n) * BLOCK] = 0.0
                v[b + n:b + blocks_of(n) * BLOCK] = 0.0
                b += blocks_of(n) * BLOCK
            self.s8, self.e8 = pack(m, v, (0.5, 0.5))

    def cut(self, t, flat):
        return flat[self.places[t]:self.places[t] + self.sizes[t]]

    def cut8(self, t):
        b = sum(blocks_of(n) for n in self.sizes[:t])
        k = blocks_of(self.sizes[t])
        return self.s8[b * 512:(b + k) * 512], self.e8[b * 2:(b + k) * 2]

    def set(self, lo=0, hi=None):
        r = range(len(self.sizes))[lo:hi]
        if self.bits == 32:
            state = dict(exp_avg=[self.cut(t, self.m) for t in r], exp_avg_sq=[self.cut(t, self.v) for t in r])
        else:
            state = dict(state8=[self.cut8(t)[0] for t in r], scale8=[self.cut8(t)[1] for t in r])
        return Z.TensorSet(master=[self.cut(t, self.master) for t in r], grad=[self.cut(t, self.grad) for t in r],
                           param=[self.cut(t, self.param) for t in r], group=[self.group[t] for t in r], **state)

    def sumsq(self, lo=0, hi=None):
        return sum(float(self.cut(t, self.grad).double().square().sum()) for t in range(len(self.sizes))[lo:hi])

    def expected(self, t, coef, seed, first_block):
        """(master, param, first state, second state) of tensor t after the step."""
        h, n = GROUPS[self.group[t]], self.sizes[t]
        g = self.cut(t, self.grad).float() * f32(coef)
        if self.bits == 32:
            m, v = self.cut(t, self.m), self.cut(t, self.v)
        else:
            m, v = (x[:n] for x in unpack(*self.cut8(t)))
        m = m * f32(h.beta1) + g * f32(1 - h.beta1)
        v = v * f32(h.beta2) + (g * g) * f32(1 - h.beta2)
        d = v.sqrt() * f32(1 / (1 - h.beta2**STEP)**0.5) + f32(h.eps)
        p = self.cut(t, self.master) * f32(1 - h.lr * h.weight_decay) - (m / d) * f32(h.lr / (1 - h.beta1**STEP))
        if self.bits == 8:
            k = blocks_of(n)
            m, v = (torch.nn.functional.pad(x, (0, k * BLOCK - n)) for x in (m, v))
            m, v = pack(m, v, noises(first_block, k, seed))
        return p, p.to(torch.bfloat16), m, v

    def found(self, t):
        state = (self.cut(t, self.m), self.cut(t, self.v)) if self.bits == 32 else self.cut8(t)
        return (self.cut(t, self.master), self.cut(t, self.param)) + tuple(state)

    def check_against(self, want, lo=0):
        for t, w in enumerate(want, lo):
            for name, a, b in zip(("master", "param", "first state", "second state"), self.found(t), w):
                assert torch.equal(a, b), (t, name, int((a != b).sum()))


def step_and_check(q, max_norm, seed=(3 << 32) + 5):
    ts = q.set()
    sumsq = q.sumsq()
    # the kernel's coef, bounded here, is what the expected values take: fp64
    # sums of another order can round it to the fp32 beside
    want = min(1.0, max_norm / (sumsq**0.5 + 1e-6)) if max_norm else 1.0
    coef = f32(want)
    first = [sum(blocks_of(n) for n in q.sizes[:t]) for t in range(len(q.sizes))]
    before = {c: [q.expected(t, c, seed, first[t]) for t in range(len(q.sizes))]
              for c in ({coef} if coef == 1.0 else {coef, f32(np.nextafter(np.float32(coef), np.float32(0))),
                                                    f32(np.nextafter(np.float32(coef), np.float32(2)))})}
    info = Z.zero_tensors_step(ts, GROUPS, step=STEP, max_grad_norm=max_norm, seed=seed, want_info=True)
    say("%d chunks: sumsq %.17g, %.17g expected" % (ts.plan.n_chunks, info.sumsq, sumsq))
    assert info.overflow == 0 and info.clipped == (1 if want < 1 else 0)
    assert abs(info.sumsq - sumsq) <= 1e-12 * sumsq and abs(info.norm - sumsq**0.5) <= 1e-12 * sumsq**0.5
    assert info.coef in before
    q.check_against(before[info.coef])
    return ts


def ragged(chunks):
    """Sizes of exactly `chunks` chunks: long and short tensors that end inside
    a chunk, a half chunk, a block and a quad."""
    sizes = [1, 511, 513, 1023, 1025, 255, 3]            # 8 chunks
    rest = chunks - 8
    return [n + (rest // 2 * CHUNK if i == 3 else (rest - rest // 2) * CHUNK if i == 5 else 0)
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("chunks", [2048, 2049, 16385, 40000])
@pytest.mark.parametrize("max_norm", [0.0, 0.5], ids=["whole", "clipped"])
def test_step_of_many_chunks(bits, chunks, max_norm):
    say("bits %d, %d chunks" % (bits, chunks))
    q = Large(ragged(chunks), bits, grad=torch.float32 if chunks == 16385 else torch.bfloat16, seed=chunks)
    ts = step_and_check(q, max_norm)
    assert ts.plan.n_chunks == chunks


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("where", ["first", "late", "last"])
def test_one_bad_element_of_many_skips_the_step(bits, where):
    # late: in a run that a block of the norm has in flight behind others
    q = Large(ragged(40000), bits, seed=1)
    at = {"first": 3, "late": 3 + 7 * 2048 * CHUNK + 77, "last": 3 + sum(q.sizes) - 1}[where]
    q.grad[at] = float("inf")
    old = [x.clone() for x in ((q.master, q.param, q.m, q.v) if bits == 32 else (q.master, q.param, q.s8, q.e8))]
    info = Z.zero_tensors_step(q.set(), GROUPS, step=STEP, max_grad_norm=1.0, seed=1, want_info=True)
    assert info.overflow == 1
    for a, b in zip(old, (q.master, q.param, q.m, q.v) if bits == 32 else (q.master, q.param, q.s8, q.e8)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[5000, 300, 777], ragged(2500)], ids=["short", "long"])
def test_two_lists_by_one_norm(bits, sizes):
    # norm, combine and apply of two lists: every field is the definition's under
    # the coef that the combine left, each list's blocks counted from 0
    q = Large(sizes, bits, seed=11)
    cut = len(sizes) // 2
    parts = [q.set(0, cut), q.set(cut)]
    table = torch.empty(Z.zero_partials_bytes(2), dtype=torch.uint8, device="cuda")
    glob = torch.zeros(32, dtype=torch.uint8, device="cuda")
    for k, p in enumerate(parts):
        Z.zero_tensors_norm(p, GROUPS, STEP, k, table)
    Z.zero_shard_combine(table, 2, 1e-2, glob)
    sumsq, coef = glob.view(torch.float64)[0].item(), glob.view(torch.float32)[4].item()
    want = q.sumsq()
    assert abs(sumsq - want) <= 1e-12 * want
    assert abs(coef - 1e-2 / (want**0.5 + 1e-6)) <= 2.0**-23 * coef and coef < 1.0
    seed = 99
    expected = []
    for lo, hi in ((0, cut), (cut, len(sizes))):
        block = 0
        for t in range(lo, hi):
            expected.append(q.expected(t, coef, seed, block))
            block += blocks_of(sizes[t])
    for p in parts:
        Z.zero_tensors_apply(p, GROUPS, STEP, glob, seed=seed)
    torch.cuda.synchronize()
    q.check_against(expected)


# the 8-bit codes of a list pass 2^32 bytes, and so do fp32 fields of less
@pytest.mark.parametrize("bits,n", [(32, (1 << 30) + 3333), (8, (1 << 31) + 3333)])
def test_offsets_past_32_bits(bits, n):
    say("bits %d, n %d" % (bits, n))
    g = torch.Generator(device="cuda").manual_seed(2)
    grad = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1e-3, generator=g)
    master = torch.empty(n, device="cuda").normal_(0.0, 0.02, generator=g)
    param = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    if bits == 32:
        state = [torch.zeros(n, device="cuda") for _ in range(2)]
        ts = Z.TensorSet(master=[master], grad=[grad], param=[param], exp_avg=state[:1], exp_avg_sq=state[1:])
    else:
        k = blocks_of(n)
        state = [torch.zeros(512 * k, dtype=torch.uint8, device="cuda"),
                 torch.ones(2 * k, dtype=torch.uint8, device="cuda")]
        ts = Z.TensorSet(master=[master], grad=[grad], param=[param], state8=state[:1], scale8=state[1:])
    windows = [(a, min(a + (1 << 20), n)) for a in (0, 1 << 29, (1 << 30) - (1 << 19), 1 << 30, (1 << 31) - (1 << 19), 1 << 31)
               if a < n] + [((n - 1) // BLOCK * BLOCK - (1 << 20), n)]
    old = [master[a:b].clone() for a, b in windows]
    sumsq = sum(float(x.double().square().sum()) for x in grad.split(1 << 27))
    info = Z.zero_tensors_step(ts, GROUPS[:1], step=STEP, max_grad_norm=0.0, seed=5, want_info=True)
    assert abs(info.sumsq - sumsq) <= 1e-12 * sumsq and info.overflow == 0
    for (a, b), p0 in zip(windows, old):
        q = Large.__new__(Large)
        q.sizes, q.bits, q.group, q.places = [b - a], bits, [0], [0]
        q.grad, q.master = grad[a:b], p0
        if bits == 32:
            q.m = q.v = torch.zeros(b - a, device="cuda")
        else:
            q.s8 = torch.zeros(512 * blocks_of(b - a), dtype=torch.uint8, device="cuda")
            q.e8 = torch.ones(2 * blocks_of(b - a), dtype=torch.uint8, device="cuda")
        p, c, m, v = q.expected(0, 1.0, 5, a // BLOCK)
        at, to = a // BLOCK, blocks_of(b)
        got = [s[a:b] for s in state] if bits == 32 else [state[0][at * 512:to * 512], state[1][at * 2:to * 2]]
        for name, x, y in (("master", master[a:b], p), ("param", param[a:b], c), ("first", got[0], m), ("second", got[1], v)):
            assert torch.equal(x, y), (a, name)


def test_state8_offsets_past_32_bits():
    n = (1 << 31) + 777                                   # codes: 2 n bytes; moments: 4 n
    g = torch.Generator(device="cuda").manual_seed(4)
    m = torch.empty(n, device="cuda").normal_(0.0, 1e-4, generator=g)
    v = torch.empty(n, device="cuda").normal_(0.0, 1e-3, generator=g).square_()
    k = blocks_of(n)
    s8 = torch.empty(512 * k, dtype=torch.uint8, device="cuda")
    e8 = torch.empty(2 * k, dtype=torch.uint8, device="cuda")
    Z.zero_state8_encode(m, v, s8, e8)
    mo, vo = torch.empty_like(m), torch.empty(n, device="cuda")
    Z.zero_state8_decode(s8, e8, mo, vo)
    mh, vh = (torch.empty(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Z.zero_state8_decode(s8, e8, mh, vh)
    for a in range(0, n, 1 << 28):                        # every element
        b = min(a + (1 << 28), n)
        wm, wv = unpack(s8[a * 2:blocks_of(b) * 512], e8[a // BLOCK * 2:blocks_of(b) * 2])
        wm, wv = wm[:b - a], wv[:b - a]
        for got, want in ((mo, wm), (vo, wv)):
            assert torch.equal(got[a:b], want), a
        for got, want in ((mh, wm), (vh, wv)):
            assert torch.equal(got[a:b], want.to(torch.bfloat16)), a
        # the code is the nearest: half a step of an eighth of the binade, below
        # the least binade of its exponent half of that one's step
        for x, e, field, want in ((m, 0, 15, wm), (v, 1, 31, wv)):
            top = e8[a // BLOCK * 2:blocks_of(b) * 2].view(-1, 2)[:, e].long().repeat_interleave(BLOCK)[:b - a]
            least = scaled(torch.ones(b - a, dtype=torch.float64, device="cuda"), 1 - field + top - 127)
            step = torch.maximum(x[a:b].abs().double(), least) * (1 / 16)
            low = least / 8 if field == 31 else 0.0       # a second moment above zero is at least code 1
            assert bool(((x[a:b].double() - want.double()).abs() <= step + low).all()), a
            del top, least, step
