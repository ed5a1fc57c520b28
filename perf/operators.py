"""What the training operators are measured on: AdamW over a list of tensors
with 32-bit and with 8-bit states, the conversion between the two, and the
softmax cross entropy of a large vocabulary with and without its gradient.

Every tensor list is carved out of flat buffers, one per field, each tensor
starting at a multiple of `align` elements (256: as separate allocations lie;
1: packed, so most tensors start off any vector boundary).  The fields come
back as the whole flat buffers.

The 8-bit state.  Blocks of 256 elements of a tensor share a biased fp32
exponent E per moment: that of the block's largest magnitude, one more where
its mantissa is above 1.875, clamped to [1, 254].  The first moment is a sign
and 4 exponent and 3 mantissa bits below E, the second 5 and 3 bits without a
sign, both with gradual underflow; a second moment above zero is never held as
zero.  Block b's 256 codes of the first moment are followed by its 256 codes
of the second, and `scale8` holds its two exponents.  An update rounds
stochastically, with 16 bits per moment of a hash of the element's place (block
ordinal in the list * 256 + place in the block) and a key made of the seed.
"""
import math
import random

import torch

own = False

BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 6e-5, 0.9, 0.999, 1e-8, 0.01
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = "512x512 512 512x1024 1024"
SHARD_13B = 1_625_000_064


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # the four tensors of a tiny fp16 model at loss scale 2^16: latency counts
        dict(name="adamw32 tiny fp16", op="adamw", bits=32, kind="tiny", grad="fp16", param="fp16",
             align=256, groups=1, loss_scale=65536.0, max_norm=1.0, step=3),
        # 300 ragged tensors, log-uniform 1e3..3e6, weights decayed and vectors not
        dict(name="adamw32 ragged bf16", op="adamw", bits=32, kind="ragged", count=300, lo=1000,
             hi=3_000_000, sizes_seed=0, grad="bf16", param="bf16", align=256, groups=2,
             loss_scale=1.0, max_norm=1.0, step=100),
        # one rank's shard of a 13B model over 8 ranks, as a single tensor
        dict(name="adamw32 13B/8 shard bf16", op="adamw", bits=32, kind="shard", grad="bf16",
             param="bf16", align=256, groups=1, loss_scale=1.0, max_norm=1.0, step=10),
        # packed small tensors with fp32 gradients summed over micro-batches: off every boundary
        dict(name="adamw8 packed small fp32", op="adamw", bits=8, kind="ragged", count=200, lo=1,
             hi=40_000, sizes_seed=1, grad="fp32", param="bf16", align=1, groups=2, loss_scale=1.0,
             max_norm=1.0, step=1000),
        # an encoder layer at d_model 4096: four projections and their biases
        dict(name="adamw8 encoder layer bf16", op="adamw", bits=8, kind="encoder", grad="bf16",
             param="bf16", align=256, groups=2, loss_scale=1.0, max_norm=1.0, step=10),
        # the 13B/8 shard with its moments in 8 bits
        dict(name="adamw8 13B/8 shard bf16", op="adamw", bits=8, kind="shard", grad="bf16",
             param="bf16", align=256, groups=1, loss_scale=1.0, max_norm=1.0, step=10),
        # a saved 32-bit state taken over into 8 bits and read back: one encoder layer
        dict(name="state8 there and back", op="state8", way="both", n=67_125_248),
        # an 8-bit state written out as fp32 for a checkpoint, odd length
        dict(name="state8 to fp32", op="state8", way="decode", n=500_000_003),
        # scoring one token: the weights are read once, latency and bandwidth count
        dict(name="loss one token bf16", op="loss", tokens=1, dim=4096, vocab=32000, dtype="bf16",
             ignored=0.0),
        # evaluation of a full batch: perplexity without a gradient
        dict(name="loss 4096 tokens bf16", op="loss", tokens=4096, dim=4096, vocab=128000,
             dtype="bf16", ignored=0.0),
        # a short ragged fp16 batch, nothing a multiple of anything, some tokens masked
        dict(name="loss+grad odd fp16", op="grad", tokens=509, dim=1000, vocab=10007, dtype="fp16",
             ignored=0.3),
        # the training step of a large head
        dict(name="loss+grad 4096 tokens bf16", op="grad", tokens=4096, dim=4096, vocab=128000,
             dtype="bf16", ignored=0.05),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "state8", "loss", "grad"])
    if op == "adamw":
        hi = _log(rng, 1000, 3_000_000)
        return dict(op=op, bits=rng.choice([8, 32]), kind="ragged", count=_log(rng, 1, 300), lo=1,
                    hi=hi, sizes_seed=rng.randrange(1 << 30), grad=rng.choice(["bf16", "fp16", "fp32"]),
                    param=rng.choice(["bf16", "fp16", "none"]), align=rng.choice([1, 256]),
                    groups=rng.choice([1, 2]), loss_scale=rng.choice([1.0, 1024.0]),
                    max_norm=rng.choice([0.0, 1.0]), step=_log(rng, 1, 10000))
    if op == "state8":
        return dict(op=op, way=rng.choice(["both", "decode"]), n=_log(rng, 1, 200_000_000))
    tokens, dim = _log(rng, 1, 8192), _log(rng, 64, 8192)
    if rng.random() < 0.5:
        dim = max(64, dim // 64 * 64)
    top = min(128000, 4096 * 4096 * 128000 // (tokens * dim))
    return dict(op=op, tokens=tokens, dim=dim, vocab=_log(rng, 100, max(200, top)),
                dtype=rng.choice(["bf16", "fp16"]), ignored=rng.choice([0.0, 0.1, 0.5]))


def _sizes(case):
    if case["kind"] == "tiny":
        return [math.prod(int(d) for d in s.split("x")) for s in TINY.split()]
    if case["kind"] == "encoder":
        return [4096 * 4096, 4096] * 4
    if case["kind"] == "shard":
        return [SHARD_13B]
    r = random.Random(case["sizes_seed"])
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    return [max(1, int(math.exp(r.uniform(lo, hi)))) for _ in range(case["count"])]


def _up(n, a):
    return -(-n // a) * a


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        grad = 4 if case["grad"] == "fp32" else 2
        cast = 0 if case["param"] == "none" else 2
        # the 8-bit moments come back as bf16 values, which reads them once more
        state = 16 if case["bits"] == 32 else 4 + 2 + 4
        return {"bytes": n * (grad + 8 + cast + state), "flops": 25 * n}
    if case["op"] == "state8":
        n = case["n"]
        return {"bytes": n * (8 + 2 + 2 + 4 if case["way"] == "both" else 2 + 8), "flops": 8 * n}
    t, d, v = case["tokens"], case["dim"], case["vocab"]
    if case["op"] == "loss":
        return {"bytes": 2 * (t * d + v * d) + 16 * t, "flops": 2 * t * d * v}
    return {"bytes": 4 * (t * d + v * d) + 16 * t, "flops": 8 * t * d * v}


# ------------------------------------------------------------ the 8-bit state
def _scaled(x, k):
    """x (fp64) times 2^k, k whole and within fp64's normal range: exact."""
    return x * ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _bits(x):
    return x.view(torch.int32)


def _top(x):
    """Shared biased exponents [blocks, 1] of nonnegative fp32 x [blocks, 256]."""
    return ((_bits(x.amax(1, keepdim=True)) + 0xFFFFF) >> 23).clamp_(1, 254)


def _codes(x, e, fields, noise):
    """Codes of fp32 x >= 0 under exponents e: the top bits of x moved so that
    E's exponent field is `fields`; `noise` (20 bits) is added below them."""
    y = _scaled(x.double(), fields - e).float()
    return ((_bits(y) + noise) >> 20).clamp_(0, 8 * fields + 7)


def _near(y, fields, e):
    """The noise that rounds to nearest, ties to even."""
    b = _bits(_scaled(y.double(), fields - e).float())
    return ((b >> 20) & 1) + 0x7FFFF


def _value(code, e, fields):
    return _scaled((code.int() << 20).view(torch.float32).double(), e - fields).float()


def _unpack(state8, scale8):
    s, e = state8.view(-1, 2, BLOCK), scale8.view(-1, 2).int()
    cm, em, ev = s[:, 0].int(), e[:, :1], e[:, 1:]
    m = _value(cm & 127, em, 15)
    return torch.where(cm > 127, -m, m), _value(s[:, 1], ev, 31)


def _pack(m, v, noise_m, noise_v, state8, scale8):
    a = m.abs()
    em, ev = _top(a), _top(v)
    cm = _codes(a, em, 15, _near(a, 15, em) if noise_m is None else noise_m)
    cv = _codes(v, ev, 31, _near(v, 31, ev) if noise_v is None else noise_v)
    cv = torch.where(v > 0, cv.clamp(min=1), cv)
    cm = torch.where(torch.signbit(m) & (cm > 0), cm + 128, cm)
    s, e = state8.view(-1, 2, BLOCK), scale8.view(-1, 2)
    s[:, 0], s[:, 1] = cm.to(torch.uint8), cv.to(torch.uint8)
    e[:, :1], e[:, 1:] = em.to(torch.uint8), ev.to(torch.uint8)


def _i32(x):
    x &= 0xFFFFFFFF
    return x - (1 << 32) if x >> 31 else x


def _fmix_host(x):
    x &= 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _key(seed):
    return (seed ^ _fmix_host(seed >> 32)) & 0xFFFFFFFF


def _noise(blocks, seed, device):
    """Two 20-bit noises [blocks, 256] (16 random bits, centred), from the
    32-bit finalizer of MurmurHash3 over place * 0x9E3779B1 + key."""
    x = torch.arange(blocks * BLOCK, device=device, dtype=torch.int32).view(-1, BLOCK)
    x = x.mul_(_i32(0x9E3779B1)).add_(_i32(_key(seed)))
    x ^= (x >> 16) & 0xFFFF
    x *= _i32(0x85EBCA6B)
    x ^= (x >> 13) & 0x7FFFF
    x *= _i32(0xC2B2AE35)
    x ^= (x >> 16) & 0xFFFF
    return ((x & 0xFFFF) << 4) + 8, (((x >> 16) & 0xFFFF) << 4) + 8


# ------------------------------------------------------------------- prepare
def _normal(n, sigma, g, dtype=torch.float32):
    out = torch.empty(n, dtype=dtype, device="cuda")
    for at in range(0, n, 1 << 28):
        k = min(1 << 28, n - at)
        out[at:at + k] = torch.randn(k, generator=g, device="cuda").mul_(sigma)
    return out


def _moments(n, g):
    """Moments as a run leaves them: blocks of unlike size, v above m^2."""
    m = _normal(n, 1e-4, g)
    for at in range(0, n, 1 << 28):
        part = m[at:at + (1 << 28)]
        part.mul_(torch.randn(part.numel(), generator=g, device="cuda").exp_())
    v = _normal(n, 1e-3, g).abs_().add_(1e-7)
    for at in range(0, n, 1 << 28):
        v[at:at + (1 << 28)].square_()
    return m, v


def _encode_into(m, v, state8, scale8):
    for at in range(0, m.numel() // BLOCK, 1 << 18):
        to = min(at + (1 << 18), m.numel() // BLOCK)
        _pack(m[at * BLOCK:to * BLOCK].view(-1, BLOCK), v[at * BLOCK:to * BLOCK].view(-1, BLOCK), None,
              None, state8[at * 512:to * 512], scale8[at * 2:to * 2])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case, "seed": seed}
    if case["op"] == "adamw":
        sizes = _sizes(case)
        align = case["align"]
        at, places = 0, []
        for n in sizes:
            places.append(at)
            at += _up(n, align)
        total = at
        grad = DTYPES[case["grad"]]
        s.update(sizes=sizes, places=places, total=total, step=case["step"],
                 group=[(0 if n > 4096 else 1) if case["groups"] == 2 else 0 for n in sizes],
                 grad=_normal(total, 1e-3 * case["loss_scale"], g, grad),
                 master=_normal(total, 0.02, g))
        s["param"] = None if case["param"] == "none" else s["master"].to(DTYPES[case["param"]])
        # what lies between tensors holds zeros and is not written
        hole = torch.ones(total, dtype=torch.bool, device="cuda") if align > 1 and total > sum(sizes) else None
        if hole is not None:
            for p, n in zip(places, sizes):
                hole[p:p + n] = False
            for name in ("grad", "master", "param"):
                if s[name] is not None:
                    s[name][hole] = 0
        if case["bits"] == 32:
            s["m"], s["v"] = _moments(total, g)
            if hole is not None:
                s["m"][hole] = 0
                s["v"][hole] = 0
        else:
            blocks = sum(_up(n, BLOCK) for n in sizes) // BLOCK
            m, v = _moments(blocks * BLOCK, g)
            b = 0
            for n in sizes:
                m[b + n:b + _up(n, BLOCK)] = 0
                v[b + n:b + _up(n, BLOCK)] = 0
                b += _up(n, BLOCK)
            s["state8"] = torch.zeros(blocks * 512, dtype=torch.uint8, device="cuda")
            s["scale8"] = torch.zeros(blocks * 2, dtype=torch.uint8, device="cuda")
            _encode_into(m, v, s["state8"], s["scale8"])
            del m, v
            for name in ("m", "v"):
                s[name] = torch.empty(blocks * BLOCK, dtype=torch.bfloat16, device="cuda")
        if own:
            s["set"] = _tensor_set(s)
    elif case["op"] == "state8":
        n = _up(case["n"], BLOCK)
        s["m"], s["v"] = _moments(n, g)
        s["m"][case["n"]:] = 0
        s["v"][case["n"]:] = 0
        s["state8"] = torch.zeros(n * 2, dtype=torch.uint8, device="cuda")
        s["scale8"] = torch.zeros(n // BLOCK * 2, dtype=torch.uint8, device="cuda")
        if case["way"] == "decode":
            _encode_into(s["m"], s["v"], s["state8"], s["scale8"])
        out = torch.bfloat16 if case["way"] == "both" else torch.float32
        s["mo"], s["vo"] = (torch.empty(case["n"], dtype=out, device="cuda") for _ in range(2))
    else:
        t, d, v, dt = case["tokens"], case["dim"], case["vocab"], DTYPES[case["dtype"]]
        s["x"] = _normal(t * d, 1.0, g, dt).view(t, d)
        # logits of spread about 3, as a trained head gives
        s["w"] = _normal(v * d, 3.0 / math.sqrt(d), g, dt).view(v, d)
        s["target"] = torch.randint(0, v, (t,), generator=g, device="cuda")
        if case["ignored"]:
            s["target"][torch.rand(t, generator=g, device="cuda") < case["ignored"]] = -100
        s["loss"], s["lse"] = (torch.empty(t, device="cuda") for _ in range(2))
        s["result"] = torch.zeros(32, dtype=torch.uint8, device="cuda")
        if case["op"] == "grad":
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        if own:
            import zero_sharded_optimizer_step_amd as Z
            s["workspace"] = torch.empty(Z.zero_xent_workspace_bytes(t, d, v), dtype=torch.uint8,
                                         device="cuda")
    return s


def _tensor_set(s):
    import zero_sharded_optimizer_step_amd as Z

    def cut(name):
        return None if s.get(name) is None else [s[name][p:p + n] for p, n in zip(s["places"], s["sizes"])]

    if s["case"]["bits"] == 32:
        return Z.TensorSet(master=cut("master"), grad=cut("grad"), exp_avg=cut("m"), exp_avg_sq=cut("v"),
                           param=cut("param"), group=s["group"])
    b, codes, scales = 0, [], []
    for n in s["sizes"]:
        k = _up(n, BLOCK) // BLOCK
        codes.append(s["state8"][b * 512:(b + k) * 512])
        scales.append(s["scale8"][b * 2:(b + k) * 2])
        b += k
    return Z.TensorSet(master=cut("master"), grad=cut("grad"), state8=codes, scale8=scales,
                       param=cut("param"), group=s["group"])


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        return (_own_adamw if own else _plain_adamw)(s)
    if op == "state8":
        return (_own_state8 if own else _plain_state8)(s)
    return (_own_xent if own else _plain_xent)(s)


def _own_adamw(s):
    import zero_sharded_optimizer_step_amd as Z
    c = s["case"]
    groups = [Z.AdamGroup(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY),
              Z.AdamGroup(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=0.0)][:c["groups"]]
    Z.zero_tensors_step(s["set"], groups, step=s["step"], loss_scale=c["loss_scale"],
                        max_grad_norm=c["max_norm"], seed=s["seed"])
    if c["bits"] == 8:
        Z.zero_state8_decode(s["state8"], s["scale8"], s["m"], s["v"])
    return _adamw_out(s, s["set"].result.view(torch.float32)[4:5], s["set"].result.view(torch.int32)[5:6])


def _own_state8(s):
    import zero_sharded_optimizer_step_amd as Z
    n = s["case"]["n"]
    if s["case"]["way"] == "both":
        Z.zero_state8_encode(s["m"], s["v"], s["state8"], s["scale8"], n=n)
    Z.zero_state8_decode(s["state8"], s["scale8"], s["mo"], s["vo"], n=n)
    return {"m": s["mo"], "v": s["vo"]}


def _own_xent(s):
    import zero_sharded_optimizer_step_amd as Z
    a = Z.XentArgs(x=s["x"], w=s["w"], target=s["target"], loss=s["loss"], lse=s["lse"],
                   result=s["result"], workspace=s["workspace"], dx=s.get("dx"), dw=s.get("dw"))
    Z.zero_xent_forward(a)
    out = {"loss": s["loss"], "lse": s["lse"], "mean": s["result"].view(torch.float32)[6:7]}
    if "dx" in s:
        Z.zero_xent_backward(a)
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def _adamw_out(s, coef, overflow):
    out = {"master": s["master"], "m": s["m"], "v": s["v"], "coef": coef, "overflow": overflow}
    if s["param"] is not None:
        out["param"] = s["param"]
    return out


# --------------------------------------------------------------- plain forms
def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _spread(s, values):
    """One value for all, or a value per element by its tensor's group."""
    if s["case"]["groups"] == 1:
        return values[0]
    per = torch.tensor([values[k] for k in s["group"]], dtype=torch.float32, device="cuda")
    ends = s["places"][1:] + [s["total"]]
    return per.repeat_interleave(torch.tensor(ends, device="cuda") - torch.tensor(s["places"], device="cuda"),
                                 output_size=s["total"])


def _padded(s):
    """Element of the flat buffers -> element of the blocks of 256, where the two differ."""
    if s["case"]["align"] == BLOCK:
        return None
    sizes = torch.tensor(s["sizes"], device="cuda")
    up = (sizes + BLOCK - 1) // BLOCK * BLOCK
    shift = (up.cumsum(0) - up) - (sizes.cumsum(0) - sizes)
    return torch.arange(s["total"], device="cuda") + shift.repeat_interleave(sizes, output_size=s["total"])


def _plain_adamw(s):
    c, t = s["case"], s["step"]
    g = s["grad"].float() * _f32(1.0 / c["loss_scale"])
    sumsq = g.double().square().sum()
    norm = sumsq.sqrt()
    coef = torch.where((c["max_norm"] / (norm + 1e-6) < 1) & (c["max_norm"] > 0), c["max_norm"] / (norm + 1e-6),
                       1.0).float()
    overflow = (~torch.isfinite(sumsq)).int().view(1)
    g *= coef
    decay = _spread(s, [_f32(1.0 - LR * DECAY), 1.0])
    step_size, inv = _f32(LR / (1.0 - BETA1 ** t)), _f32(1.0 / math.sqrt(1.0 - BETA2 ** t))
    b1, c1, b2, c2, eps = _f32(BETA1), _f32(1.0 - BETA1), _f32(BETA2), _f32(1.0 - BETA2), _f32(EPS)
    where = _padded(s) if c["bits"] == 8 else None
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m, v = (x.reshape(-1) for x in _unpack(s["state8"], s["scale8"]))
        if where is not None:
            m, v = m[where], v[where]
    m = b1 * m + c1 * g
    v = b2 * v + c2 * (g * g)
    s["master"].copy_(s["master"] * decay - step_size * (m / (v.sqrt() * inv + eps)))
    if s["param"] is not None:
        s["param"].copy_(s["master"])
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        if where is not None:
            full = torch.zeros(2, s["m"].numel(), device="cuda")
            full[0, where], full[1, where] = m, v
            m, v = full
        noise = _noise(s["scale8"].numel() // 2, s["seed"], "cuda")
        _pack(m.view(-1, BLOCK), v.view(-1, BLOCK), noise[0], noise[1], s["state8"], s["scale8"])
        m, v = _unpack(s["state8"], s["scale8"])
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    return _adamw_out(s, coef.view(1), overflow)


def _plain_state8(s):
    if s["case"]["way"] == "both":
        _pack(s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK), None, None, s["state8"], s["scale8"])
    m, v = _unpack(s["state8"], s["scale8"])
    n = s["case"]["n"]
    s["mo"].copy_(m.view(-1)[:n])
    s["vo"].copy_(v.view(-1)[:n])
    return {"m": s["mo"], "v": s["vo"]}


def _plain_xent(s):
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    p = (logits - top).exp_()
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    kept = target >= 0
    at = target.clamp(min=0).view(-1, 1)
    s["lse"].copy_(lse.view(-1))
    s["loss"].copy_(torch.where(kept, (lse - logits.gather(1, at)).view(-1), 0.0))
    count = kept.sum().clamp(min=1)
    out = {"loss": s["loss"], "lse": s["lse"], "mean": (s["loss"].double().sum() / count).float().view(1)}
    if "dx" in s:
        p /= total
        p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        p *= kept.view(-1, 1) / count
        s["dx"].copy_(p @ w)
        s["dw"].copy_(p.t() @ x)
        out.update(dx=s["dx"], dw=s["dw"])
    return out


# ------------------------------------------------------ the definition, 64 bits
def _exact_round(x, top, low, noise):
    """x >= 0 (fp64, [blocks, 256]) on the grid of 8 steps per power of two
    that ends at 2^top * 1.875 (top: [blocks, 1]) and is even below 2^low;
    noise in [0, 1) of a step rounds down or up, None to nearest even."""
    e = torch.maximum(torch.frexp(x).exponent.to(torch.int64) - 1, low.expand_as(x))
    t = _scaled(x, 3 - e)
    t = torch.round(t) if noise is None else torch.floor(t + noise)
    return torch.minimum(_scaled(t, e - 3), _scaled(torch.full_like(x, 1.875), top))


def _exact_state(m, v, noise_m, noise_v):
    """fp64 moments as the 8-bit state holds them."""
    out = []
    for x, fields, noise in ((m.abs(), 15, noise_m), (v, 31, noise_v)):
        big = x.amax(1, keepdim=True)
        f, e = torch.frexp(big)
        top = (e.to(torch.int64) - 1 + (f > 0.9375)).clamp(-126, 127)
        low = top - fields + 1
        y = _exact_round(x, top, low, noise)
        if fields == 31:
            y = torch.where(x > 0, torch.maximum(y, _scaled(torch.ones_like(big), low - 3)), y)
        out.append(y)
    return torch.copysign(out[0], m), out[1]


def _exact_noise(first, blocks, seed):
    x = torch.arange(first * BLOCK, (first + blocks) * BLOCK, device="cuda", dtype=torch.int64)
    x = (x * 0x9E3779B1 + _key(seed)) & 0xFFFFFFFF
    for shift, factor in ((16, 0x85EBCA6B), (13, 0xC2B2AE35), (16, 1)):
        x = ((x ^ (x >> shift)) * factor) & 0xFFFFFFFF
    x = x.view(-1, BLOCK)
    return [((y * 16 + 8).double() / (1 << 20)) for y in (x & 0xFFFF, x >> 16)]


def _exact_moments(s):
    """The state's moments in fp64, [blocks, 256]; by the bits of the codes."""
    c = s["state8"].view(-1, 2, BLOCK).to(torch.int64)
    e = s["scale8"].view(-1, 2, 1).to(torch.int64) - 127
    out = []
    for k, fields in ((0, 15), (1, 31)):
        code = c[:, k] & 127 if k == 0 else c[:, k]
        field, frac = code >> 3, code & 7
        power = torch.clamp(field, min=1) - fields + e[:, k] - 3
        x = _scaled((frac + torch.where(field > 0, 8, 0)).double(), power)
        out.append(torch.where(c[:, k] > 127, -x, x) if k == 0 else x)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "state8":
        n, ms, vs = case["n"], [], []
        for at in range(0, s["scale8"].numel() // 2, 1 << 19):
            part = slice(at * BLOCK, (at + (1 << 19)) * BLOCK)
            if case["way"] == "both":
                m, v = _exact_state(s["m"][part].view(-1, BLOCK).double(), s["v"][part].view(-1, BLOCK).double(), None, None)
            else:
                m, v = _exact_moments({"state8": s["state8"][at * 512:(at + (1 << 19)) * 512],
                                       "scale8": s["scale8"][at * 2:(at + (1 << 19)) * 2]})
            ms.append(m.view(-1))
            vs.append(v.view(-1))
        return {"m": torch.cat(ms)[:n], "v": torch.cat(vs)[:n]}
    if case["op"] == "adamw":
        return _exact_adamw(s)
    x, w, target = s["x"].double(), s["w"].double(), s["target"]
    logits = x @ w.t()
    lse = torch.logsumexp(logits, 1)
    kept = target >= 0
    at = target.clamp(min=0)
    loss = torch.where(kept, lse - logits[torch.arange(len(at), device="cuda"), at], 0.0)
    count = max(1, int(kept.sum()))
    out = {"loss": loss, "lse": lse, "mean": (loss.sum() / count).view(1)}
    if case["op"] == "grad":
        logits.sub_(lse.view(-1, 1)).exp_()
        logits[torch.arange(len(at), device="cuda"), at] -= 1.0
        logits[~kept] = 0.0
        out.update(dx=logits @ w / count, dw=logits.t() @ x / count)
    return out


def _exact_adamw(s):
    c, t = s["case"], s["step"]
    sumsq = 0.0
    for at in range(0, s["total"], 1 << 28):
        sumsq += float((s["grad"][at:at + (1 << 28)].double() / c["loss_scale"]).square().sum())
    coef = c["max_norm"] / (math.sqrt(sumsq) + 1e-6) if c["max_norm"] > 0 else 1.0
    coef = min(coef, 1.0)
    eight = c["bits"] == 8
    out = {"master": s["master"].double(), "coef": torch.tensor([coef], dtype=torch.float64),
           "overflow": None, "m": None, "v": None}
    if eight:
        m_all, v_all = [], []
    else:
        out["m"], out["v"] = s["m"].double(), s["v"].double()
    first = 0
    for p, n, k in zip(s["places"], s["sizes"], s["group"]):
        blocks = _up(n, BLOCK) // BLOCK
        for b in range(0, blocks, 1 << 19):
            nb = min(1 << 19, blocks - b)
            lo, hi = b * BLOCK, min((b + nb) * BLOCK, n)
            g = s["grad"][p + lo:p + hi].double() / c["loss_scale"] * coef
            if eight:
                at = first + b
                m, v = _exact_moments({"state8": s["state8"][at * 512:(at + nb) * 512],
                                       "scale8": s["scale8"][at * 2:(at + nb) * 2]})
                m, v = m.view(-1)[:hi - lo], v.view(-1)[:hi - lo]
            else:
                m, v = out["m"][p + lo:p + hi], out["v"][p + lo:p + hi]
            m = BETA1 * m + (1 - BETA1) * g
            v = BETA2 * v + (1 - BETA2) * g * g
            w = out["master"][p + lo:p + hi]
            w.mul_(1 - LR * (DECAY if k == 0 else 0.0))
            w.sub_(LR / (1 - BETA1 ** t) * m / ((v / (1 - BETA2 ** t)).sqrt() + EPS))
            if eight:
                full = torch.zeros(2, nb * BLOCK, dtype=torch.float64, device="cuda")
                full[0, :hi - lo], full[1, :hi - lo] = m, v
                m, v = _exact_state(full[0].view(-1, BLOCK), full[1].view(-1, BLOCK), *_exact_noise(first + b, nb, s["seed"]))
                m_all.append(m.view(-1).to(torch.bfloat16))   # every value of the format is a bf16 value
                v_all.append(v.view(-1).to(torch.bfloat16))
            else:
                out["m"][p + lo:p + hi], out["v"][p + lo:p + hi] = m, v
        first += blocks
    if eight:
        out["m"], out["v"] = torch.cat(m_all), torch.cat(v_all)
    if s["param"] is not None:
        out["param"] = out["master"]
    return out
