"""Plain definitions of the training operators (include/zero/train.h) for
their tests: AdamW and the 8-bit state in numpy, the cross entropy in torch
float64.  Nothing here uses the library."""
import numpy as np
import torch

BLOCK = 256


# ------------------------------------------------------------- the 8-bit state
def exponents(x):
    """Shared exponents of blocks [b, 256] of magnitudes (fp32), biased."""
    big = x.max(axis=1).astype(np.float64)
    f, e = np.frexp(big)                                  # big = f 2^e, f in [0.5, 1)
    e = np.where(big > 0, e - 1 + (f > 0.9375), -127)
    return np.clip(e + 127, 1, 254)


def codes(x, e, field, noise=None):
    """Codes of fp32 magnitudes x [b, 256] under exponents e [b]; noise in
    [0, 1) of a step, or None for nearest even."""
    y = np.ldexp(x.astype(np.float64), (field - e)[:, None]).astype(np.float32).astype(np.float64)
    _, k = np.frexp(y)
    k = np.maximum(k - 1, -126)                           # fp32's subnormals share a step
    steps = np.ldexp(y, 3 - k)                            # in [8, 16), below 8 when subnormal
    n = np.rint(steps) if noise is None else np.floor(steps + noise)
    up = n >= 16
    k, n = np.where(up, k + 1, k), np.where(up, 8, n)
    c = np.where(n < 8, n, (k + 127) * 8 + n - 8)
    return np.clip(c, 0, 8 * field + 7).astype(np.int64)


def values(c, e, field):
    """What codes stand for, fp32."""
    c = c.astype(np.int64)
    k = np.maximum(c >> 3, 1)
    n = (c & 7) + np.where(c >> 3 > 0, 8, 0)
    return np.ldexp(n.astype(np.float64), k - field + e[:, None] - 127 - 3).astype(np.float32)


def _blocks(x):
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def encode(m, v, noise=(None, None)):
    """(state8, scale8) of fp32 moments of any length."""
    m, v = _blocks(m), _blocks(v)
    em, ev = exponents(np.abs(m)), exponents(v)
    cm = codes(np.abs(m), em, 15, noise[0])
    cv = codes(v, ev, 31, noise[1])
    cv = np.where((v > 0) & (cv == 0), 1, cv)
    cm = np.where(np.signbit(m) & (cm > 0), cm + 128, cm)
    return (np.stack([cm, cv], 1).astype(np.uint8).reshape(-1),
            np.stack([em, ev], 1).astype(np.uint8).reshape(-1))


def decode(state8, scale8, n):
    s = state8.reshape(-1, 2, BLOCK)
    e = scale8.reshape(-1, 2).astype(np.int64)
    m = values(s[:, 0] & 127, e[:, 0], 15)
    m = np.where(s[:, 0] > 127, -m, m)
    return m.reshape(-1)[:n], values(s[:, 1], e[:, 1], 31).reshape(-1)[:n]


def _fmix(x):
    x = x.astype(np.uint64)
    for shift, factor in ((16, 0x85EBCA6B), (13, 0xC2B2AE35), (16, 1)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x


def noises(first_block, n_blocks, seed):
    """The two noises of every element of the blocks, in steps."""
    key = (seed & 0xFFFFFFFF) ^ int(_fmix(np.array([(seed >> 32) & 0xFFFFFFFF], dtype=np.uint64))[0])
    place = np.arange(first_block * BLOCK, (first_block + n_blocks) * BLOCK, dtype=np.uint64)
    h = _fmix((place * np.uint64(0x9E3779B1) + np.uint64(key)) & np.uint64(0xFFFFFFFF)).reshape(-1, BLOCK)
    to = [((x * np.uint64(16) + np.uint64(8)).astype(np.float64) / 2**20)
          for x in (h & np.uint64(0xFFFF), h >> np.uint64(16))]
    return to


# ------------------------------------------------------------------------ AdamW
def adamw(g, p, m, v, lr, b1, b2, eps, wd, t):
    """One update in fp32, one rounding per operation, of arrays (g already
    unscaled and clipped)."""
    f = np.float32
    with np.errstate(over="ignore"):
        m = f(b1) * m + f(1 - b1) * g
        v = f(b2) * v + f(1 - b2) * (g * g)
        d = np.sqrt(v) * f(1 / np.sqrt(1 - b2**t)) + f(eps)
        p = p * f(1 - lr * wd) - f(lr / (1 - b1**t)) * (m / d)
    return p, m, v


# ---------------------------------------------------------------- cross entropy
def xent(x, w, target, grad_scale=1.0):
    """The definition in fp64 (inputs of any dtype, on the CPU): a dict of
    outputs and of what the error bounds need."""
    x, w = x.double(), w.double()
    logits = x @ w.t()
    lse = torch.logsumexp(logits, 1)
    kept = (target >= 0) & (target < w.shape[0])
    at = torch.where(kept, target, torch.zeros_like(target))
    rows = torch.arange(len(at))
    loss = torch.where(kept, lse - logits[rows, at], torch.zeros_like(lse))
    count = max(1, int(kept.sum()))
    soft = (logits - lse[:, None]).exp() * kept[:, None]
    p = soft.clone()
    p[rows, at] -= kept.double()
    c = grad_scale / count
    return {"loss": loss, "lse": lse, "sum": loss.sum(), "count": int(kept.sum()), "mean": loss.sum() / count,
            "dx": c * (p @ w), "dw": c * (p.t() @ x), "p": p, "soft": soft, "kept": kept,
            "at": at, "c": c, "size": x.abs() @ w.abs().t()}


def xent_bounds(r, x, w, dtype):
    """How far the kernels' outputs may be from xent()'s.

    A logit: exact products, dim sums in fp32, each off by at most 2^-23 of
    the sum of magnitudes (2^-24 if rounded to nearest, twice that where the
    matrix core truncates).  An exponential: 2^-20 relative (its argument's
    rounding, the hardware's exp and the sums).  P: half a step of the
    16-bit type, u, plus what the logit's error makes of it; the products
    with P: vocab or tokens fp32 sums; the result: another half step."""
    u = torch.finfo(dtype).eps / 2
    x, w = x.double().abs(), w.double().abs()
    e_row = (x.shape[1] * 2.0**-23 * r["size"]).amax(1)          # of a row's logits
    lse = e_row + 2.0**-20 + 2.0**-22 * r["lse"].abs()
    loss = 2 * e_row + 2.0**-20 + 2.0**-22 * (r["lse"].abs() + (r["lse"] - r["loss"]).abs())
    # of P, before the count's factor: fp16's P is held times 2^15, its
    # smallest step 2^-24
    flush = 2.0**-25 / 2**15 if dtype == torch.float16 else 2.0**-134
    dp = r["p"].abs() * u + r["soft"] * (2 * e_row + 2.0**-19)[:, None] + flush * r["kept"].double()[:, None]
    rows = torch.arange(len(r["at"]))
    dp[rows, r["at"]] += 2.0**-23 * r["kept"]
    c = abs(r["c"])
    tiny = 2.0**-25 if dtype == torch.float16 else 2.0**-134     # half the smallest step
    ap = r["p"].abs()
    dx = c * (dp @ w + w.shape[0] * 2.0**-23 * (ap @ w)) * (1 + u) + u * r["dx"].abs() + tiny
    dw = c * (dp.t() @ x + x.shape[0] * 2.0**-23 * (ap.t() @ x)) * (1 + u) + u * r["dw"].abs() + tiny
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
