"""What the 8-bit training operators are measured on: rows of activations held
in 8 bits, the gated activation that leaves its checkpoint so and takes its
gradient from it, and the product of 8-bit rows with 8-bit weights with its
gradient.

Rows of 8-bit codes.  A row (a token of an activation, an output channel of a
weight) is held as whole numbers q of [-127, 127] and a scale s: it stands for
q s.  s is the power of two 2^e with the smallest e under which the row's
largest magnitude rounds to 127 or less, e clamped to what the row's type
holds every q s of: [-24, 9] for fp16, [-126, 121] for bf16 and fp32; q is
row / s to nearest even, clamped.  A row of codes is padded with zeros to a
multiple of 16 bytes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RANGE = {torch.float16: (-24, 9), torch.bfloat16: (-126, 121), torch.float32: (-126, 121)}


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # a few short rows of a tiny fp16 model held and read back: latency counts
        dict(name="rows8 64 x 512 fp16", op="rows8", rows=64, dim=512, dtype="fp16", gap=0),
        # one layer's input of a long batch at d_model 4096, held and read back
        dict(name="rows8 16384 x 4096 bf16", op="rows8", rows=16384, dim=4096, dtype="bf16", gap=0),
        # fp32 rows off every boundary, each a view into a wider buffer
        dict(name="rows8 odd fp32", op="rows8", rows=2047, dim=10007, dtype="fp32", gap=3),
        # a short ragged batch through a small gated layer, there and back
        dict(name="glu8 odd fp16", op="glu8", tokens=37, width=1001, kind="gelu", gated=True,
             dtype="fp16", out8=True),
        # the ungated activation of an encoder layer at d_model 4096: its output goes on in 16 bits
        dict(name="glu8 4096 x 16384 gelu bf16", op="glu8", tokens=4096, width=16384, kind="gelu",
             gated=False, dtype="bf16", out8=False),
        # the gated activation of a large layer between two 8-bit products
        dict(name="glu8 8192 x 16384 silu bf16", op="glu8", tokens=8192, width=16384, kind="silu",
             gated=True, dtype="bf16", out8=True),
        # scoring one token: the weights are read once
        dict(name="linear8 one token bf16", op="linear8", tokens=1, dim=4096, out=16384,
             dtype="bf16", bias=False),
        # a small batch through one projection with its bias
        dict(name="linear8 48 tokens fp16", op="linear8", tokens=48, dim=4096, out=4096,
             dtype="fp16", bias=True),
        # an odd batch, nothing a multiple of anything
        dict(name="linear8 odd fp16", op="linear8", tokens=509, dim=1000, out=10007, dtype="fp16",
             bias=True),
        # a full batch through the wide projection of a layer
        dict(name="linear8 8192 tokens bf16", op="linear8", tokens=8192, dim=4096, out=16384,
             dtype="bf16", bias=False),
        # the gradient of an odd batch
        dict(name="linear8 grad odd fp16", op="grad8", tokens=509, dim=1000, out=2053, dtype="fp16",
             bias=True),
        # the gradient of that projection's full batch
        dict(name="linear8 grad 8192 tokens bf16", op="grad8", tokens=8192, dim=4096, out=16384,
             dtype="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["rows8", "glu8", "linear8", "linear8", "grad8", "grad8"])
    if op == "rows8":
        rows = _log(rng, 1, 16384)
        return dict(op=op, rows=rows, dim=_log(rng, 1, min(65536, 16384 * 4096 // rows)),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), gap=rng.choice([0, 0, 1, 8]))
    if op == "glu8":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, width=_log(rng, 16, 16384), kind=rng.choice(["silu", "gelu"]),
                    gated=rng.random() < 0.7, dtype=rng.choice(["bf16", "fp16"]), out8=rng.random() < 0.5)
    dim, out = _log(rng, 16, 16384), _log(rng, 16, 16384)
    if rng.random() < 0.5:
        dim, out = max(16, dim // 16 * 16), max(16, out // 16 * 16)
    tokens = _log(rng, 1, min(16384, 8192 * 4096 * 16384 // (dim * out)))
    return dict(op=op, tokens=tokens, dim=dim, out=out, dtype=rng.choice(["bf16", "fp16"]),
                bias=rng.random() < 0.5)


def work(case):
    two = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rows8":
        n, r = case["rows"] * case["dim"], case["rows"]
        return {"bytes": n * (two + 1 + 1 + two) + 8 * r, "flops": 4 * n}
    if case["op"] == "glu8":
        n, t, parts = case["tokens"] * case["width"], case["tokens"], 2 if case["gated"] else 1
        # there: the parts read and held, the result as 8 bits (read back) or as 16
        there = parts * (two + 1) + (1 + 1 + two if case["out8"] else two)
        back = two + parts + parts * two
        return {"bytes": n * (there + back) + 8 * t * (parts + 1), "flops": 40 * n}
    t, k, n = case["tokens"], case["dim"], case["out"]
    if case["op"] == "linear8":
        return {"bytes": t * k + n * k + two * t * n + 4 * (t + n), "flops": 2 * t * k * n}
    return {"bytes": (1 + two) * (t * k + n * k) + two * t * n + 4 * (t + n), "flops": 4 * t * k * n}


# ------------------------------------------------------------- rows in 8 bits
def _scales(x):
    """fp32 scales [rows, 1] of rows x of a 16- or 32-bit type."""
    top = x.abs().amax(1, keepdim=True).float()
    bits = top.view(torch.int32)
    # 2^p 1.f: p - 6, one more from 127.5 / 64 on (it would round to 128)
    e = ((bits + 0x10000) >> 23) - 127 - 6
    lo, hi = RANGE[x.dtype]
    return torch.where(top > 0, e, lo).clamp_(lo, hi).add_(127).clamp_(min=1).bitwise_left_shift_(23).view(torch.float32)


def _codes(x, s):
    # 1 / s and the product are exact, s being a power of two
    return (x.float() * (1.0 / s)).round_().clamp_(-127, 127)


def _values(x):
    """x as its rows in 8 bits stand for it, fp32."""
    s = _scales(x)
    return _codes(x, s).mul_(s)


def _up16(n):
    return (n + 15) // 16 * 16


def _hold(x):
    """(codes int8 [rows, dim up to 16], scales fp32 [rows]) of rows x."""
    s = _scales(x)
    q = torch.zeros(x.shape[0], _up16(x.shape[1]), dtype=torch.int8, device="cuda")
    q[:, :x.shape[1]] = _codes(x, s)
    return q, s.view(-1)


# ------------------------------------------------------------------- prepare
def _rand(rows, dim, sigma, g, dtype):
    x = torch.empty(rows, dim, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // dim)
    for at in range(0, rows, step):
        k = min(step, rows - at)
        x[at:at + k] = torch.randn(k, dim, generator=g, device="cuda").mul_(sigma)
    return x


def _activations(rows, dim, g, dtype):
    """Tokens of unlike size and a channel in 64 that is eight times the others."""
    x = _rand(rows, dim, 1.0, g, dtype)
    x *= torch.randn(rows, 1, generator=g, device="cuda").mul_(0.5).exp_().to(dtype)
    x[:, torch.rand(dim, generator=g, device="cuda") < 1.0 / 64] *= 8
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "dtype": dt}
    if case["op"] == "rows8":
        r, d = case["rows"], case["dim"]
        s["x"] = _activations(r, d + case["gap"], g, dt)[:, :d]
        s["codes"] = torch.empty(r, _up16(d), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(r, device="cuda")
        s["y"] = torch.empty(r, d, dtype=dt, device="cuda")
    elif case["op"] == "glu8":
        t, f = case["tokens"], case["width"]
        # gate and up are the halves of one product's output
        both = _rand(t, 2 * f if case["gated"] else f, 1.0, g, dt)
        s["gate"], s["up"] = both[:, :f], both[:, f:] if case["gated"] else None
        s["dh"] = _rand(t, f, 1e-2, g, dt)
        grads = torch.empty_like(both)
        s["dgate"], s["dup"] = grads[:, :f], grads[:, f:] if case["gated"] else None
        s["h"] = torch.empty(t, f, dtype=dt, device="cuda")
        if own:
            s["args"] = _glu_args(s)
    else:
        t, k, n = case["tokens"], case["dim"], case["out"]
        s["x8"], s["x_scale"] = _hold(_activations(t, k, g, dt))
        s["w8"], s["w_scale"] = _hold(_rand(n, k, 1.0 / math.sqrt(k), g, dt))
        s["bias"] = _rand(1, n, 0.1, g, dt).view(-1) if case["bias"] else None
        if case["op"] == "linear8":
            s["y"] = torch.empty(t, n, dtype=dt, device="cuda")
        else:
            s["dy"] = _rand(t, n, 1e-2, g, dt)
            s["dx"] = torch.empty(t, k, dtype=dt, device="cuda")
            s["dw"] = torch.empty(n, k, dtype=dt, device="cuda")
            s["db"] = torch.empty(n, dtype=dt, device="cuda") if case["bias"] else None
        if own:
            s["args"] = _linear_args(s)
    return s


def _glu_args(s):
    import zero_sharded_optimizer_step_amd as Z
    t, f = s["gate"].shape

    def rows():
        return (torch.empty(t, Z.rows8_stride(f), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda"))

    gate8, gate_scale = rows()
    up8, up_scale = rows() if s["case"]["gated"] else (None, None)
    h8, h_scale = rows() if s["case"]["out8"] else (None, None)
    return Z.Glu8Args(kind=s["case"]["kind"], gate=s["gate"], up=s["up"], gate8=gate8, gate_scale=gate_scale, up8=up8,
                      up_scale=up_scale, h=None if s["case"]["out8"] else s["h"], h8=h8, h_scale=h_scale,
                      dh=s["dh"], dgate=s["dgate"], dup=s["dup"])


def _linear_args(s):
    import zero_sharded_optimizer_step_amd as Z
    c = s["case"]
    room = torch.empty(Z.zero_linear8_workspace_bytes(c["tokens"], c["dim"], c["out"]), dtype=torch.uint8, device="cuda")
    return Z.Linear8Args(x8=s["x8"], x_scale=s["x_scale"], w8=s["w8"], w_scale=s["w_scale"], dim=c["dim"],
                         workspace=room, bias=s["bias"], y=s.get("y"), dy=s.get("dy"), dx=s.get("dx"),
                         dw=s.get("dw"), db=s.get("db"))


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op == "rows8":
        return (_own_rows if own else _plain_rows)(s)
    if op == "glu8":
        return (_own_glu if own else _plain_glu)(s)
    return (_own_linear if own else _plain_linear)(s)


def _own_rows(s):
    import zero_sharded_optimizer_step_amd as Z
    Z.zero_rows8_encode(s["x"], s["codes"], s["scale"])
    Z.zero_rows8_decode(s["codes"], s["scale"], s["y"])
    return {"y": s["y"], "scale": s["scale"]}


def _own_glu(s):
    import zero_sharded_optimizer_step_amd as Z
    Z.zero_glu8_forward(s["args"])
    if s["case"]["out8"]:
        Z.zero_rows8_decode(s["args"].h8, s["args"].h_scale, s["h"])
    Z.zero_glu8_backward(s["args"])
    return _glu_out(s)


def _own_linear(s):
    import zero_sharded_optimizer_step_amd as Z
    if s["case"]["op"] == "linear8":
        Z.zero_linear8_forward(s["args"])
        return {"y": s["y"]}
    Z.zero_linear8_backward(s["args"])
    return _grad_out(s)


def _glu_out(s):
    out = {"h": s["h"], "dgate": s["dgate"]}
    if s["up"] is not None:
        out["dup"] = s["dup"]
    return out


def _grad_out(s):
    out = {"dx": s["dx"], "dw": s["dw"]}
    if s["db"] is not None:
        out["db"] = s["db"]
    return out


# --------------------------------------------------------------- plain forms
GELU_K, GELU_C = math.sqrt(8.0 / math.pi), 0.044715


def _plain_rows(s):
    scale = _scales(s["x"])
    s["scale"].copy_(scale.view(-1))
    s["y"].copy_(_codes(s["x"], scale).mul_(scale))
    return {"y": s["y"], "scale": s["scale"]}


def _act(x, kind):
    """The activation of fp32 x and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    # gelu with the tanh in its sigmoid form
    p = 1.0 / (1.0 + torch.exp(-GELU_K * (x + GELU_C * x * x * x)))
    return x * p, p + x * p * (1.0 - p) * (GELU_K * (1.0 + 3.0 * GELU_C * x * x))


def _plain_glu(s):
    kind, gate, up, dh = s["case"]["kind"], s["gate"], s["up"], s["dh"].float()
    h = _act(gate.float(), kind)[0]
    if up is not None:
        h *= up.float()
    h = h.to(s["dtype"])
    s["h"].copy_(_values(h) if s["case"]["out8"] else h)
    a, da = _act(_values(gate), kind)
    if up is None:
        s["dgate"].copy_(dh * da)
    else:
        s["dgate"].copy_(dh * _values(up) * da)
        s["dup"].copy_(dh * a)
    return _glu_out(s)


def _plain_linear(s):
    k = s["case"]["dim"]
    x = s["x8"][:, :k].float() * s["x_scale"].view(-1, 1)
    w = s["w8"][:, :k].float() * s["w_scale"].view(-1, 1)
    if s["case"]["op"] == "linear8":
        y = x @ w.t()
        if s["bias"] is not None:
            y += s["bias"].float()
        s["y"].copy_(y)
        return {"y": s["y"]}
    dy = s["dy"].float()
    s["dx"].copy_(dy @ w)
    s["dw"].copy_(dy.t() @ x)
    if s["db"] is not None:
        s["db"].copy_(dy.sum(0))
    return _grad_out(s)


# ------------------------------------------------------ the definition, 64 bits
def _exact_rows(x):
    """(values, scales) in fp64 of rows x of their own type."""
    lo, hi = RANGE[x.dtype]
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    e = torch.frexp(top).exponent.double() - 7.0
    e = e + (torch.round(top * torch.exp2(-e)) > 127).double()
    scale = torch.exp2(torch.where(top > 0, e, torch.full_like(e, lo)).clamp(lo, hi))
    return torch.round(x / scale).clamp(-127, 127) * scale, scale.view(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows8":
        y, scale = _exact_rows(s["x"])
        return {"y": y, "scale": scale}
    if case["op"] == "glu8":
        return _exact_glu(s)
    k = case["dim"]
    x = s["x8"][:, :k].double() * s["x_scale"].double().view(-1, 1)
    w = s["w8"][:, :k].double() * s["w_scale"].double().view(-1, 1)
    if case["op"] == "linear8":
        y = torch.matmul(x, w.t())
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    dy = s["dy"].double()
    out = {"dx": torch.matmul(dy, w), "dw": torch.matmul(dy.t(), x)}
    if s["db"] is not None:
        out["db"] = dy.sum(0)
    return out


def _exact_glu(s):
    kind, dt, parts = s["case"]["kind"], s["dtype"], {"h": [], "dgate": [], "dup": []}

    def act(x):
        if kind == "silu":
            p = torch.sigmoid(x)
            return x * p, p + x * p * torch.sigmoid(-x)
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x**3))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x**2)

    for at in range(0, s["case"]["tokens"], 1024):
        rows = slice(at, at + 1024)
        gate, dh = s["gate"][rows], s["dh"][rows].double()
        h = act(gate.double())[0]
        up = None if s["up"] is None else s["up"][rows]
        h = (h if up is None else h * up.double())
        # held in 8 bits, it is the 16-bit result that is held
        parts["h"].append(_exact_rows(h.to(dt))[0] if s["case"]["out8"] else h)
        a, da = act(_exact_rows(gate)[0])
        if up is None:
            parts["dgate"].append(dh * da)
        else:
            parts["dgate"].append(dh * _exact_rows(up)[0] * da)
            parts["dup"].append(dh * a)
    return {name: torch.cat(p) for name, p in parts.items() if p}
