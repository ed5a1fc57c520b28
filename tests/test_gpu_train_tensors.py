"""AdamW over tensor lists and the 8-bit state on the GPU, against the numpy
definitions of train_ref: codes and exponents are equal, fp32 values are
equal where the arithmetic is one rounding per operation."""
import numpy as np
import pytest
import torch

import train_ref as R
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu


def say(msg):
    print(msg, flush=True)


def moments(n, seed, scale=1.0):
    r = np.random.default_rng(seed)
    m = (r.standard_normal(n) * np.exp(3 * r.standard_normal(n)) * 1e-4 * scale).astype(np.float32)
    v = ((r.standard_normal(n) * np.exp(3 * r.standard_normal(n)) * 1e-3 * scale) ** 2).astype(np.float32)
    return m, v


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def encode_gpu(m, v):
    k = Z.state8_blocks(len(m))
    s8 = torch.full((512 * k + 16,), 77, dtype=torch.uint8, device="cuda")
    e8 = torch.full((2 * k + 2,), 77, dtype=torch.uint8, device="cuda")
    Z.zero_state8_encode(gpu(m), gpu(v), s8, e8, n=len(m))
    assert bool((s8[512 * k:] == 77).all()) and bool((e8[2 * k:] == 77).all())
    return s8[:512 * k].cpu().numpy(), e8[:2 * k].cpu().numpy()


@pytest.mark.parametrize("n", [1, 3, 255, 256, 257, 1024, 5003])
@pytest.mark.parametrize("scale", [1.0, 1e-30, 1e15])
def test_state8_encode_decode(n, scale):
    say("state8 n=%d scale=%g" % (n, scale))
    m, v = moments(n, n, scale)
    s8, e8 = encode_gpu(m, v)
    rs, re = R.encode(m, v)
    assert np.array_equal(e8, re)
    assert np.array_equal(s8, rs)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        out = [torch.full((n + 8,), -3.0, dtype=dtype, device="cuda") for _ in range(2)]
        Z.zero_state8_decode(gpu(s8), gpu(e8), out[0], out[1], n=n)
        for got, want in zip(out, R.decode(rs, re, n)):
            assert torch.equal(got[:n].cpu(), torch.from_numpy(want).to(dtype))
            assert bool((got[n:] == -3.0).all())


def test_state8_edges():
    # zeros; one value alone; the 1.875 edge; subnormals; the top; infinities
    f = np.float32
    big = np.finfo(f).max
    blocks = [np.zeros(256, f), np.r_[f(1), np.zeros(255, f)], np.full(256, 1.875, f),
              np.full(256, np.nextafter(f(1.875), f(2)), f), np.full(256, 1e-45, f),
              np.r_[f(1e-38), np.full(255, 1e-44, f)], np.full(256, big, f),
              np.r_[f(np.inf), np.full(255, 1, f)], np.geomspace(1e-12, 1, 256).astype(f)]
    m = np.concatenate([b * np.where(np.arange(256) % 2, -1, 1).astype(f) for b in blocks])
    v = np.concatenate(blocks)
    finite = np.where(np.isfinite(v), v, big)
    s8, e8 = encode_gpu(m, v)
    rs, re = R.encode(np.where(np.isfinite(m), m, np.sign(m) * big).astype(f), finite)
    assert np.array_equal(e8, re) and np.array_equal(s8, rs)
    # no positive second moment is held as zero, no zero as positive
    cv = s8.reshape(-1, 2, 256)[:, 1].reshape(-1)
    assert np.array_equal(cv > 0, v > 0)


class List:
    """A list of tensors carved out of flat buffers at `align` elements."""

    def __init__(self, sizes, bits, grad=torch.bfloat16, param=torch.bfloat16, align=1, groups=1, seed=0,
                 loss_scale=1.0, grad_sigma=1e-3):
        r = np.random.default_rng(seed)
        self.sizes, self.bits, self.groups = sizes, bits, groups
        self.group = [t % groups for t in range(len(sizes))]
        at, self.places = 3 if align == 1 else 0, []
        for n in sizes:
            self.places.append(at)
            at += -(-n // align) * align
        total = at + 5
        self.flat = {"grad": gpu((r.standard_normal(total) * grad_sigma * loss_scale).astype(np.float32)).to(grad),
                     "master": gpu((r.standard_normal(total) * 0.02).astype(np.float32)),
                     "param": None if param is None else torch.full((total,), 9.0, dtype=param, device="cuda")}
        ms = [moments(n, 10 * seed + t, 1.0) for t, n in enumerate(sizes)]
        if bits == 32:
            for k, name in enumerate(("m", "v")):
                self.flat[name] = torch.full((total,), 9.0, device="cuda")
                for p, n, x in zip(self.places, sizes, ms):
                    self.flat[name][p:p + n] = gpu(x[k])
        else:
            enc = [R.encode(*x) for x in ms]
            self.s8 = [gpu(e[0]) for e in enc]
            self.e8 = [gpu(e[1]) for e in enc]

    def cut(self, name):
        f = self.flat[name]
        return None if f is None else [f[p:p + n] for p, n in zip(self.places, self.sizes)]

    def set(self):
        state = dict(exp_avg=self.cut("m"), exp_avg_sq=self.cut("v")) if self.bits == 32 else \
            dict(state8=self.s8, scale8=self.e8)
        return Z.TensorSet(master=self.cut("master"), grad=self.cut("grad"), param=self.cut("param"),
                           group=self.group, **state)

    def expected(self, groups, t, coef, inv_scale, seed):
        """Per tensor (master, m or codes, v or exponents) after a step."""
        out, block = [], 0
        f = np.float32
        for i, n in enumerate(self.sizes):
            p = self.cut("master")[i].cpu().numpy()
            g = self.cut("grad")[i].float().cpu().numpy() * f(inv_scale) * f(coef)
            if self.bits == 32:
                m, v = (self.cut(k)[i].cpu().numpy() for k in ("m", "v"))
            else:
                m, v = R.decode(self.s8[i].cpu().numpy(), self.e8[i].cpu().numpy(), n)
            h = groups[self.group[i]]
            p, m, v = R.adamw(g, p, m, v, h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, t)
            if self.bits == 8:
                k = -(-n // 256)
                out.append((p,) + R.encode(m, v, R.noises(block, k, seed)))
                block += k
            else:
                out.append((p, m, v))
        return out


GROUPS = [Z.AdamGroup(lr=1e-3), Z.AdamGroup(lr=2e-4, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0)]
SIZES = [1, 700, 256, 1024, 0, 1025, 5000, 3]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("param", [torch.bfloat16, torch.float16, None], ids=["pbf16", "pfp16", "none"])
@pytest.mark.parametrize("align", [1, 256])
def test_step(bits, grad, param, align):
    say("list bits=%d grad=%s param=%s align=%d" % (bits, grad, param, align))
    q = List(SIZES, bits, grad, param, align, groups=2, seed=bits, loss_scale=64.0)
    before = {k: (None if v is None else v.clone()) for k, v in q.flat.items()}
    ts = q.set()
    sumsq = sum(float((x.double() * np.float32(1 / 64.0)).square().sum()) for x in q.cut("grad"))
    for step, max_norm in ((1, 0.0), (7, 0.01)):
        seed = (step << 40) + 12345
        coef = min(1.0, max_norm / (sumsq**0.5 + 1e-6)) if max_norm else 1.0
        info_want = q.expected(GROUPS, step, coef, 1 / 64.0, seed)
        info = Z.zero_tensors_step(ts, GROUPS, step=step, loss_scale=64.0, max_grad_norm=max_norm, seed=seed,
                                   want_info=True)
        assert info.overflow == 0 and info.clipped == (1 if coef < 1 else 0)
        # fp64 sums in another order
        assert abs(info.sumsq - sumsq) <= 1e-12 * sumsq and abs(info.coef - coef) <= 2.0**-23 * coef
        if info.coef != np.float32(coef):
            info_want = None                              # the clip factor rounded the other way
        for i, n in enumerate(q.sizes):
            if info_want is None or n == 0:
                continue
            p, a, b = info_want[i]
            assert np.array_equal(q.cut("master")[i].cpu().numpy(), p), i
            if bits == 32:
                assert np.array_equal(q.cut("m")[i].cpu().numpy(), a), i
                assert np.array_equal(q.cut("v")[i].cpu().numpy(), b), i
            else:
                assert np.array_equal(q.e8[i].cpu().numpy(), b), i
                assert np.array_equal(q.s8[i].cpu().numpy(), a), i
            if param is not None:
                assert torch.equal(q.cut("param")[i].cpu(), torch.from_numpy(p).to(param)), i
        assert info_want is not None or max_norm
    for name, old in before.items():                      # nothing outside the tensors
        if old is None:
            continue
        keep = torch.ones(len(old), dtype=torch.bool, device="cuda")
        for p, n in zip(q.places, q.sizes):
            keep[p:p + n] = False
        assert torch.equal(q.flat[name][keep], old[keep]), name


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_overflow_skips_the_step(bits, bad):
    q = List([300, 2000], bits)
    q.cut("grad")[1][1999] = bad
    keep = [t.clone() for t in (q.flat["master"], q.flat["param"])]
    state = [t.clone() for t in (q.s8 + q.e8 if bits == 8 else [q.flat["m"], q.flat["v"]])]
    info = Z.zero_tensors_step(q.set(), GROUPS, step=1, want_info=True)
    assert info.overflow == 1
    for a, b in zip(keep + state, [q.flat["master"], q.flat["param"]] +
                    (q.s8 + q.e8 if bits == 8 else [q.flat["m"], q.flat["v"]])):
        assert torch.equal(a, b)


def test_one_tensor_equals_the_shard_step():
    # the same arithmetic as zero_shard_step with one replica, bit for bit
    n = 4096 + 1024
    q = List([n], 32, align=256)
    st = [q.cut(k)[0].clone() for k in ("master", "m", "v")]
    full = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(Z.zero_shard_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    Z.zero_shard_step(Z.StepArgs(world_size=1, rank=0, shard_numel=n, valid_numel=n, replica_grads=q.cut("grad"),
                                 master=st[0], exp_avg=st[1], exp_avg_sq=st[2], full_params=full, workspace=ws,
                                 lr=1e-3, step=5, max_grad_norm=0.0))
    Z.zero_tensors_step(q.set(), GROUPS, step=5, max_grad_norm=0.0)
    for a, b in zip(st + [full], [q.cut("master")[0], q.cut("m")[0], q.cut("v")[0], q.cut("param")[0]]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_two_ranks_join_their_norms(bits):
    # two lists as two ranks: norm, combine, apply equals one list of both
    whole = List([5000, 300, 777], bits, seed=3)
    a, b = List([5000, 300, 777], bits, seed=3), None
    parts = []
    for lo, hi in ((0, 1), (1, 3)):
        state = dict(exp_avg=a.cut("m")[lo:hi], exp_avg_sq=a.cut("v")[lo:hi]) if bits == 32 else \
            dict(state8=a.s8[lo:hi], scale8=a.e8[lo:hi])
        parts.append(Z.TensorSet(master=a.cut("master")[lo:hi], grad=a.cut("grad")[lo:hi],
                                 param=a.cut("param")[lo:hi], **state))
    table = torch.empty(Z.zero_partials_bytes(2), dtype=torch.uint8, device="cuda")
    glob = torch.zeros(32, dtype=torch.uint8, device="cuda")
    for k, p in enumerate(parts):
        Z.zero_tensors_norm(p, GROUPS, 2, k, table)
    Z.zero_shard_combine(table, 2, 1e-3, glob)
    for p in parts:
        Z.zero_tensors_apply(p, GROUPS, 2, glob, seed=9)
    info = Z.zero_tensors_step(whole.set(), GROUPS, step=2, max_grad_norm=1e-3, seed=9, want_info=True)
    coef = glob.view(torch.float32)[4].item()
    assert abs(coef - info.coef) <= 2.0**-23 * coef
    if coef == info.coef:
        assert torch.equal(whole.flat["master"], a.flat["master"])
        assert torch.equal(whole.flat["param"], a.flat["param"])


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_with_device_scalars(bits):
    eager, graph = List(SIZES, bits, seed=4), List(SIZES, bits, seed=4)
    es, gs = eager.set(), graph.set()
    dev = torch.zeros(288, dtype=torch.uint8, device="cuda")

    def put(step):
        k = Z.zero_tensors_scalars(gs, GROUPS, step, seed=step * 7, loss_scale=2.0, max_grad_norm=1e-3)
        dev.copy_(torch.frombuffer(bytearray(bytes(k)), dtype=torch.uint8))
    put(1)
    warm = List([10], bits).set()
    Z.zero_tensors_step(warm, GROUPS, step=1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Z.zero_tensors_step(gs, GROUPS, step=1, scalars=dev)
    for step in (1, 2, 3):
        put(step)
        g.replay()
        _ = torch.ones(1000, device="cuda").sum().item()
        Z.zero_tensors_step(es, GROUPS, step=step, seed=step * 7, loss_scale=2.0, max_grad_norm=1e-3)
        for name in eager.flat:
            assert torch.equal(eager.flat[name], graph.flat[name]), (step, name)
        if bits == 8:
            assert all(torch.equal(x, y) for x, y in zip(eager.s8 + eager.e8, graph.s8 + graph.e8))
        assert torch.equal(es.result, gs.result)


def test_empty_list():
    ts = Z.TensorSet(master=[], grad=[], exp_avg=[], exp_avg_sq=[])
    info = Z.zero_tensors_step(ts, GROUPS, step=1, want_info=True)
    assert info.sumsq == 0.0 and info.overflow == 0 and info.coef == 1.0
