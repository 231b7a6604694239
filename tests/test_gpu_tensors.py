"""zs_adam_tensors on the GPU against the update in 64 bits.

Tolerances, with u = 2^-24 (one float32 rounding), from the operations in
their order (include/zs.h, zs_adam_tensors):
  dg = u (|grad coef| + 2 wd |p|)                       the gradient (wd: Adam-L2 only)
  dm = 4u (|b1 m| + |(1-b1) g|) + (1-b1) dg             2-3 products, a sum, 1-b1 rounded
  dr = 5u r + sqrt(1-b2) dg                             6u on the square, halved by the root, rounded
  dp = 4u (|p| + |update|) + lr/bc1 (dm + |m| (dr / sqrt(bc2) / den + 6u)) / den
A code rounded to nearest is within half a spacing of the value, plus dm or dr.
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests import lowbit_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, adamw=1, bias_correction=1)
KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GUARD = 64


class Buf:
    """n elements with guard bytes on both sides, `shift` elements past a 256-byte boundary."""

    def __init__(self, values, dtype, shift=0):
        t = torch.as_tensor(values).to(dtype)
        size = t.element_size()
        self.raw = torch.full(((t.numel() + 2 * GUARD + shift) * size,), 0xA5, dtype=torch.uint8, device="cuda")
        lo = (GUARD + shift) * size
        self.lo, self.hi = lo, lo + t.numel() * size
        self.t = self.raw[lo:self.hi].view(dtype)
        self.t.copy_(t)

    def guards_ok(self):
        return bool((self.raw[:self.lo] == 0xA5).all() and (self.raw[self.hi:] == 0xA5).all())


def rand_state(n, bits, rng, grad_kind, sigma=1e-3):
    g = rng.standard_normal(n) * sigma
    g[rng.random(n) < 0.05] = 0.0
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    m = (rng.standard_normal(n) * sigma * 0.3).astype(np.float32)
    r = np.abs(rng.standard_normal(n) * sigma).astype(np.float32)
    s = dict(grad=torch.from_numpy(g).to(KINDS[grad_kind]), p=p)
    if bits == 32:
        s.update(m=m, v=r * r)
        return s
    for name, x in (("m", m), ("r", r)):
        scale = ref.state_scales(x)
        y = torch.from_numpy(ref.blocks(x) / scale[:, None]).float().to(torch.float8_e4m3fn)
        s[name + "_code"] = y.view(torch.uint8).numpy().ravel()[:n].copy()
        s[name + "_scale"] = scale.astype(np.float32)
    return s


def held(code, scale):
    v = np.pad(ref.E4M3[code], (0, -len(code) % ref.BLOCK)).reshape(-1, ref.BLOCK)
    return (v * scale.astype(np.float64)[:, None]).ravel()[:len(code)]


def upload(items, bits, **kw):
    got = zs.zs_build_tensors(items, state_bits=bits, **kw)
    table = torch.empty(max(zs.zs_tensors_info(got)["device_table_bytes"], 16), dtype=torch.uint8, device="cuda")
    zs.zs_tensors_upload(got, table, table.numel())
    return got


def make(states, bits, grad_kind, param_kind, shift=0):
    bufs, items = [], []
    for s in states:
        n = len(s["p"])
        b = dict(grad=Buf(s["grad"], KINDS[grad_kind], shift), master=Buf(s["p"], torch.float32, shift))
        if param_kind:
            b["param"] = Buf(np.zeros(n), KINDS[param_kind], shift)
        if bits == 32:
            b["exp_avg"], b["exp_avg_sq"] = Buf(s["m"], torch.float32, shift), Buf(s["v"], torch.float32, shift)
        else:
            b["exp_avg"], b["exp_avg_sq"] = Buf(s["m_code"], torch.uint8, shift), Buf(s["r_code"], torch.uint8, shift)
            b["exp_avg_scale"], b["exp_avg_sq_scale"] = Buf(s["m_scale"], torch.float32), Buf(s["r_scale"], torch.float32)
        bufs.append(b)
        items.append({k: v.t for k, v in b.items()})
    return bufs, upload(items, bits)


def bounds(s, m0, v0, hp, step, coef):
    """64-bit results and how far the float32 ones may be."""
    f = lambda x: float(np.float32(x))  # noqa: E731
    lr, b1, b2, eps, wd = (f(hp[k]) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    g = s["grad"].double().numpy() * coef
    p, m, v = ref.adam64(s["p"], m0, v0, s["grad"].double().numpy(), hp, step, coef)
    l2 = 0.0 if hp["adamw"] else wd
    dg = U * (np.abs(g) + 2 * l2 * np.abs(s["p"]))
    dm = 4 * U * (np.abs(b1 * m0) + (1 - b1) * (np.abs(g) + l2 * np.abs(s["p"]))) + (1 - b1) * dg
    r = np.sqrt(v)
    dr = 5 * U * r + np.sqrt(1 - b2) * dg
    bc1, bc2 = (1 - b1 ** step, 1 - b2 ** step) if hp["bias_correction"] else (1.0, 1.0)
    den = r / np.sqrt(bc2) + eps
    upd = lr / bc1 * np.abs(m) / den
    dp = 4 * U * (np.abs(s["p"]) + upd) + lr / bc1 * (dm + np.abs(m) * (dr / np.sqrt(bc2) / den + 6 * U)) / den
    return p, m, r, dp, dm, dr


def check_param(b):
    """The 16-bit copy is the new master, rounded to nearest even: bit for bit."""
    want = b["master"].t.to(b["param"].t.dtype)
    assert torch.equal(b["param"].t.view(torch.int16), want.view(torch.int16))


def check_codes(code, scale, x, dx, random=None, least=False):
    want = ref.state_scales(x)
    # the largest value may lie within dx of a power of two
    edge = np.abs(np.log2(scale.astype(np.float64) / want))
    assert np.all((edge == 0) | ((edge == 1) & (ref.blocks(dx).max(1) > 0)))
    assert np.mean(edge == 0) > 0.99 or len(want) < 100 and np.all(edge == 0)
    s = np.repeat(scale.astype(np.float64), ref.BLOCK)[:len(x)]
    y, q, d = x / s, ref.E4M3[code], dx / s
    sp = ref.spacing(y)
    lifted = least & (x > 0) & (np.abs(y) < 2.0 ** -9)
    if least:
        assert np.all(code[x > 0] != 0)
    if random is None:
        assert np.all((np.abs(q - y) <= sp / 2 * (1 + 1e-12) + d) | (lifted & (q == 2.0 ** -9)))
        return
    low = np.floor(np.abs(y) / sp) * sp
    place = (np.abs(y) - low) / sp + (random + 0.5) / 65536 - 1
    near = np.abs(place) <= 2.0 ** -18 + d / sp * 2
    up = low + sp * (place >= 0)
    assert np.all(near | (np.abs(q) == up) | (lifted & (q == 2.0 ** -9)))
    assert np.all(np.abs(np.abs(q) - np.abs(y)) <= sp + d)
    assert near.mean() < 0.01 or len(x) < 1000
    assert np.all((np.sign(q) == np.sign(y)) | (q == 0))


SIZES = [1, 7, 255, 256, 257, 4096, 8191, 8192, 8193, 30011]


@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "nearest"), (8, "stochastic")])
@pytest.mark.parametrize("grad_kind,param_kind", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", None), ("fp32", "bf16"), ("bf16", "fp16")])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(bits, rounding, grad_kind, param_kind, shift):
    rng = np.random.default_rng(bits + 7 * shift)
    states = [rand_state(n, bits, rng, grad_kind) for n in SIZES]
    bufs, lst = make(states, bits, grad_kind, param_kind, shift)
    info = zs.zs_tensors_info(lst)
    assert info["numel"] == sum(SIZES) and info["n_tensors"] == len(SIZES)
    assert info["n_blocks"] == sum(-(-n // 256) for n in SIZES)
    coef = torch.full((1,), 0.625, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    step, seed = 5, 0x1234567890ABCDEF
    zs.zs_adam_tensors(lst, HP, step, coef, flags, rounding=rounding, seed=seed)
    torch.cuda.synchronize()
    for i, (s, b) in enumerate(zip(states, bufs)):
        assert all(x.guards_ok() for x in b.values())
        n = len(s["p"])
        m0, v0 = (s["m"].astype(np.float64), s["v"].astype(np.float64)) if bits == 32 else \
            (held(s["m_code"], s["m_scale"]), held(s["r_code"], s["r_scale"]) ** 2)
        p, m, r, dp, dm, dr = bounds(s, m0, v0, HP, step, 0.625)
        got = {k: x.t.cpu().numpy() for k, x in b.items() if k not in ("grad", "param")}
        assert np.all(np.abs(got["master"] - p) <= dp)
        if param_kind:
            check_param(b)
        if bits == 32:
            assert np.all(np.abs(got["exp_avg"] - m) <= dm)
            assert np.all(np.abs(np.sqrt(got["exp_avg_sq"].astype(np.float64)) - r) <= dr)
            continue
        a, c = ref.random16(n, i, step, seed) if rounding == "stochastic" else (None, None)
        check_codes(got["exp_avg"], got["exp_avg_scale"], m, dm, a)
        check_codes(got["exp_avg_sq"], got["exp_avg_sq_scale"], r, dr, c, least=True)


@pytest.mark.parametrize("adamw,bias_correction", [(0, 1), (1, 0), (0, 0)])
@pytest.mark.parametrize("bits", [8, 32])
def test_modes(adamw, bias_correction, bits):
    """Adam-L2, no bias correction; no coefficient and no flags; another stream."""
    hp = dict(HP, adamw=adamw, bias_correction=bias_correction)
    rng = np.random.default_rng(3)
    states = [rand_state(n, bits, rng, "bf16") for n in (300, 9000)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        bufs, lst = make(states, bits, "bf16", "bf16")
        zs.zs_adam_tensors(lst, hp, 3, stream=stream)
    stream.synchronize()
    for s, b in zip(states, bufs):
        m0, v0 = (s["m"].astype(np.float64), s["v"].astype(np.float64)) if bits == 32 else \
            (held(s["m_code"], s["m_scale"]), held(s["r_code"], s["r_scale"]) ** 2)
        p, m, r, dp, dm, dr = bounds(s, m0, v0, hp, 3, 1.0)
        assert np.all(np.abs(b["master"].t.cpu().numpy() - p) <= dp)


def test_32_equals_plan_step():
    """A list over a plan's shard rows and persistent space gives zs_adam_step's bits."""
    from tests.gpu_harness import DevicePlan
    d = DevicePlan([4096, 64, 33333, 256, 5000, 64], 4, threshold=100, B=20_000)
    d.init_weights()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for k in ("grad_shards", "persist_grads"):
        t = d.bufs[k].t
        t.copy_((torch.randn(t.numel(), device="cuda", generator=gen) * 1e-3).bfloat16().view(torch.int16))
    for k in ("exp_avg", "p_exp_avg", "exp_avg_sq", "p_exp_avg_sq"):
        t = d.bufs[k].t
        t.copy_(torch.rand(t.numel(), device="cuda", generator=gen) * (1e-6 if "sq" in k else 1e-3))
    d.d_coef.t.fill_(0.3)
    d.d_flags.t.zero_()
    mine = {k: b.t.clone() for k, b in d.bufs.items()}
    N, S = d.op.group, d.op.S
    items = [dict(grad=mine["grad_shards"][r * S:(r + 1) * S].view(torch.bfloat16),
                  param=mine["param_shards"][r * S:(r + 1) * S].view(torch.bfloat16),
                  **{k: mine[k][r * S:(r + 1) * S] for k in ("master", "exp_avg", "exp_avg_sq")}) for r in range(N)]
    items.append(dict(grad=mine["persist_grads"].view(torch.bfloat16), param=mine["persist_params"].view(torch.bfloat16),
                      master=mine["p_master"], exp_avg=mine["p_exp_avg"], exp_avg_sq=mine["p_exp_avg_sq"]))
    lst = upload(items, 32)
    for step in (1, 2):
        zs.zs_adam_step(d.plan, -1, HP, step, d.d_coef.t, d.d_flags.t, d.state)
        zs.zs_adam_tensors(lst, HP, step, d.d_coef.t, d.d_flags.t)
    torch.cuda.synchronize()
    for k, b in d.bufs.items():
        assert torch.equal(b.t.view(torch.uint8), mine[k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [8, 32])
def test_skip_and_empty(bits):
    rng = np.random.default_rng(0)
    s = rand_state(1000, bits, rng, "bf16")
    bufs, lst = make([s], bits, "bf16", "bf16")
    before = {k: b.t.clone() for k, b in bufs[0].items()}
    flags = torch.full((1,), zs.ZS_SKIP_NONFINITE, dtype=torch.int32, device="cuda")
    zs.zs_adam_tensors(lst, HP, 1, None, flags)
    torch.cuda.synchronize()
    for k, b in bufs[0].items():
        assert torch.equal(b.t.view(torch.uint8), before[k].view(torch.uint8)), k
    zs.zs_adam_tensors(upload([], bits), HP, 1)                      # no tensors
    e = lambda dt: torch.empty(0, dtype=dt, device="cuda")  # noqa: E731
    st = torch.uint8 if bits == 8 else torch.float32
    empty = dict(grad=e(torch.bfloat16), master=e(torch.float32), exp_avg=e(st), exp_avg_sq=e(st))
    bufs, lst = make([s], bits, "bf16", "bf16")
    lst = upload([empty, {k: b.t for k, b in bufs[0].items()}, empty], bits)
    zs.zs_adam_tensors(lst, HP, 1)
    torch.cuda.synchronize()
    assert not torch.equal(bufs[0]["master"].t, before["master"])


def test_first_step_from_zero_bytes():
    """A state of zero bytes is a run that has not begun: the first update is lr in size, of the gradient's sign."""
    n = 5000
    g = torch.randn(n, generator=torch.Generator().manual_seed(2)) * 1e-3
    z8 = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    zs_ = lambda: torch.zeros(-(-n // 256), device="cuda")  # noqa: E731
    t = dict(grad=g.cuda(), master=torch.zeros(n, device="cuda"), exp_avg=z8(), exp_avg_sq=z8(), exp_avg_scale=zs_(),
             exp_avg_sq_scale=zs_())
    zs.zs_adam_tensors(upload([t], 8), dict(HP, weight_decay=0.0), 1)
    want = -1e-3 * g.double() / (g.double().abs() + 1e-8)
    assert torch.allclose(t["master"].cpu().double(), want, rtol=1e-5, atol=0)


def test_nonfinite_gradients():
    """An element whose moments are not finite gets NaN codes; its block's others are as without it."""
    rng = np.random.default_rng(5)
    s = rand_state(700, 8, rng, "fp32")
    clean, dirty = dict(s), dict(s)
    g = s["grad"].clone()
    at = [3, 255, 256, 699]
    g[at] = 0.0
    clean["grad"] = g.clone()
    g[at] = torch.tensor([float("nan"), float("inf"), float("-inf"), 1e30])
    dirty["grad"] = g
    # the elements themselves must not decide the clean block's scale
    for k in ("m_code", "r_code"):
        clean[k] = s[k].copy()
        clean[k][at] = 0
        dirty[k] = clean[k]
    a, la = make([clean], 8, "fp32", "bf16")
    b, lb = make([dirty], 8, "fp32", "bf16")
    for lst in (la, lb):
        zs.zs_adam_tensors(lst, HP, 2, rounding="stochastic", seed=9)
    torch.cuda.synchronize()
    keep = np.ones(700, bool)
    keep[at] = False
    for k in ("exp_avg", "exp_avg_sq"):
        x, y = a[0][k].t.cpu().numpy(), b[0][k].t.cpu().numpy()
        if k == "exp_avg_sq":
            assert np.all((y[at[:3]] & 0x7F) == 0x7F)
            assert (y[699] & 0x7F) == 0x7F                            # 1e60 is past float32
        else:
            assert np.all((y[at[:3]] & 0x7F) == 0x7F)
            continue                                                 # 1e29 decides its block's exp_avg scale
        assert np.array_equal(x[keep], y[keep])
    x, y = a[0]["exp_avg"].t.cpu().numpy(), b[0]["exp_avg"].t.cpu().numpy()
    assert np.array_equal(x[:512][keep[:512]], y[:512][keep[:512]])
    assert np.array_equal(a[0]["master"].t.cpu().numpy()[keep], b[0]["master"].t.cpu().numpy()[keep])


def test_range_of_moments():
    """Blocks of zeros, of the smallest and of large values: scales stay normal numbers, nothing overflows."""
    n = 256 * 6
    g = np.zeros(n, np.float32)
    g[256:512] = 1e-30
    g[512:768] = 1e-38
    g[768:1024] = 1e15
    g[1024:1280] = np.logspace(-12, 2, 256)
    g[1280:] = np.where(np.arange(256) == 7, 3e-3, 0)
    z = dict(grad=torch.from_numpy(g), p=np.zeros(n, np.float32), m_code=np.zeros(n, np.uint8), r_code=np.zeros(n, np.uint8),
             m_scale=np.zeros(6, np.float32), r_scale=np.zeros(6, np.float32))
    bufs, lst = make([z], 8, "fp32", None)
    zs.zs_adam_tensors(lst, dict(HP, eps=1e-20), 1)
    torch.cuda.synchronize()
    b = {k: x.t.cpu().numpy() for k, x in bufs[0].items()}
    assert np.all(b["exp_avg_scale"] >= 2.0 ** -126) and np.all(np.isfinite(b["exp_avg_scale"]))
    assert np.all(b["exp_avg"][:256] == 0) and np.all(b["exp_avg_sq"][:256] == 0)
    assert np.all(np.isfinite(ref.E4M3[b["exp_avg"]])) and np.all(np.isfinite(ref.E4M3[b["exp_avg_sq"]]))
    assert np.all(b["exp_avg_sq"][1024:1280] != 0)                    # a positive root is never held as zero
    assert np.all(np.isfinite(b["master"]))


def test_stochastic_rounding_has_no_bias():
    """The mean of many roundings of one value is the value: 2^16 elements, within 5 standard deviations."""
    n = 1 << 16
    hp = dict(HP, beta1=0.0, beta2=0.0, weight_decay=0.0)
    g = torch.full((n,), 1.03, device="cuda")
    g[::256] = 2.0                                                     # the block's scale: 2^(1 - 7)
    t = dict(grad=g, master=torch.zeros(n, device="cuda"), exp_avg=torch.zeros(n, dtype=torch.uint8, device="cuda"),
             exp_avg_sq=torch.zeros(n, dtype=torch.uint8, device="cuda"), exp_avg_scale=torch.zeros(256, device="cuda"),
             exp_avg_sq_scale=torch.zeros(256, device="cuda"))
    zs.zs_adam_tensors(upload([t], 8), hp, 1, rounding="stochastic", seed=77)
    for name in ("exp_avg", "exp_avg_sq"):
        v = ref.E4M3[t[name].cpu().numpy()].reshape(-1, 256)[:, 1:] * 2.0 ** -6
        assert set(np.unique(v)) == {1.0, 1.125}
        assert abs(v.mean() - 1.03) < 5 * 0.125 * 0.5 / np.sqrt(v.size)
    # another seed and another step round otherwise
    first = t["exp_avg"].clone()
    zs.zs_adam_tensors(upload([t], 8), hp, 1, rounding="stochastic", seed=78)
    assert not torch.equal(first, t["exp_avg"])


def test_same_bits_twice():
    rng = np.random.default_rng(11)
    s = rand_state(20000, 8, rng, "bf16")
    out = []
    for _ in range(2):
        bufs, lst = make([s], 8, "bf16", "bf16")
        for step in (1, 2, 3):
            zs.zs_adam_tensors(lst, HP, step, rounding="stochastic", seed=4)
        torch.cuda.synchronize()
        out.append({k: b.t.clone() for k, b in bufs[0].items()})
    for k in out[0]:
        assert torch.equal(out[0][k].view(torch.uint8), out[1][k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [8, 32])
def test_past_32_bits(bits):
    """A tensor of more than 2^31 elements: its end equals a small tensor's."""
    n, tail = 2 ** 31 + 5003, 4 * 6144 + 5003
    dev = dict(device="cuda")
    t = dict(grad=torch.zeros(n, dtype=torch.bfloat16, **dev), param=torch.zeros(n, dtype=torch.bfloat16, **dev), master=torch.zeros(n, **dev))
    kind = torch.uint8 if bits == 8 else torch.float32
    t.update(exp_avg=torch.zeros(n, dtype=kind, **dev), exp_avg_sq=torch.zeros(n, dtype=kind, **dev))
    if bits == 8:
        blocks = -(-n // 256)
        t.update(exp_avg_scale=torch.zeros(blocks, **dev), exp_avg_sq_scale=torch.zeros(blocks, **dev))
    g = torch.Generator(device="cuda").manual_seed(3)
    t["grad"][-tail:].normal_(0, 1e-3, generator=g)
    t["master"][-tail:].normal_(0, 0.02, generator=g)
    small = {k: v[-(-(-tail // 256)):].clone() if k.endswith("scale") else v[-tail:].clone() for k, v in t.items()}
    a, b = upload([t], bits), upload([small], bits)
    for step in (1, 2):
        zs.zs_adam_tensors(a, HP, step)
        zs.zs_adam_tensors(b, HP, step)
    for k, v in small.items():
        assert torch.equal(t[k][-len(v):], v), k
    assert not t["master"][:-tail].any()
