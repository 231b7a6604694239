"""zs_norm_tensors and zs_clip_tensors on the GPU against the definition in 64 bits.

Tolerances: the root is good to 2^-32 (include/zs.h) and rounded once to
float32, so the norm is within (2^-24 + 2^-32) of itself, twice 2^-24 with a
loss scale that is no power of two.  The coefficient is computed from the norm
that came back with float32's own operations, and clipped gradients with
torch's one product and rounding: bit for bit.
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests.test_gpu_tensors import KINDS, Buf

pytestmark = pytest.mark.gpu
ROOT = 2.0 ** -24 + 2.0 ** -32
A16 = 1 << 20        # an address that neither call follows


class List:
    """Gradients with guards around each, the list over them, and the norm's outputs and scratch."""

    def __init__(self, values, kind, shift=0, bits=8):
        self.bufs = [Buf(v, KINDS[kind], shift) for v in values]
        code = {"bf16": zs.ZS_DTYPE_BF16, "fp16": zs.ZS_DTYPE_FP16, "fp32": zs.ZS_DTYPE_FP32}[kind]
        items = [dict(numel=b.t.numel(), grad=b.t.data_ptr(), master=A16, exp_avg=A16, exp_avg_sq=A16, exp_avg_scale=A16,
                      exp_avg_sq_scale=A16) for b in self.bufs]
        self.list = zs.zs_build_tensors(items, state_bits=bits, grad_dtype=code)
        info = zs.zs_tensors_info(self.list)
        self.table = torch.empty(max(info["device_table_bytes"], 16), dtype=torch.uint8, device="cuda")
        zs.zs_tensors_upload(self.list, self.table, self.table.numel())
        self.scratch = Buf(np.full(info["n_chunks"], np.nan), torch.float64)
        self.out = [Buf(np.full(1, 7), dt) for dt in (torch.float32, torch.float32, torch.int32)]

    def norm(self, max_norm=1.0, scaler=None, **kw):
        zs.zs_norm_tensors(self.list, self.scratch.t, max_norm, *(b.t for b in self.out), scaler=scaler, **kw)
        torch.cuda.synchronize()
        assert all(b.guards_ok() for b in self.bufs + self.out + [self.scratch])
        return tuple(b.t.cpu().numpy()[0] for b in self.out)

    def clip(self, coef=None, flags=None, **kw):
        zs.zs_clip_tensors(self.list, self.out[1].t if coef is None else coef, flags, **kw)
        torch.cuda.synchronize()
        assert all(b.guards_ok() for b in self.bufs)


def want_norm(values, kind):
    total = sum(float((torch.as_tensor(v).to(KINDS[kind]).double() ** 2).sum()) for v in values)
    return np.sqrt(total)


def want_coef(norm, max_norm, scale=1.0):
    f = np.float32
    clip = f(1) if max_norm <= 0 else min(f(1), f(max_norm) / (f(norm) + f(1e-6)))
    return f(clip) / f(scale)


SIZES = [1, 7, 8, 255, 2047, 2048, 2049, 4096, 8191, 30011]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bits", [8, 32])
def test_norm(kind, shift, bits):
    rng = np.random.default_rng(shift + bits)
    values = [rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 0) for n in SIZES]
    li = List(values, kind, shift, bits)
    before = [b.t.clone() for b in li.bufs]
    for max_norm in (0.25, 1e6, 0.0, -1.0):
        norm, coef, flags = li.norm(max_norm)
        want = want_norm(values, kind)
        assert abs(float(norm) - want) <= ROOT * want
        assert coef == want_coef(norm, max_norm) and flags == 0
    assert all(torch.equal(b.t, x) for b, x in zip(li.bufs, before))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("numel", [3_000_000, 6_000_001])
def test_long_lists(kind, numel):
    """Chunks of the long kind, several a CTA; and one of the tensors all but alone in its size."""
    gen = torch.Generator(device="cuda").manual_seed(numel)
    g = torch.randn(numel, device="cuda", generator=gen).to(KINDS[kind])
    g[12345] = 3000.0
    values = [g.cpu(), torch.ones(5)]
    li = List(values, kind)
    norm, coef, flags = li.norm(1.0)
    want = want_norm(values, kind)
    assert abs(float(norm) - want) <= ROOT * want and coef == want_coef(norm, 1.0) and flags == 0


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** -126, 1e-30, 2.0 ** -41, 2.0 ** -39, 2.0 ** 55, 2.0 ** 57, 1e30])
def test_range(kind, size):
    """Magnitudes at and past both ends of the range that float32 squares have."""
    rng = np.random.default_rng(5)
    values = [rng.uniform(0.5, 1.0, n) * size for n in (3, 5000, 20000)]
    for v in (values, [values[1], rng.standard_normal(4000) * 1e-3]):
        li = List(v, kind)
        norm, coef, flags = li.norm(1.0)
        want = want_norm(v, kind)
        # a norm among float32's subnormals is off by half of 2^-149 more
        assert abs(float(norm) - want) <= ROOT * want + 2.0 ** -150
        assert coef == want_coef(norm, 1.0) and flags == 0


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("at", [0, 9998, 9999])
def test_not_finite(kind, bad, at):
    values = [np.ones(100), np.ones(9999 + 1)]
    values[1][at] = bad
    li = List(values, kind)
    before = [b.t.clone() for b in li.bufs]
    norm, coef, flags = li.norm(1.0)
    assert not np.isfinite(norm) and coef == 1 and flags == zs.ZS_SKIP_NONFINITE
    half = torch.full((1,), 0.5, device="cuda")
    li.clip(half, li.out[2].t)                      # the flag keeps the gradients
    assert all(torch.equal(b.t.view(torch.uint8), x.view(torch.uint8)) for b, x in zip(li.bufs, before))


def test_overflow_of_the_norm():
    """fp32 gradients that are finite, and a norm that is not."""
    li = List([np.full(100, 3e38)], "fp32")
    norm, coef, flags = li.norm(1.0)
    assert np.isinf(norm) and coef == 1 and flags == zs.ZS_SKIP_NONFINITE


def test_nothing():
    e = np.zeros(0)
    for values in ([], [e], [e, np.zeros(5), e]):
        norm, coef, flags = List(values, "bf16").norm(1.0)
        assert norm == 0 and coef == 1 and flags == 0
        List(values, "bf16").clip(torch.full((1,), 0.5, device="cuda"))
    values = [e, np.full(3, 2.0), e]
    assert List(values, "bf16").norm(1.0)[0] == np.float32(np.sqrt(12.0))


@pytest.mark.parametrize("scale", [1024.0, 3.0])
@pytest.mark.parametrize("bad", [False, True])
def test_loss_scale(scale, bad):
    """The scaler's part: the norm and coefficient over S, and S afterwards as zs_unscale_and_clip leaves it."""
    values = [np.random.default_rng(1).standard_normal(5000) * scale]
    if bad:
        values[0][77] = np.inf
    li = List(values, "fp16")
    d_scale, d_good = torch.full((1,), scale, device="cuda"), torch.full((1,), 1, dtype=torch.int32, device="cuda")
    static = zs.make_loss_scaler(d_scale, scale_window=0)
    dynamic = zs.make_loss_scaler(d_scale, d_good, scale_factor=2.0, min_scale=1.0, scale_window=3)
    for scaler, good, left in ((static, 1, scale), (dynamic, 0 if bad else 2, scale / 2 if bad else scale),
                               (dynamic, 0, scale / 4 if bad else 2 * scale)):
        at = float(d_scale)
        norm, coef, flags = li.norm(1.0, scaler)
        assert (int(d_good), float(d_scale)) == (good, np.float32(max(left, 1.0)))
        if bad:
            assert not np.isfinite(norm) and coef == 1 and flags == zs.ZS_SKIP_NONFINITE
            continue
        want = want_norm(values, "fp16") / at
        assert abs(float(norm) - want) <= 2 * ROOT * want
        assert coef == want_coef(norm, 1.0, at) and flags == 0


def test_equals_the_plan():
    """A list of what a plan's parameters have in its shard rows and persistent space (the norm of a plan leaves the padding
    between them out): zs_grad_norm's norm, but for a rounding at a border."""
    from tests.gpu_harness import DevicePlan
    d = DevicePlan([4096, 64, 33333, 256, 5000, 64], 4, threshold=100, B=20_000)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in ("grad_shards", "persist_grads"):
        t = d.bufs[k].t
        t.copy_((torch.randn(t.numel(), device="cuda", generator=gen) * 1e-3).bfloat16().view(torch.int16))
    info = zs.zs_plan_info(d.plan)
    scratch = torch.empty(info["norm_scratch_elems"], dtype=torch.float64, device="cuda")
    zs.zs_grad_norm(d.plan, d.bufs["grad_shards"].t, d.bufs["persist_grads"].t, scratch, True, 0.01, d.d_norm.t, d.d_coef.t, d.d_flags.t)
    N, S = d.op.group, d.op.S
    values = []
    for i in range(info["n_params"]):
        p = zs.zs_param_info(d.plan, i)
        if p["persistent"]:
            at = p["persist_offset"]
            values.append(d.bufs["persist_grads"].t[at:at + p["numel"]])
            continue
        for r in range(N):
            at, ps = r * S + p["shard_offset"], p["partition_size"]
            values.append(d.bufs["grad_shards"].t[at:at + max(0, min(ps, p["numel"] - r * ps))])
    li = List([v.view(torch.bfloat16).cpu() for v in values], "bf16")
    norm, coef, flags = li.norm(0.01)
    assert abs(float(norm) - float(d.d_norm.t[0])) <= 2.0 ** -23 * float(norm)
    assert coef == want_coef(norm, 0.01) and flags == int(d.d_flags.t[0])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip(kind, shift):
    rng = np.random.default_rng(9)
    values = [rng.standard_normal(n) for n in SIZES]
    values[5][:4] = [np.inf, -np.inf, np.nan, 1e-7]
    li = List(values, kind, shift)
    before = [b.t.clone() for b in li.bufs]
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8)) or torch.equal(a.nan_to_num(nan=-77.0), b.nan_to_num(nan=-77.0))  # noqa: E731
    for c in (1.0, 0.37, 1.0 / 3, 2.0 ** -10):
        coef = torch.full((1,), c, device="cuda")
        li.clip(coef, torch.zeros(1, dtype=torch.int32, device="cuda"))
        for b, x in zip(li.bufs, before):
            x.copy_((x.float() * coef).to(x.dtype))
            assert same(b.t, x), (c, b.t.numel())


def test_norm_then_clip_then_update():
    """Clipping in place and then updating is updating with the coefficient, but for the gradients' rounding (fp32: the same product)."""
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    gen = torch.Generator(device="cuda").manual_seed(4)
    grads = [torch.randn(n, device="cuda", generator=gen) for n in (300, 9001)]

    def state():
        ts = [dict(grad=g.clone(), master=torch.ones_like(g), exp_avg=torch.zeros_like(g), exp_avg_sq=torch.zeros_like(g)) for g in grads]
        lst = zs.zs_build_tensors(ts)
        info = zs.zs_tensors_info(lst)
        table = torch.empty(info["device_table_bytes"], dtype=torch.uint8, device="cuda")
        zs.zs_tensors_upload(lst, table, table.numel())
        norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        flags = torch.empty(1, dtype=torch.int32, device="cuda")
        zs.zs_norm_tensors(lst, torch.empty(info["n_chunks"], dtype=torch.float64, device="cuda"), 0.5, norm, coef, flags)
        return ts, lst, coef, flags, table

    a, la, coef, flags, _t = state()
    zs.zs_adam_tensors(la, hp, 1, coef, flags)
    b, lb, coef, flags, _u = state()
    zs.zs_clip_tensors(lb, coef, flags)
    zs.zs_adam_tensors(lb, hp, 1, None, flags)
    torch.cuda.synchronize()
    assert 0 < float(coef) < 1
    for x, y in zip(a, b):
        assert torch.equal(x["master"], y["master"]) and not torch.equal(x["grad"], y["grad"])


def test_stream_graph_and_same_bits():
    rng = np.random.default_rng(11)
    values = [rng.standard_normal(n) for n in (5000, 70001, 12)]
    li, other = List(values, "bf16"), List([2 * v for v in values], "bf16")
    first = li.norm(1.0)
    stream = torch.cuda.Stream()
    assert li.norm(1.0, stream=stream) == first
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g, x in ((g1, li), (g2, other)):
        with torch.cuda.graph(g):
            zs.zs_norm_tensors(x.list, x.scratch.t, 1.0, *(b.t for b in x.out))
            zs.zs_clip_tensors(x.list, x.out[1].t, x.out[2].t)
    others = other.norm(1.0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        g1.replay()
    with torch.cuda.stream(s2):
        g2.replay()
    torch.cuda.synchronize()
    for x, before in ((li, first), (other, others)):
        assert tuple(b.t.cpu().numpy()[0] for b in x.out) == before
        after = x.norm(1.0)[0]
        # each gradient is rounded to 8 bits after the product: the norm within half a step of max_norm, and 1e-6 of it
        assert abs(float(after) - 1.0) <= 2.0 ** -8 + 2e-6


def test_one_tensor_past_2_31():
    n = (1 << 31) + 5000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[1 << 31], g[n - 1] = 3.0, 4.0, 12.0
    item = dict(numel=n, grad=g.data_ptr(), master=A16, exp_avg=A16, exp_avg_sq=A16, exp_avg_scale=A16, exp_avg_sq_scale=A16)
    lst = zs.zs_build_tensors([item], state_bits=8, grad_dtype=zs.ZS_DTYPE_BF16)
    info = zs.zs_tensors_info(lst)
    table = torch.empty(info["device_table_bytes"], dtype=torch.uint8, device="cuda")
    zs.zs_tensors_upload(lst, table, table.numel())
    norm, coef, flags = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    zs.zs_norm_tensors(lst, torch.empty(info["n_chunks"], dtype=torch.float64, device="cuda"), 6.5, norm, coef, flags)
    zs.zs_clip_tensors(lst, coef, flags)
    assert float(norm) == 13.0 and int(flags) == 0
    assert [float(g[i]) for i in (0, 1 << 31, n - 1, 5)] == [1.5, 2.0, 6.0, 0.0]


def test_refused_tensors():
    li = List([np.ones(5000)], "bf16")
    norm, coef, flags = (b.t for b in li.out)
    for bad in (dict(scratch=torch.empty(1, device="cuda")), dict(scratch=torch.empty(100, dtype=torch.float64)), dict(d_norm=norm.cpu())):
        a = dict(scratch=li.scratch.t, d_norm=norm)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            zs.zs_norm_tensors(li.list, a["scratch"], 1.0, a["d_norm"], coef, flags)
    with pytest.raises(TypeError):
        zs.zs_norm_tensors(li.list, li.scratch.t, 1.0, norm, coef.double(), flags)
    with pytest.raises(ValueError):
        zs.zs_clip_tensors(li.list, coef.cpu())
