"""zs_mx4_matvec on the GPU against the sum in 64 bits of the values held.

Tolerance, from include/zs.h: (ceil(k / 32) + 24) 2^-22 sum |x w|, and 2^-39
(fp32: 2^-50) of the row's largest magnitude times sum |w|, then half a step of
the output's type.  fp32 tokens: 2^-22 |x w| more, which the 24 holds.
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests import lowbit_ref as ref
from tests.test_gpu_rms_norm import HALF, LEAST, Mat, same
from tests.test_gpu_tensors import KINDS

pytestmark = pytest.mark.gpu


def weight(n, k, rng, span=6):
    """Random codes and scale bytes of a weight, and the values that they stand for."""
    kp = -(-k // 32) * 32
    code = rng.integers(0, 16, (n, kp)).astype(np.uint8)
    code[:, k:] = 0
    byte = rng.integers(120 - span, 120 + span + 1, (n, kp // 32)).astype(np.uint8)
    held = dict(codes=torch.from_numpy(ref.pack(code)).cuda(), scales=torch.from_numpy(ref.tile_scales(byte)).cuda())
    return held, torch.from_numpy(ref.mx4_values(code, byte)[:, :k]).cuda()


def check(x, held, w, out_kind, extra=0, shift=0, **kw):
    m, n, k = len(x), len(w), x.shape[1]
    out = Mat(m, n, out_kind, extra=extra, shift=shift)
    assert zs.zs_mx4_matvec(x, held, out.t, **kw) is out.t
    torch.cuda.synchronize()
    x64 = x.double()
    want = x64 @ w.t()
    small = 2.0 ** -50 if x.dtype == torch.float32 else 2.0 ** -39
    tol = (-(-k // 32) + 24) * 2.0 ** -22 * (x64.abs() @ w.abs().t()) + small * x64.abs().amax(1, keepdim=True) * w.abs().sum(1)[None, :]
    tol = tol * (1 + HALF[out_kind]) + HALF[out_kind] * want.abs() + LEAST[out_kind]
    assert bool(((out.t.double() - want).abs() <= tol).all()), float(((out.t.double() - want).abs() / tol).max())
    assert out.outside_ok()
    return out.t


SHAPES = [(1, 1, 1), (1, 16, 32), (2, 17, 33), (1, 128, 128), (3, 129, 127), (5, 777, 1490), (8, 64, 4096), (9, 100, 5000), (16, 1024, 300), (17, 33, 2050),
          (32, 300, 1100), (33, 130, 640), (1, 4096, 14336), (65, 40, 9000), (4, 3000, 96), (1, 2, 20000), (130, 20, 50)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind,out_kind", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_product(m, n, k, kind, out_kind):
    rng = np.random.default_rng(m + n + k)
    held, w = weight(n, k, rng)
    x = torch.from_numpy(rng.standard_normal((m, k)) * 10.0 ** rng.uniform(-2, 1, (m, 1))).cuda()
    check(x.to(KINDS[kind]), held, w * 1.0, out_kind) if out_kind != "fp16" else check((x / 100).to(KINDS[kind]), held, w, out_kind)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_strides_and_addresses(kind):
    rng = np.random.default_rng(2)
    for m, n, k, extra, shift in ((3, 70, 200, 5, 1), (12, 50, 333, 8, 3), (20, 31, 64, 1, 0)):
        held, w = weight(n, k, rng)
        x = Mat(m, k, kind, torch.from_numpy(rng.standard_normal((m, k))).cuda(), extra, shift)
        check(x.t, held, w, "fp32", extra, shift)


@pytest.mark.parametrize("m", [1, 8, 11, 32])
def test_exact(m):
    """Small whole numbers and scales of 1: every sum is exact, in every type."""
    rng = np.random.default_rng(m)
    n, k = 150, 900
    code = rng.integers(0, 16, (n, 928)).astype(np.uint8)
    code[:, k:] = 0
    byte = np.full((n, 29), 127, np.uint8)
    held = dict(codes=torch.from_numpy(ref.pack(code)).cuda(), scales=torch.from_numpy(ref.tile_scales(byte)).cuda())
    w = torch.from_numpy(ref.mx4_values(code, byte)[:, :k]).cuda()
    x = torch.from_numpy(rng.integers(-4, 5, (m, k))).cuda()
    for kind in KINDS:
        out = torch.empty(m, n, device="cuda")
        zs.zs_mx4_matvec(x.to(KINDS[kind]), held, out)
        assert torch.equal(out.double(), x.double() @ w.t())


def test_equals_the_4_bit_product():
    """Tokens that 4 bits hold exactly: what zs_mx4_matmul gives, to both calls' rounding."""
    rng = np.random.default_rng(8)
    held, w = weight(200, 512, rng)
    tokens, x = weight(6, 512, rng)
    a, b = torch.empty(6, 200, device="cuda"), torch.empty(6, 200, device="cuda")
    zs.zs_mx4_matmul(tokens, held, 512, a)
    zs.zs_mx4_matvec(x.float(), held, b)
    bound = (512 // 64 + 8 + 512 // 32 + 24) * 2.0 ** -22 * (x.abs() @ w.abs().t()) + 2.0 ** -50 * x.abs().amax(1, keepdim=True) * w.abs().sum(1)[None, :]
    assert bool(((a.double() - b.double()).abs() <= bound).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_range(kind):
    """Tokens far from 1 and far from one another, and scales at both ends."""
    rng = np.random.default_rng(4)
    held, w = weight(64, 700, rng, span=40)
    x = torch.from_numpy(rng.standard_normal((7, 700))).cuda()
    x[0] *= 1e-30
    x[1] *= 1e25
    x[2] = 0
    x[3, ::2] *= 1e-12
    x[4, 5:] = 0
    x[5] *= 10.0 ** torch.linspace(-20, 0, 700, device="cuda").double()
    x[6] *= 1e-39
    check(x.to(KINDS[kind]), held, w, "fp32")
    code = np.full((3, 64), 2, np.uint8)                         # 1
    byte = np.array([[0, 0], [254, 0], [1, 3]], np.uint8)
    held = dict(codes=torch.from_numpy(ref.pack(code)).cuda(), scales=torch.from_numpy(ref.tile_scales(byte)).cuda())
    x = torch.zeros(2, 64, device="cuda")
    x[0, 0], x[1, 40] = 2.0 ** -8, 1.0
    out = torch.empty(2, 3, device="cuda")
    zs.zs_mx4_matvec(x.to(KINDS[kind]), held, out)
    # results among float32's subnormals may lose a bit to the scaling by powers of two
    want = torch.tensor([[2.0 ** -135, 2.0 ** 119, 2.0 ** -134], [2.0 ** -127, 2.0 ** -127, 2.0 ** -124]], dtype=torch.float64)
    assert bool(((out.cpu().double() - want).abs() <= 2.0 ** -149).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m", [2, 20])
def test_not_finite(kind, m):
    """An infinity or NaN of one token, a NaN group of one feature: theirs alone."""
    rng = np.random.default_rng(6)
    n, k = 40, 300
    code = rng.integers(1, 8, (n, 320)).astype(np.uint8)         # positive, not 0
    code[:, k:] = 0
    byte = rng.integers(120, 130, (n, 10)).astype(np.uint8)
    byte[7, 3] = 255
    held = dict(codes=torch.from_numpy(ref.pack(code)).cuda(), scales=torch.from_numpy(ref.tile_scales(byte)).cuda())
    x = torch.from_numpy(rng.uniform(0.5, 1, (m, k))).cuda()
    clean = torch.empty(m, n, device="cuda")
    zs.zs_mx4_matvec(x.to(KINDS[kind]), held, clean)
    assert bool(torch.isnan(clean[:, 7]).all()) and bool(torch.isfinite(clean[:, :7]).all()) and bool(torch.isfinite(clean[:, 8:]).all())
    x[0, 17], x[1, 250] = float("inf"), float("nan")
    out = torch.empty(m, n, device="cuda")
    zs.zs_mx4_matvec(x.to(KINDS[kind]), held, out)
    assert bool(torch.isnan(out[:, 7]).all()) and bool(torch.isnan(out[1]).all())
    rest = [i for i in range(n) if i != 7]
    assert bool((out[0, rest] == float("inf")).all()) and same(out[2:], clean[2:])


def test_nothing():
    held, w = weight(40, 64, np.random.default_rng(0))
    out = Mat(3, 40, "fp32", extra=4)
    zs.zs_mx4_matvec(torch.empty(3, 0, device="cuda"), dict(codes=torch.empty(0, dtype=torch.uint8, device="cuda"),
                                                            scales=torch.empty(0, dtype=torch.uint8, device="cuda")), out.t)
    assert bool((out.t == 0).all()) and out.outside_ok()
    zs.zs_mx4_matvec(torch.empty(0, 64, device="cuda"), held, torch.empty(0, 40, device="cuda"))
    zs.zs_mx4_matvec(torch.empty(3, 64, device="cuda"), dict(codes=torch.empty(0, dtype=torch.uint8, device="cuda"),
                                                             scales=torch.empty(0, dtype=torch.uint8, device="cuda")), torch.empty(3, 0, device="cuda"))


def test_offsets_past_32_bits():
    """A weight whose codes take more than 2^32 bytes; the last rows are compared."""
    n, k = 300_000, 32_000
    size = zs.zs_mx4_sizes(n, k)
    assert size["code_bytes"] > 1 << 32
    held = dict(codes=torch.zeros(size["code_bytes"], dtype=torch.uint8, device="cuda"), scales=torch.full((size["scale_bytes"],), 127, dtype=torch.uint8, device="cuda"))
    held["codes"].view(n, -1)[-3:] = 0x22                        # 1 everywhere
    x = torch.ones(2, k, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, n, device="cuda")
    zs.zs_mx4_matvec(x, held, out)
    assert bool((out[:, -3:] == k).all()) and not bool(out[:, :-3].any())


def test_streams_graphs_and_the_kernel_before():
    rng = np.random.default_rng(12)
    held, w = weight(500, 3000, rng)
    x = torch.from_numpy(rng.standard_normal((3, 3000))).cuda().bfloat16()
    first = check(x, held, w, "bf16").clone()
    out = torch.empty_like(first)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    zs.zs_mx4_matvec(x, held, out, stream=stream)
    torch.cuda.synchronize()
    assert same(out, first)
    outs, graphs = [torch.empty_like(first) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zs.zs_mx4_matvec(x, held, o)
        graphs.append(g)
    for g in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            g.replay()
    torch.cuda.synchronize()
    assert all(same(o, first) for o in outs)
    late, codes = torch.zeros_like(x), dict(held, codes=torch.zeros_like(held["codes"]))
    zs.zs_test_late_copy(late, x, x.nbytes // 16 * 16, 3_000_000)
    zs.zs_mx4_matvec(late, held, out)
    zs.zs_test_late_copy(codes["codes"], held["codes"], held["codes"].nbytes, 3_000_000)
    zs.zs_mx4_matvec(x, codes, outs[0])
    torch.cuda.synchronize()
    assert same(out, first) and same(outs[0], first)


def test_refused_tensors():
    held, w = weight(40, 64, np.random.default_rng(0))
    x, out = torch.ones(3, 64, device="cuda"), torch.empty(3, 40, device="cuda")
    for a in ((x.cpu(), held, out), (x, held, out.cpu()), (x[:2], held, out), (x.t(), held, out), (x.double(), held, out), (x, held, torch.empty(3, 41, device="cuda")),
              (torch.ones(3, 128, device="cuda"), held, out), (x, dict(held, codes=held["codes"].cpu()), out)):
        with pytest.raises((ValueError, TypeError)):
            zs.zs_mx4_matvec(*a)
