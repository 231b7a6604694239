"""Microscaled 4-bit matrices on the GPU: quantiser, values and product, against 64-bit definitions.

The quantiser and the values are exact (powers of two and a table): compared
bit for bit.  The product's tolerance, derived: every product of two codes and
its scales is exact; the tensor cores add 64 of them and the accumulator in
float32, each addition off by at most 2^-22 of the sum of magnitudes (one
rounding, or a truncation of two bits more), ceil(K/64) of them, and a split
adds up to 8 partial sums:
  |out - exact| <= (ceil(K/64) + 8) 2^-22 sum|a b| + u_out |exact|
with u_out = 2^-8 (bf16), 2^-11 (fp16; and 2^-25 absolute, its subnormals), 2^-24 (fp32).
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests import lowbit_ref as ref

pytestmark = pytest.mark.gpu
KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GUARD = 256


def room(rows, cols):
    """Buffers of a held matrix with guard bytes after them."""
    size = zs.zs_mx4_sizes(rows, cols)
    codes = torch.full((size["code_bytes"] + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((size["scale_bytes"] + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    return dict(codes=codes[:size["code_bytes"]], scales=scales[:size["scale_bytes"]]), (codes[size["code_bytes"]:], scales[size["scale_bytes"]:])


def ends_ok(ends):
    return all(bool((e == 0xA5).all()) for e in ends)


def put(code, byte):
    """A held matrix on the GPU from reference codes and scale bytes."""
    return dict(codes=torch.from_numpy(ref.pack(code)).cuda().contiguous(), scales=torch.from_numpy(ref.tile_scales(byte)).cuda())


def check_held(h, x):
    code, byte = ref.mx4(x)
    got = h["codes"].cpu().numpy().reshape(x.shape[0], -1)
    assert np.array_equal(h["scales"].cpu().numpy(), ref.tile_scales(byte))
    # -0 and 0 are one value
    a, b = ref.E2M1[ref.unpack(got)], ref.E2M1[code]
    assert np.array_equal(a, b)


def matrix(rows, cols, kind, seed, ld=None, offset=0):
    """A matrix as a view of a larger buffer of NaN: row stride ld, first element `offset` past its start."""
    ld = cols if ld is None else ld
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, cols), generator=g).float())
    buf = torch.full((offset + max(rows, 1) * ld,), float("nan"), dtype=KINDS[kind], device="cuda")
    v = buf[offset:].view(max(rows, 1), ld)[:rows, :cols]
    v.copy_(x.to(KINDS[kind]))
    return v


SHAPES = [(1, 1), (1, 32), (3, 31), (7, 33), (32, 32), (33, 64), (127, 129), (128, 128), (129, 257), (200, 1000), (1000, 200), (256, 256)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", list(KINDS))
def test_quantize(rows, cols, kind):
    for ld, offset in ((cols, 0), (cols + 8 + (-cols) % 8, 0), (cols + 3, 1)):
        x = matrix(rows, cols, kind, rows + cols, ld, offset)
        want = x.double().cpu().numpy()
        for along in (("rows",), ("cols",), ("rows", "cols")):
            (hr, er), (hc, ec) = room(rows, cols), room(cols, rows)
            zs.zs_mx4_quantize(x, rows=hr if "rows" in along else None, cols=hc if "cols" in along else None)
            torch.cuda.synchronize()
            assert ends_ok(er) and ends_ok(ec)
            if "rows" in along:
                check_held(hr, want)
            if "cols" in along:
                check_held(hc, want.T)


@pytest.mark.parametrize("extra,offset", [(4, 0), (3, 1)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_quantize_long(kind, extra, offset):
    """More tiles than a GPU takes at once: the same bytes as its parts one by one, which are few tiles each."""
    rows, cols, part = 20000, 1100, 2560
    x = matrix(rows, cols, kind, 5, cols + extra, offset)
    (hr, er), (hc, ec) = room(rows, cols), room(cols, rows)
    zs.zs_mx4_quantize(x, rows=hr, cols=hc)
    torch.cuda.synchronize()
    assert ends_ok(er) and ends_ok(ec)
    for r in range(0, rows, part):
        n = min(part, rows - r)
        (h, _), size = room(n, cols), zs.zs_mx4_sizes(n, cols)
        zs.zs_mx4_quantize(x[r:r + n], rows=h)
        at, per = r * size["row_bytes"], size["scale_bytes"] // (-(-n // 128)) * (r // 128)
        assert torch.equal(hr["codes"][at:at + size["code_bytes"]], h["codes"])
        assert torch.equal(hr["scales"][per:per + size["scale_bytes"]], h["scales"])
    for c in range(0, cols, 128):
        n = min(128, cols - c)
        (h, _), size = room(n, rows), zs.zs_mx4_sizes(n, rows)
        zs.zs_mx4_quantize(x[:, c:c + n], cols=h)
        at, per = c * size["row_bytes"], size["scale_bytes"] * (c // 128)
        assert torch.equal(hc["codes"][at:at + size["code_bytes"]], h["codes"])
        assert torch.equal(hc["scales"][per:per + size["scale_bytes"]], h["scales"])


@pytest.mark.parametrize("kind", list(KINDS))
def test_quantize_ties_and_ends(kind):
    """Every midpoint of the grid, both neighbours of each, values that saturate, signs and zeros."""
    grid = ref.E2M1[:8]
    mids = (grid[:-1] + grid[1:]) / 2
    eps = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[kind]
    v = np.concatenate([mids, mids * (1 - eps), mids * (1 + eps), grid, [6.5, 7.0, 7.5, 7.9]])
    v = np.concatenate([v, -v])
    x = np.zeros((len(v), 32))
    x[:, 0] = v
    x[:, 1] = 4.0                                    # scale 1 (values up to 8)
    x[:, 2] = 0.0
    t = torch.from_numpy(x).to(KINDS[kind]).cuda()
    assert torch.equal(t.double().cpu(), torch.from_numpy(x).to(KINDS[kind]).double())
    (h, e) = room(len(v), 32)
    zs.zs_mx4_quantize(t, rows=h)
    torch.cuda.synchronize()
    check_held(h, t.double().cpu().numpy())
    assert ends_ok(e)


@pytest.mark.parametrize("kind", list(KINDS))
def test_quantize_special(kind):
    """Groups of zeros, of the type's smallest and largest values, and with NaN and infinities."""
    dt = KINDS[kind]
    f = torch.finfo(dt)
    x = torch.zeros(70, 96, dtype=dt)
    x[1, :] = f.tiny
    x[2, 5] = f.smallest_normal * 2.0 ** -3          # subnormal
    x[3, :] = f.max
    x[4, 0], x[4, 40] = float("nan"), 1.0
    x[5, 33] = float("inf")
    x[6, 95] = float("-inf")
    x[7, 0] = -0.0
    t = x.cuda()
    (hr, er), (hc, ec) = room(70, 96), room(96, 70)
    zs.zs_mx4_quantize(t, rows=hr, cols=hc)
    out = torch.empty(70, 96, dtype=torch.float32, device="cuda")
    zs.zs_mx4_dequantize(hr, out)
    torch.cuda.synchronize()
    want = t.double().cpu().numpy()
    check_held(hr, want)
    check_held(hc, want.T)
    v = out.cpu().numpy()
    assert np.isnan(v[4, :32]).all() and np.all(v[4, 32:64] == want[4, 32:64])
    assert np.isnan(v[5, 32:64]).all() and np.isnan(v[6, 64:]).all() and not np.isnan(v[[0, 1, 2, 3, 7]]).any()
    assert ends_ok(er) and ends_ok(ec)


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (128, 96), (130, 1000)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_dequantize(rows, cols, kind):
    rng = np.random.default_rng(rows * cols)
    groups = -(-cols // 32)
    code = rng.integers(0, 16, (rows, groups * 32)).astype(np.uint8)
    byte = rng.integers(118, 136, (rows, groups)).astype(np.uint8)
    if kind == "fp32":
        byte[0, 0] = 1
    want = ref.mx4_values(code, byte)[:, :cols]
    h = put(code, byte)
    for ld in (cols, cols + 5, cols + (-cols) % 8 + 8):
        buf = torch.full((rows, ld), 77.0, dtype=KINDS[kind], device="cuda")
        zs.zs_mx4_dequantize(h, buf[:, :cols])
        assert np.array_equal(buf[:, :cols].double().cpu().numpy(), want)
        assert bool((buf[:, cols:] == 77.0).all())


def product(code_a, byte_a, code_b, byte_b, k, kind="fp32", ldo=None, offset=0, stream=None):
    m, n = code_a.shape[0], code_b.shape[0]
    ldo = n if ldo is None else ldo
    buf = torch.full((offset + m * ldo + 64,), 77.0, dtype=KINDS[kind], device="cuda")
    out = buf[offset:offset + m * ldo].view(m, ldo)[:, :n]
    a, b = put(code_a, byte_a), put(code_b, byte_b)
    zs.zs_mx4_matmul(a, b, k, out, stream=stream)
    torch.cuda.synchronize()
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[offset:offset + m * ldo].view(m, ldo)[:, :n] = False
    assert bool((buf[mask] == 77.0).all())
    return out.double().cpu().numpy()


def random_held(rng, rows, k, lo=120, hi=134):
    groups = -(-k // 32)
    code = rng.integers(0, 16, (rows, groups * 32)).astype(np.uint8)
    code[:, k:] = 0
    return code, rng.integers(lo, hi, (rows, groups)).astype(np.uint8)


# tokens 1 to several tiles; features and k that end inside a tile, a group, a stage
PRODUCTS = [(1, 1, 1), (1, 8, 32), (1, 129, 31), (2, 130, 33), (16, 128, 256), (17, 256, 257), (33, 100, 700), (64, 300, 512),
            (65, 128, 1000), (128, 257, 2048), (129, 1, 96), (130, 127, 64), (200, 300, 500), (256, 256, 4096), (300, 513, 1056),
            (1, 1024, 8192), (1000, 77, 40), (520, 9000, 288), (2600, 2600, 544),
            (129, 9800, 256), (385, 5121, 1300), (4097, 640, 3000), (1024, 2560, 512), (10100, 100, 300)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_exact(m, n, k):
    """Scales of 1: every sum is a multiple of 1/4 below 2^22, so any order gives the exact one."""
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    (ca, sa), (cb, sb) = random_held(rng, m, k, 127, 128), random_held(rng, n, k, 127, 128)
    want = ref.mx4_values(ca, sa) @ ref.mx4_values(cb, sb).T
    assert np.array_equal(product(ca, sa, cb, sb, k), want)


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("kind", list(KINDS))
def test_product(m, n, k, kind):
    rng = np.random.default_rng(m + n + k)
    (ca, sa), (cb, sb) = random_held(rng, m, k), random_held(rng, n, k, 112, 122)
    a, b = ref.mx4_values(ca, sa), ref.mx4_values(cb, sb)
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    u, least = {"bf16": (2.0 ** -8, 0), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 0)}[kind]
    tol = (-(-k // 64) + 8) * 2.0 ** -22 * mag * (1 + u) + u * np.abs(want) + least
    assert np.abs(want).max() < 60000
    for ldo, offset in ((n, 0), (n + 1, 1), (n + (-n) % 8 + 16, 0)):
        assert np.all(np.abs(product(ca, sa, cb, sb, k, kind, ldo, offset) - want) <= tol)


# parts of k that go around every ring of stages several times, by kernel and tile: 16, 32 and 64 tokens, 128, pairs of SMs
# with few stages and with many
@pytest.mark.parametrize("m,n,k", [(5, 9800, 2592), (20, 9801, 2592), (48, 9800, 4128), (100, 9900, 4128), (1290, 1801, 4128),
                                   (1290, 1801, 32800)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_product_deep(m, n, k, kind):
    """Scales of 1: sums are multiples of 1/4 below 2^22, exact in 32 bits in any order, and rounded once."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    table = torch.tensor(ref.E2M1, dtype=torch.float32, device="cuda")

    def held(rows):
        size = zs.zs_mx4_sizes(rows, k)
        codes = torch.randint(0, 256, (rows, size["row_bytes"]), dtype=torch.uint8, device="cuda", generator=g)
        values = table[torch.stack((codes & 15, codes >> 4), 2).long()].view(rows, k)
        return dict(codes=codes, scales=torch.full((size["scale_bytes"],), 127, dtype=torch.uint8, device="cuda")), values

    (a, va), (b, vb) = held(m), held(n)
    want = (va @ vb.T).to(KINDS[kind])
    for ldo in (n, n + (-n) % 8 + 8):
        out = torch.full((m, ldo), 77.0, dtype=KINDS[kind], device="cuda")
        zs.zs_mx4_matmul(a, b, k, out[:, :n])
        assert torch.equal(out[:, :n], want)
        assert bool((out[:, n:] == 77.0).all())
    assert zs.zs_device_wait_timeouts() == 0


@pytest.mark.parametrize("m,n", [(1, 200), (40, 130), (300, 260)])
def test_product_scales(m, n):
    """Each group's scale reaches its own row and elements: one nonzero element a row, all scales different."""
    k = 600
    rng = np.random.default_rng(m)
    groups = -(-k // 32)
    ca, cb = np.zeros((m, groups * 32), np.uint8), np.full((n, groups * 32), 2, np.uint8)      # B: ones
    at = rng.integers(0, k, m)
    ca[np.arange(m), at] = rng.integers(1, 16, m)
    sa = rng.integers(100, 150, (m, groups)).astype(np.uint8)
    sb = rng.integers(100, 150, (n, groups)).astype(np.uint8)
    want = ref.mx4_values(ca, sa) @ ref.mx4_values(cb, sb).T
    assert np.array_equal(product(ca, sa, cb, sb, k), want)


@pytest.mark.parametrize("m", [3, 200])
def test_product_nan(m):
    """A NaN group is NaN in its row of the product and nowhere else."""
    n, k = 150, 320
    rng = np.random.default_rng(1)
    (ca, sa), (cb, sb) = random_held(rng, m, k, 127, 128), random_held(rng, n, k, 127, 128)
    sa[1, 3], ca[1, 96:128] = 255, 0
    sb[77, 0], cb[77, :32] = 255, 0
    got = product(ca, sa, cb, sb, k)
    bad = np.zeros((m, n), bool)
    bad[1, :], bad[:, 77] = True, True
    assert np.array_equal(np.isnan(got), bad)
    with np.errstate(invalid="ignore"):
        want = ref.mx4_values(ca, sa) @ ref.mx4_values(cb, sb).T
    assert np.array_equal(got[~bad], want[~bad])


def test_product_of_nothing():
    out = torch.full((3, 5), 9.0, device="cuda")
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    zs.zs_mx4_matmul(dict(codes=e, scales=e), dict(codes=e, scales=e), 0, out)
    assert bool((out == 0).all())
    zs.zs_mx4_matmul(dict(codes=e, scales=e), dict(codes=e, scales=e), 64, torch.empty(0, 0, device="cuda"))
    x = torch.empty(0, 64, device="cuda")
    zs.zs_mx4_quantize(x, rows=dict(codes=e, scales=e))


def test_other_stream_and_graph():
    rng = np.random.default_rng(4)
    (ca, sa), (cb, sb) = random_held(rng, 70, 400, 127, 128), random_held(rng, 90, 400, 127, 128)
    want = ref.mx4_values(ca, sa) @ ref.mx4_values(cb, sb).T
    a, b = put(ca, sa), put(cb, sb)
    out = torch.empty(70, 90, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    zs.zs_mx4_matmul(a, b, 400, out, stream=s)
    s.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)
    out.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zs.zs_mx4_matmul(a, b, 400, out)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)
    assert zs.zs_device_wait_timeouts() == 0


def exact_matrix(rng, rows, cols):
    """Small whole numbers that 4 bits hold exactly along either dimension."""
    return rng.choice([-3.0, -2.0, -1.0, 0.0, 1.0, 2.0, 3.0], (rows, cols))


def linear(x, w, dy, kind=torch.float32):
    m, k, n = x.shape[0], x.shape[1], w.shape[0]
    h = {}
    for name, t in (("x", x), ("w", w), ("dy", dy)):
        h[name], h[name + "t"] = room(*t.shape)[0], room(*t.T.shape)[0]
        zs.zs_mx4_quantize(torch.from_numpy(t).float().cuda(), rows=h[name], cols=h[name + "t"])
    o = lambda a, b: torch.empty(a, b, dtype=kind, device="cuda")  # noqa: E731
    y = zs.zs_mx4_matmul(h["x"], h["w"], k, o(m, n))
    dx = zs.zs_mx4_matmul(h["dy"], h["wt"], n, o(m, k))
    dw = zs.zs_mx4_matmul(h["dyt"], h["xt"], m, o(n, k))
    torch.cuda.synchronize()
    return [t.double().cpu().numpy() for t in (y, dx, dw)]


@pytest.mark.parametrize("m,n,k", [(1, 40, 33), (50, 70, 90), (140, 129, 260)])
def test_gradients(m, n, k):
    """dx and dw of sum(dy * (x w^T)): the formula, and differences of the loss itself (all numbers exact)."""
    rng = np.random.default_rng(m + n + k)
    x, w, dy = exact_matrix(rng, m, k), exact_matrix(rng, n, k), exact_matrix(rng, m, n)
    y, dx, dw = linear(x, w, dy)
    assert np.array_equal(y, x @ w.T)
    assert np.array_equal(dx, dy @ w)
    assert np.array_equal(dw, dy.T @ x)
    loss = float((dy * y).sum())
    for _ in range(4):
        i, j, o = rng.integers(m), rng.integers(k), rng.integers(n)
        for at, t, grad in (((i, j), x, dx), ((o, j), w, dw)):
            d = -1.0 if t[at] > 0 else 1.0
            t[at] += d
            moved = float((dy * linear(x, w, dy)[0]).sum())
            t[at] -= d
            assert (moved - loss) / d == grad[at]


def test_gradients_of_rounded_matrices():
    """Matrices that 4 bits round: each product is of the values held along its own dimension."""
    rng = np.random.default_rng(8)
    m, n, k = 70, 90, 130
    x, w, dy = (rng.standard_normal(s) for s in ((m, k), (n, k), (m, n)))
    x, w, dy = (t.astype(np.float32).astype(np.float64) for t in (x, w, dy))
    v = lambda t: ref.mx4_values(*ref.mx4(t))[:, :t.shape[1]]  # noqa: E731
    for got, a, b in zip(linear(x, w, dy), (v(x), v(dy), v(dy.T)), (v(w), v(w.T), v(x.T))):
        tol = (-(-a.shape[1] // 64) + 8) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T) + 2.0 ** -24 * np.abs(a @ b.T)
        assert np.all(np.abs(got - a @ b.T) <= tol)


def test_past_32_bits():
    """2.3e9 elements: the last rows (of the transposed form: the last columns) equal those of a small matrix."""
    rows, cols, k = 70000, 32768, 64
    last = 539 * 128                                                   # the first row of the last scale tiles
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(9))
    (hr, er), (hc, ec) = room(rows, cols), room(cols, rows)
    zs.zs_mx4_quantize(x, rows=hr, cols=hc)
    assert ends_ok(er) and ends_ok(ec)
    (tail, _), size = room(rows - last, cols), zs.zs_mx4_sizes(rows - last, cols)
    zs.zs_mx4_quantize(x[last:].clone(), rows=tail)
    assert torch.equal(hr["codes"][-size["code_bytes"]:], tail["codes"])
    assert torch.equal(hr["scales"][-size["scale_bytes"]:], tail["scales"])
    (tail_c, _), size = room(128, rows), zs.zs_mx4_sizes(128, rows)
    zs.zs_mx4_quantize(x[:, -128:].clone(), cols=tail_c)
    assert torch.equal(hc["codes"][-size["code_bytes"]:], tail_c["codes"])
    assert torch.equal(hc["scales"][-size["scale_bytes"]:], tail_c["scales"])
    # values, into x
    zs.zs_mx4_dequantize(hr, x)
    out = torch.empty(rows - last, cols, dtype=torch.bfloat16, device="cuda")
    zs.zs_mx4_dequantize(tail, out)
    assert torch.equal(x[last:], out)
    # a product into x
    a, b = x[:, :k].clone(), x[:cols, k:2 * k].clone()
    (ha, _), (hb, _), (ta, _) = room(rows, k), room(cols, k), room(rows - last, k)
    for m, h in ((a, ha), (b, hb), (a[last:], ta)):
        zs.zs_mx4_quantize(m, rows=h)
    zs.zs_mx4_matmul(ha, hb, k, x)
    zs.zs_mx4_matmul(ta, hb, k, out)
    assert torch.equal(x[last:], out)
