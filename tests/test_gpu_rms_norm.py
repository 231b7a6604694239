"""zs_rms_norm and zs_rms_norm_backward on the GPU against the formulas in 64 bits.

Tolerances, with U = 2^-24 (one float32 rounding) and H = half a step of the
matrix's type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32), from include/zs.h:
  sum     one float32 sum of two exact numbers, rounded: torch's bits
  rstd    the nearest float32 but for 2^-40: U (1 + 2^-14) of itself
  y       (h rstd) w of the rstd that came back: torch's bits
  held    zs_mx4_quantize's bytes of that y (or dx)
  slope   c is rounded once and its mean off by (2^-40 + U) of the magnitudes'
          mean: U because each g in it is a float32 product, rounded, while the
          reference takes the exact one (|sum (g' - g) x| <= U sum |g x|)
  dx      rstd (U |g| + 2 U |x c| + 2 U |g - x c| + |x| (2^-40 + U) rstd^2 mean|g x|)
          + U (|v| + |dx|) + H |dx|, v the product with rstd; and 2^-25 where fp16 is subnormal
  dw      (rows + 3) U sum |dy x rstd| + H |dw|: each sum in any order, three roundings of a term
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests.test_gpu_tensors import KINDS

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
LEAST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}     # half of the smallest number
FILL = 0xA5


class Mat:
    """rows x cols inside a larger, filled buffer: a row stride and an offset of its own."""

    def __init__(self, rows, cols, kind, values=None, extra=0, shift=0):
        size = torch.empty(0, dtype=KINDS[kind]).element_size()
        self.raw = torch.full(((rows * (cols + extra) + shift + 64) * size,), FILL, dtype=torch.uint8, device="cuda")
        self.t = self.raw.view(KINDS[kind])[shift:shift + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
        self.before = None
        if values is not None:
            self.t.copy_(values)

    def outside_ok(self):
        """Nothing but the matrix itself was written."""
        copy = self.raw.clone()
        size = self.t.element_size()
        view = copy.view(self.t.dtype)
        at = (self.t.data_ptr() - self.raw.data_ptr()) // size
        view[at:at + self.t.shape[0] * self.t.stride(0)].as_strided(self.t.shape, self.t.stride()).view(torch.int16 if size == 2 else torch.int32).fill_(0)
        want = torch.full_like(copy, FILL)
        want.view(self.t.dtype)[at:at + self.t.shape[0] * self.t.stride(0)].as_strided(self.t.shape, self.t.stride()) \
            .view(torch.int16 if size == 2 else torch.int32).fill_(0)
        return torch.equal(copy, want)


def room(rows, cols):
    """Buffers of a 4-bit matrix with 64 filled bytes behind each."""
    size = zs.zs_mx4_sizes(rows, cols)
    raw = [torch.full((size[k] + 64,), FILL, dtype=torch.uint8, device="cuda") for k in ("code_bytes", "scale_bytes")]
    return dict(codes=raw[0][:-64], scales=raw[1][:-64], raw=raw)


def same_held(got, y, way):
    """The whole of both buffers is what zs_mx4_quantize writes."""
    rows, cols = y.shape if way == "rows" else y.shape[::-1]
    want = room(rows, cols)
    zs.zs_mx4_quantize(y, **{way: want})
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(got["raw"], want["raw"]))


def same(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    nan = torch.isnan(a) & torch.isnan(b)
    return bool((nan | (a.contiguous().view(kind) == b.contiguous().view(kind))).all())


def call(x, w, eps, residual=None, inplace=False, out=True, held=("rows", "cols"), kind=None, extra=0, shift=0, **kw):
    rows, cols = x.shape
    got = dict(rstd=torch.full((rows,), 7.0, device="cuda"))
    if residual is not None:
        got["sum"] = residual if inplace else Mat(rows, cols, kind, extra=extra, shift=shift)
    if out:
        got["out"] = Mat(rows, cols, kind, extra=extra, shift=shift)
    for way in held:
        got[way] = room(rows, cols) if way == "rows" else room(cols, rows)
    zs.zs_rms_norm(x, w, eps, got["rstd"], residual=None if residual is None else residual.t, sum=got["sum"].t if residual is not None else None,
                   out=got["out"].t if out else None, rows=got.get("rows"), cols=got.get("cols"), **kw)
    torch.cuda.synchronize()
    return got


def check_forward(x, r, w, eps, got):
    """x, r, w: what went in (r or None); rstd of rows whose formula is finite."""
    h = x.float() if r is None else x.float() + r.float()
    if r is not None:
        assert same(got["sum"].t, h.to(x.dtype)) and got["sum"].outside_ok()
    want = 1 / torch.sqrt(h.double().square().sum(1) / h.shape[1] + float(np.float32(eps)))
    rstd = got["rstd"].double()
    assert bool(((rstd - want).abs() <= want * U * (1 + 2.0 ** -14)).logical_or(rstd == want).logical_or(torch.isnan(rstd) & torch.isnan(want)).all())
    y = (h * got["rstd"][:, None] * w.float()).to(x.dtype)
    if "out" in got:
        assert same(got["out"].t, y) and got["out"].outside_ok()
    for way in ("rows", "cols"):
        if way in got:
            assert same_held(got[way], y, way), way


def data(rows, cols, kind, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * rows + cols)
    x = torch.randn(rows, cols, device="cuda", generator=g) * scale
    x = torch.where(torch.rand(cols, device="cuda", generator=g) < 0.02, 20 * x, x)
    return x.to(KINDS[kind]), g


COLS = [1, 7, 31, 32, 33, 250, 256, 257, 513, 777, 1024, 1490, 2049, 4096, 4104, 8200, 12288, 12289, 16392]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_forward(cols, kind):
    for rows, residual, extra, shift, out, held in ((33, True, 0, 0, True, ("rows", "cols")), (5, False, 0, 0, True, ()), (130, True, 3, 1, True, ("rows",)),
                                                    (65, False, 8, 0, False, ("cols",)), (1, True, 0, 0, True, ("rows",))):
        x, g = data(rows, cols, kind)
        r = Mat(rows, cols, kind, torch.randn(rows, cols, device="cuda", generator=g), extra, shift) if residual else None
        w = (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(KINDS[kind if rows != 5 else "fp32"])
        xm = Mat(rows, cols, kind, x, extra, shift)
        got = call(xm.t, w, 1e-5, r, out=out, held=held, kind=kind, extra=extra, shift=shift)
        check_forward(x, None if r is None else r.t, w, 1e-5, got)


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 127, 129, 256, 257, 1000])
@pytest.mark.parametrize("cols", [64, 320])
def test_forward_rows(rows, cols):
    """The last tile of rows, padding scales among it; many rows a CTA."""
    x, g = data(rows, cols, "bf16")
    w = torch.randn(cols, device="cuda", generator=g).bfloat16()
    for held in (("rows",), ("rows", "cols")):
        for out in (False, True):
            check_forward(x, None, w, 1e-6, call(x, w, 1e-6, out=out, held=held, kind="bf16"))


@pytest.mark.parametrize("cols", [96, 4096, 8192, 13000, 20000])
@pytest.mark.parametrize("held", [("rows",), ("rows", "cols")])
def test_in_place(cols, held):
    """The new stream in the old one's memory, or in x's."""
    for kind in ("bf16", "fp32"):
        x, g = data(40, cols, kind)
        old = torch.randn(40, cols, device="cuda", generator=g).to(KINDS[kind])
        w = torch.ones(cols, device="cuda")
        r = Mat(40, cols, kind, old)
        got = call(x, w, 1e-5, r, inplace=True, held=held, kind=kind)
        check_forward(x, old, w, 1e-5, got)
        xm, r = Mat(40, cols, kind, x), Mat(40, cols, kind, old)
        got = dict(rstd=torch.empty(40, device="cuda"), sum=xm, out=Mat(40, cols, kind))
        zs.zs_rms_norm(xm.t, w, 1e-5, got["rstd"], residual=r.t, sum=xm.t, out=got["out"].t)
        check_forward(x, old, w, 1e-5, got)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [200, 2048, 5000, 12400])
def test_range(kind, cols):
    """Magnitudes whose squares float32 does not have, rows of zeros, infinities and NaN in single rows."""
    x, g = data(64, cols, kind)
    x[3] *= 1e25
    x[4] *= 1e-25
    x[5] = 0
    x[6, cols // 2] = float("inf")
    x[7, 0] = float("nan")
    x[8, -1] = 3e38
    x[9] = 0
    x[9, 5] = 1e30
    x[10] = 2.0 ** 60
    w = torch.full((cols,), 1.5, device="cuda")
    for held in (("rows",), ("cols",)):
        got = call(x, w, 1e-5, out=True, held=held, kind=kind)
        check_forward(x, None, w, 1e-5, got)
    # without eps: the smallest squares that count, and a row of zeros, which is NaN
    got = call(x[[0, 3, 9, 10]].contiguous(), w, 0.0, kind=kind)
    check_forward(x[[0, 3, 9, 10]], None, w, 0.0, got)
    got = call(x[[5]].contiguous(), w, 0.0, held=(), kind=kind)
    assert bool(torch.isnan(got["out"].t).all())


def reference(dy, x, w, rstd, res):
    dy, x, w, r = dy.double(), x.double(), w.double(), rstd.double()[:, None]
    g = dy * w
    c = r * r * (g * x).mean(1, keepdim=True)
    v = (g - x * c) * r
    dx = v if res is None else v + res.double()
    return g, c, v, dx, (dy * x * r).sum(0)


def check_backward(dy, x, w, rstd, res, got, kind, dw_kind):
    g, c, v, dx, dw = reference(dy, x, w, rstd, res)
    r, x64 = rstd.double()[:, None], x.double()
    tol = r * (U * g.abs() + 2 * U * (x64 * c).abs() + 2 * U * (g - x64 * c).abs()
               + x64.abs() * (2.0 ** -40 + U) * r * r * (g * x64).abs().mean(1, keepdim=True)) + U * (v.abs() + dx.abs()) + HALF[kind] * dx.abs() + LEAST[kind]
    d = got["dx"].t.double()
    assert bool(((d - dx).abs() <= tol).all()), float(((d - dx).abs() / tol).max())
    assert got["dx"].outside_ok()
    if "dw" in got:
        tol = (len(dy) + 3) * U * (dy.double() * x64 * r).abs().sum(0) + HALF[dw_kind] * dw.abs() + LEAST[dw_kind]
        assert bool(((got["dw"].double() - dw).abs() <= tol).all())
    for way in ("rows", "cols"):
        if way in got:
            assert same_held(got[way], got["dx"].t, way), way


def back(dy, x, w, rstd, res, kind, dw_kind="fp32", dw=True, held=(), extra=0, shift=0, into=None):
    rows, cols = x.shape
    got = dict(dx=Mat(rows, cols, kind, extra=extra, shift=shift) if into is None else into)
    need = zs.zs_rms_norm_scratch(rows, cols)
    scratch = torch.full((need + 64,), FILL, dtype=torch.uint8, device="cuda")
    if dw:
        got["dw"] = torch.full((cols,), 7.0, device="cuda").to(KINDS[dw_kind])
    for way in held:
        got[way] = room(rows, cols) if way == "rows" else room(cols, rows)
    zs.zs_rms_norm_backward(dy, x, w, rstd, got["dx"].t, residual=res, dw=got.get("dw"), scratch=scratch,
                            rows=got.get("rows"), cols=got.get("cols"))
    torch.cuda.synchronize()
    assert bool((scratch[need:] == FILL).all())
    return got


def back_data(rows, cols, kind, w_kind, seed=0):
    x, g = data(rows, cols, kind, seed)
    dy = (torch.randn(rows, cols, device="cuda", generator=g) * 1e-3).to(KINDS[kind])
    res = (torch.randn(rows, cols, device="cuda", generator=g) * 1e-3).to(KINDS[kind])
    w = (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(KINDS[w_kind])
    rstd = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    return dy, x, w, rstd, res


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind,w_kind", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_backward(cols, kind, w_kind):
    for rows, with_res, extra, shift, held, dw in ((33, True, 0, 0, ("rows", "cols"), True), (130, False, 3, 1, ("rows",), True), (1, True, 0, 0, (), True),
                                                   (70, True, 8, 0, ("cols",), False)):
        dy, x, w, rstd, res = back_data(rows, cols, kind, w_kind)
        got = back(Mat(rows, cols, kind, dy, extra, shift).t, x, w, rstd, res if with_res else None, kind, w_kind, dw, held, extra, shift)
        check_backward(dy, x, w, rstd, res if with_res else None, got, kind, w_kind)


@pytest.mark.parametrize("rows", [2, 31, 32, 129, 256, 257, 2000, 5000])
@pytest.mark.parametrize("cols", [64, 4500])
def test_backward_rows(rows, cols):
    """Several row blocks a cluster, and the weight's gradient over all of them, the same bits twice."""
    dy, x, w, rstd, res = back_data(rows, cols, "bf16", "bf16")
    dy[rows // 2:rows // 2 + 3] = 0                    # rows that no loss reaches
    got = back(dy, x, w, rstd, res, "bf16", "bf16", held=("rows", "cols"))
    check_backward(dy, x, w, rstd, res, got, "bf16", "bf16")
    again = back(dy, x, w, rstd, res, "bf16", "bf16", held=("rows",))
    assert same(got["dx"].t, again["dx"].t)
    assert same(got["dw"], again["dw"])


@pytest.mark.parametrize("cols", [700, 13000])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_backward_in_place(cols, kind):
    dy, x, w, rstd, res = back_data(50, cols, kind, kind)
    want = back(dy, x, w, rstd, res, kind, kind)
    for name in ("dy", "res"):
        m = Mat(50, cols, kind, dy if name == "dy" else res)
        got = back(m.t if name == "dy" else dy, x, w, rstd, m.t if name == "res" else res, kind, kind, into=m)
        assert same(got["dx"].t, want["dx"].t) and same(got["dw"], want["dw"])


@pytest.mark.parametrize("cols", [40, 600])
def test_gradients_by_differences(cols):
    """The reference against central differences in 64 bits, and the kernels' own float32 results against theirs."""
    dy, x, w, rstd, _ = back_data(3, cols, "fp32", "fp32", seed=5)
    eps = float(np.float32(1e-5))
    x64, w64, dy64 = x.double(), w.double(), dy.double()

    def loss(x, w):
        return (dy64 * (x / (x.square().mean(1, keepdim=True) + eps).sqrt() * w)).sum()

    _, _, _, dx, dw = reference(dy, x, w, (x64.square().mean(1) + eps).rsqrt(), None)
    got = back(dy, x, w, rstd, None, "fp32")
    g = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(5):
        ux, uw = torch.randn(x.shape, device="cuda", generator=g).double(), torch.randn(w.shape, device="cuda", generator=g).double()
        # third derivatives of the norm are bounded by about 20 |dy| |w| rstd^3 |u|^3 for unit rows; step^2 of them is far below 1e-6
        step = 1e-4
        by_x, by_w = ((loss(x64 + step * ux, w64) - loss(x64 - step * ux, w64)) / (2 * step), (loss(x64, w64 + step * uw) - loss(x64, w64 - step * uw)) / (2 * step))
        size_x, size_w = (dx.abs() * ux.abs()).sum(), (dw.abs() * uw.abs()).sum()
        assert abs(by_x - (dx * ux).sum()) <= 1e-5 * size_x and abs(by_w - (dw * uw).sum()) <= 1e-5 * size_w
        assert abs(by_x - (got["dx"].t.double() * ux).sum()) <= 2e-5 * size_x and abs(by_w - (got["dw"].double() * uw).sum()) <= 2e-5 * size_w


def test_nothing():
    e = torch.empty(0, 64, device="cuda")
    zs.zs_rms_norm(e, torch.ones(64, device="cuda"), 1e-5, torch.empty(0, device="cuda"), out=e)
    n = torch.empty(5, 0, device="cuda")
    zs.zs_rms_norm(n, torch.ones(0, device="cuda"), 1e-5, torch.empty(5, device="cuda"), out=n)
    dw = torch.full((64,), 3.0, device="cuda")
    zs.zs_rms_norm_backward(e, e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), e, dw=dw,
                            scratch=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert bool((dw == 0).all())


def test_long_matrix():
    """Offsets past 2^31 elements."""
    rows, cols = (1 << 31) // 4096 + 40, 4096
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    x[-2, ::2] = 3.0
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    out = torch.empty_like(x)
    held = room(cols, rows)
    zs.zs_rms_norm(x, w, 1e-5, rstd, out=out, cols=held)
    tail = slice(rows - 70, rows)
    y = (x[tail].float() * rstd[tail][:, None]).bfloat16()
    want = 1 / torch.sqrt(x[tail].double().square().mean(1) + float(np.float32(1e-5)))
    assert bool(((rstd[tail].double() - want).abs() <= want * U * (1 + 2.0 ** -14)).all()) and same(out[tail], y)
    assert same_held(held, out, "cols")
    del held, out
    dx = torch.empty_like(x)
    dw = torch.empty(cols, device="cuda")
    zs.zs_rms_norm_backward(x, x, w, rstd, dx, dw=dw, scratch=torch.empty(zs.zs_rms_norm_scratch(rows, cols), dtype=torch.uint8, device="cuda"))
    got = dict(dx=Mat(70, cols, "bf16", dx[tail]))
    check_backward(x[tail], x[tail], w, rstd[tail], None, got, "bf16", "fp32")
    assert bool(torch.isfinite(dw).all()) and float(dw.min()) > 1e5


def test_streams_graphs_and_the_kernel_before():
    rows, cols = 200, 1100
    dy, x, w, rstd, res = back_data(rows, cols, "bf16", "bf16")
    r = Mat(rows, cols, "bf16", res)
    first = call(x, w, 1e-5, r, kind="bf16")
    back_first = back(dy, x, w, rstd, res, "bf16", held=("rows", "cols"))

    def all_of(src, into, scratch, stream=None):
        zs.zs_rms_norm(src, w, 1e-5, into["rstd"], residual=res, sum=into["sum"], out=into["out"], rows=into["rows"], cols=into["cols"], stream=stream)
        zs.zs_rms_norm_backward(dy, src, w, rstd, into["dx"], residual=res, dw=into["dw"], scratch=scratch, rows=into["rows2"], cols=into["cols2"], stream=stream)

    def fresh():
        e = lambda: torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return dict(rstd=torch.empty(rows, device="cuda"), sum=e(), out=e(), dx=e(), dw=torch.empty(cols, device="cuda"), rows=room(rows, cols),
                    cols=room(cols, rows), rows2=room(rows, cols), cols2=room(cols, rows))

    def equal(into):
        torch.cuda.synchronize()
        assert same(into["sum"], first["sum"].t) and same(into["out"], first["out"].t) and torch.equal(into["rstd"], first["rstd"])
        assert same(into["dx"], back_first["dx"].t) and torch.equal(into["dw"], back_first["dw"])
        for a, b in (("rows", first), ("cols", first)):
            assert all(torch.equal(p, q) for p, q in zip(into[a]["raw"], b[a]["raw"]))
            assert all(torch.equal(p, q) for p, q in zip(into[a + "2"]["raw"], back_first[a]["raw"]))

    scratch = lambda: torch.empty(zs.zs_rms_norm_scratch(rows, cols), dtype=torch.uint8, device="cuda")  # noqa: E731
    into, s = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    all_of(x, into, scratch(), stream=s)
    equal(into)
    graphs, outs, keep = [], [], []
    for _ in range(2):
        outs.append(fresh())
        keep.append(scratch())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_of(x, outs[-1], keep[-1])
        graphs.append(g)
    for g in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        equal(o)
    # behind a kernel that lets its dependents begin, and writes x only later
    late, into = torch.zeros_like(x), fresh()
    zs.zs_test_late_copy(late, x, x.nbytes, 3_000_000)
    all_of(late, into, scratch())
    equal(into)


def test_refused_tensors():
    x, w, rstd = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    out = torch.empty_like(x)
    for kw in (dict(out=out.bfloat16()), dict(out=out[:, :32]), dict(residual=out), dict(sum=out, out=torch.empty_like(x)), dict(),
               dict(out=out, rows=dict(codes=torch.empty(3, dtype=torch.uint8, device="cuda"), scales=torch.empty(3, dtype=torch.uint8, device="cuda")))):
        with pytest.raises((ValueError, zs.ZsError)):
            zs.zs_rms_norm(x, w, 1e-5, rstd, **kw)
    for a in ((x.cpu(), w, rstd), (x, w.cpu(), rstd), (x, w[:63], rstd), (x, w, rstd.double()), (x, w, rstd[:3]), (x[0], w, rstd), (x.t(), w, rstd)):
        with pytest.raises((ValueError, TypeError)):
            zs.zs_rms_norm(a[0], a[1], 1e-5, a[2], out=out)
    with pytest.raises(ValueError):
        zs.zs_rms_norm_backward(x, x, w, rstd, out, torch.empty(16, dtype=torch.uint8, device="cuda"), dw=w)
    with pytest.raises(ValueError):
        zs.zs_rms_norm_backward(x[:3], x, w, rstd, out, torch.empty(1 << 16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("cols", [1, 31, 256, 500, 512, 513, 1490, 2048, 2056, 4096, 4099, 8192, 8193])
@pytest.mark.parametrize("kind,w_kind", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_backward_whole(cols, kind, w_kind):
    """dx that is not held: one reading where a row fits the registers; the same bits twice."""
    for rows, with_res, extra, shift, dw in ((1, True, 0, 0, True), (7, False, 3, 1, True), (9, True, 8, 0, True), (700, True, 0, 0, True), (2500, True, 5, 3, False)):
        dy, x, w, rstd, res = back_data(rows, cols, kind, w_kind, seed=rows)
        dy[rows // 2] = 0                              # a row that no loss reaches
        m = Mat(rows, cols, kind, dy, extra, shift)
        got = back(m.t, x, w, rstd, res if with_res else None, kind, w_kind, dw, (), extra, shift)
        check_backward(dy, x, w, rstd, res if with_res else None, got, kind, w_kind)
        again = back(m.t, x, w, rstd, res if with_res else None, kind, w_kind, dw, (), extra, shift)
        assert same(got["dx"].t, again["dx"].t) and (not dw or same(got["dw"], again["dw"]))


@pytest.mark.parametrize("cols", [40, 1490, 2048, 6000])
@pytest.mark.parametrize("held", [(), ("cols",)])
def test_backward_range(cols, held):
    """Rows whose products leave float32, and rows that are not finite, beside ordinary ones."""
    rows = 45
    dy, x, w, rstd, _ = back_data(rows, cols, "bf16", "fp32", seed=8)
    big = [1, 6, 17]
    x[big] = (x[big].float() * 2.0 ** 62).bfloat16()   # x x past 2^124: mean(g x) is float32's in the end
    rstd[big] = rstd[big] * 2.0 ** -62
    dy[big] = (dy[big].float() * 2.0 ** 70).bfloat16()
    x[20, cols // 2] = float("inf")
    dy[33, 0] = float("nan")
    dy[40, cols - 1] = float("-inf")
    got = back(dy, x, w, rstd, None, "bf16", "fp32", False, held)
    finite = torch.tensor([r not in (20, 33, 40) for r in range(rows)], device="cuda")
    rest = dict(dx=Mat(int(finite.sum()), cols, "bf16", got["dx"].t[finite]))
    check_backward(dy[finite], x[finite], w, rstd[finite], None, rest, "bf16", "fp32")
    # c is an infinity or NaN: of 20 and 33 and 40 nothing stays finite
    assert not bool(torch.isfinite(got["dx"].t[~finite]).any())


def test_backward_whole_streams_and_graphs():
    """Two captured graphs with a scratch each, replayed at once, and a call on another stream."""
    rows, cols = 900, 1490
    dy, x, w, rstd, res = back_data(rows, cols, "fp16", "fp32")
    want = back(dy, x, w, rstd, res, "fp16")
    runs = []
    for _ in range(3):
        dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
        scratch = torch.empty(zs.zs_rms_norm_scratch(rows, cols), dtype=torch.uint8, device="cuda")
        runs.append((dx, dw, scratch))
    torch.cuda.synchronize()
    graphs = []
    for dx, dw, scratch in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zs.zs_rms_norm_backward(dy, x, w, rstd, dx, scratch, residual=res, dw=dw)
        graphs.append(g)
    for g in graphs:
        with torch.cuda.stream(torch.cuda.Stream()):
            g.replay()
    dx, dw, scratch = runs[2]
    zs.zs_rms_norm_backward(dy, x, w, rstd, dx, scratch, residual=res, dw=dw, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for dx, dw, _ in runs:
        assert same(dx, want["dx"].t) and same(dw, want["dw"])
