"""The sums over a row behind zs_rms_norm and zs_rms_norm_backward, where one
value leads a row, and the kernels of rows of more than 8192 columns.

Tolerances, with U = 2^-24 and from include/zs.h:
  rstd    the nearest float32 to the formula's value, in rows that lie more than
          2^-38 of it from the middle of two (the reference's own error: 2^-50)
  small   rstd of rows whose squares float32 does not have: as the other rows (check_forward)
  slope   of a column whose dy is 0, x 1 and rstd 1, dx is -c: 2^-36 of the mean
          of the magnitudes, and half a step of c
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests.test_gpu_rms_norm import HALF, U, back, back_data, call, check_backward, check_forward, data
from tests.test_gpu_tensors import KINDS

pytestmark = pytest.mark.gpu


def led_rows(cols, rows, near, far, seed):
    """Rows [rows, cols] of float32 whose first value leads and whose rstd (eps 0) lies between near and far, relative, from
    the middle of two floats; and the nearest floats."""
    rng = np.random.default_rng(seed)
    found, want = [], []
    places = [c for c in range(1, cols) if c % 256 < 8]
    while len(found) < rows:
        tail = np.float32(2.0 ** -rng.uniform(8.5, 9.5))
        first = (1 + rng.random(1 << 18)).astype(np.float32)
        s = first.astype(np.float64) ** 2 + len(places) * float(tail) ** 2
        r = 1 / np.sqrt(s / cols)
        f = r.astype(np.float32)
        # the middle on r's side of f
        other = np.nextafter(f, np.where(r > f, np.float32(np.inf), np.float32(0)))
        off = np.abs((f.astype(np.float64) + other.astype(np.float64)) / 2 - r) / r
        for i in np.nonzero((off >= near) & (off <= far))[0]:
            row = np.zeros(cols, np.float32)
            row[places], row[0] = tail, first[i]
            found.append(row)
            want.append(f[i])
    return torch.from_numpy(np.stack(found[:rows])).cuda(), torch.tensor(np.array(want[:rows])).cuda()


@pytest.mark.parametrize("cols", [250, 512, 1024, 2048, 4096, 4099, 8192, 8191, 12288, 16384, 16377, 20000, 70000])
@pytest.mark.parametrize("held", [(), ("cols",)])
def test_a_value_that_leads_its_row(cols, held):
    x, want = led_rows(cols, 64, 2.0 ** -38, 2.0 ** -35, cols)
    w = torch.ones(cols, device="cuda")
    got = call(x, w, 0.0, held=held, kind="fp32")
    assert torch.equal(got["rstd"], want), int((got["rstd"] != want).sum())


@pytest.mark.parametrize("cols", [300, 512, 2048, 1490, 4096, 8192, 8191, 8200, 12288, 12289, 20000])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lead", [8, 14])
def test_leading_values_in_different_columns(cols, kind, lead):
    """Rows whose sum of g x is 0, of columns that come twice, once negated, and of a g and an x that lead, not together."""
    rows = 40
    g = torch.Generator(device="cuda").manual_seed(cols + lead)
    half = (cols - 1) // 2
    x, dy = (torch.randn(rows, half, device="cuda", generator=g).to(KINDS[kind]) for _ in range(2))
    for at in range(0, half - 1, 70):
        x[:, at], dy[:, at] = 2.0 ** lead * (1 + at % 3), x[:, at] * 2.0 ** -lead
        dy[:, at + 1], x[:, at + 1] = 2.0 ** lead, dy[:, at + 1] * 2.0 ** -lead
    turn = torch.randperm(half, device="cuda", generator=g)
    probe = torch.zeros(rows, cols - 2 * half, dtype=KINDS[kind], device="cuda")
    x, dy = torch.cat([x, x[:, turn], probe + 1], 1), torch.cat([dy, -dy[:, turn], probe], 1)
    got = back(dy.contiguous(), x.contiguous(), torch.ones(cols, device="cuda"), torch.ones(rows, device="cuda"), None, kind, dw=False)
    c = -got["dx"].t[:, -1].double()
    size = (dy.double() * x.double()).abs().mean(1)
    assert bool((c.abs() <= 2.0 ** -36 * size * (1 + HALF[kind])).all()), float((c.abs() / size).max())


@pytest.mark.parametrize("cols", [512, 4096, 8192, 12288, 12289])
def test_slope_of_ordinary_rows(cols):
    dy, x = (torch.randn(33, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(cols + i)) for i in range(2))
    dy[:, -1], x[:, -1] = 0, 1
    got = back(dy, x, torch.ones(cols, device="cuda"), torch.ones(33, device="cuda"), None, "fp32", dw=False)
    p = dy.double() * x.double()
    want = p.mean(1)
    assert bool(((got["dx"].t[:, -1].double() + want).abs() <= U * want.abs() + 2.0 ** -36 * p.abs().mean(1)).all())


@pytest.mark.parametrize("cols", [500, 4096, 8191, 8192, 9000, 12291])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("e", [-60, -63, -66, -90])
def test_slope_of_a_small_input(cols, kind, e):
    """rstd past 2^64, whose square float32 does not have."""
    dy, x, w, _, res = back_data(20, cols, kind, "fp32")
    x = (x.float() * 2.0 ** e).to(KINDS[kind])
    rstd = x.double().square().mean(1).rsqrt().float()
    check_backward(dy, x, w, rstd, res, back(dy, x, w, rstd, res, kind), kind, "fp32")


@pytest.mark.parametrize("cols", [250, 2048, 4099, 8192, 16384, 20000])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("held", [(), ("cols",)])
def test_rows_of_small_values(cols, kind, held):
    """Without eps, or with a tiny one: squares down to far below float32's least number."""
    x, g = data(40, cols, kind)
    for i, e in enumerate([0, -40, -48, -52, -55, -58, -62, -63, -64, -66, -70, -74, -80, -100, -115]):
        x[2 * i] = (x[2 * i].float() * 2.0 ** e).to(KINDS[kind])
    x[33] = 0
    x[33, cols // 2] = 2.0 ** -70
    x[35] = 2.0 ** -126
    for eps in (0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -110, 1e-30):
        got = call(x, torch.ones(cols, device="cuda"), eps, held=held, kind=kind)
        check_forward(x, None, torch.ones(cols, device="cuda"), eps, got)
    got = call(x, torch.ones(cols, device="cuda"), 3e38, held=held, kind=kind)
    check_forward(x, None, torch.ones(cols, device="cuda"), 3e38, got)


@pytest.mark.parametrize("cols", [250, 4099, 16384])
@pytest.mark.parametrize("held", [(), ("cols",)])
def test_large_eps(cols, held):
    """An eps near float32's largest number, beside means that count and ones that take the sum past it."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.rand(90, cols, device="cuda", generator=g) * 2.0 ** torch.linspace(50, 64, 90, device="cuda")[:, None]
    for eps in (1e36, 2.9e38, 3e38):
        got = call(x, torch.ones(cols, device="cuda"), eps, held=held, kind="fp32")
        check_forward(x, None, torch.ones(cols, device="cuda"), eps, got)
        want = 1 / torch.sqrt(x.double().square().mean(1) + float(np.float32(eps)))
        near = want.float()
        # half a step of want's binade, and 2^-38: further than that is not the nearest
        half = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), torch.frexp(want).exponent - 25)
        assert bool(((got["rstd"].double() - want).abs() <= half + 2.0 ** -38 * want).all()), int((got["rstd"] != near).sum())
