"""zs_rms_norm_backward of rows of more than 8192 columns, by tiles: several
blocks of 32 rows a CTA, rows that leave float32, offsets past 2^31.  Tolerances
as in test_gpu_rms_norm.py.
"""
import pytest
import torch

import tests.test_gpu_rms_norm as norm
import zero_sharded_optimizer_bucket_gb300 as zs
from tests.test_gpu_rms_norm import Mat, back, back_data, check_backward, room, same, same_held

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [8200, 8201, 12289])
@pytest.mark.parametrize("held", [(), ("cols",), ("rows", "cols")])
def test_range(cols, held):
    norm.test_backward_range(cols, held)


@pytest.mark.parametrize("rows", [8192, 8193, 8300, 16500])
@pytest.mark.parametrize("cols", [8200, 8195])
@pytest.mark.parametrize("kind,w_kind", [("bf16", "fp32"), ("fp32", "fp32")])
def test_several_blocks_a_cta(rows, cols, kind, w_kind):
    """256 CTAs of a column block share the blocks of 32 rows: dx, its forms and the weight's gradient over all of them."""
    dy, x, w, rstd, res = back_data(rows, cols, kind, w_kind)
    dy[rows - 40:rows - 2] = 0                         # a block of rows that no loss reaches, the last rows not among them
    first = None
    for held, with_res, extra, shift in (((), True, 0, 0), (("rows", "cols"), True, 0, 0), (("cols",), False, 3, 1), (("rows",), False, 8, 0)):
        got = back(Mat(rows, cols, kind, dy, extra, shift).t, x, w, rstd, res if with_res else None, kind, w_kind, True, held, extra, shift)
        check_backward(dy, x, w, rstd, res if with_res else None, got, kind, w_kind)
        if first is None:
            first = got
        elif with_res:                                 # the forms change nothing
            assert same(got["dx"].t, first["dx"].t) and same(got["dw"], first["dw"])


def test_long_matrix():
    """Offsets past 2^31 elements."""
    rows, cols = (1 << 31) // 8200 + 70, 8200
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    x[-2, ::2] = 3.0
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.ones(rows, device="cuda")
    rstd[-2:] = torch.tensor([0.4, 0.5], device="cuda")
    dx, dw, held = torch.empty_like(x), torch.empty(cols, device="cuda"), room(cols, rows)
    dy = torch.ones_like(x)
    dy[rows - 70:, ::3] = 0.5
    zs.zs_rms_norm_backward(dy, x, w, rstd, dx, torch.empty(zs.zs_rms_norm_scratch(rows, cols), dtype=torch.uint8, device="cuda"), dw=dw, cols=held)
    tail = slice(rows - 70, rows)
    check_backward(dy[tail], x[tail], w, rstd[tail], None, dict(dx=Mat(70, cols, "bf16", dx[tail])), "bf16", "fp32")
    assert same_held(held, dx, "cols")
    # rows - 70 of ones, and the tail's; every sum below 2^24 but for halves
    want = (dy[tail].double() * x[tail].double() * rstd[tail].double()[:, None]).sum(0) + (rows - 70)
    assert bool(((dw.double() - want).abs() <= (rows + 3) * norm.U * want).all())
