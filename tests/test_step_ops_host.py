"""Refusals of the calls around the 4-bit products (no GPU: argument errors enqueue nothing)."""
import pytest

import zero_sharded_optimizer_bucket_gb300 as zs
from tests.test_lowbit_host import A16, refuses, tensor


def test_norm_and_clip_refusals():
    lst = zs.zs_build_tensors([tensor()], state_bits=8)
    a, odd = A16, A16 + 2
    refuses(zs.zs_norm_tensors, lst, a, 1.0, a, a, a, status=zs.ZS_ESTATE)
    refuses(zs.zs_clip_tensors, lst, a, status=zs.ZS_ESTATE)
    for bad in ((None, a, a, a), (A16 + 4, a, a, a), (a, None, a, a), (a, a, None, a), (a, a, a, None), (a, odd, a, a), (a, a, odd, a), (a, a, a, odd)):
        refuses(zs.zs_norm_tensors, lst, bad[0], 1.0, *bad[1:])
    refuses(zs.zs_clip_tensors, lst, None)
    refuses(zs.zs_clip_tensors, lst, odd)
    refuses(zs.zs_clip_tensors, lst, a, odd)
    for scaler in (zs.make_loss_scaler(None), zs.make_loss_scaler(odd), zs.make_loss_scaler(a, None, scale_window=1),
                   zs.make_loss_scaler(a, a, scale_factor=1.0), zs.make_loss_scaler(a, a, min_scale=0.0)):
        refuses(zs.zs_norm_tensors, lst, a, 1.0, a, a, a, scaler=scaler)
    with pytest.raises(zs.ZsError):
        zs._check(zs._lib.zs_norm_tensors(None, a, 1.0, None, a, a, a, None), "zs_norm_tensors")
    with pytest.raises(zs.ZsError):
        zs._check(zs._lib.zs_clip_tensors(None, a, None, None), "zs_clip_tensors")
    zs.zs_clip_tensors(zs.zs_build_tensors([]), a)      # nothing to do, no launch


def call(name, *a):
    got = getattr(zs._lib, name)(*a)
    assert got == zs.ZS_EINVAL, (name, a, got)
    assert zs.zs_last_error() != ""


def test_rms_norm_refusals():
    a = A16
    good = dict(x=a, ldx=64, residual=a, ldr=64, weight=a, weight_dtype=0, rows=4, cols=64, dtype=0, eps=1e-5, sum=a, lds=64, out=a, ldo=64,
                rstd=a, r_codes=a, r_scales=a, c_codes=a, c_scales=a, stream=None)
    for bad in (dict(x=None), dict(x=a + 1), dict(ldx=63), dict(ldr=63), dict(lds=63), dict(ldo=63), dict(sum=None), dict(residual=None), dict(weight=None),
                dict(weight=a + 1), dict(weight_dtype=3), dict(dtype=-1), dict(dtype=3), dict(rows=-1), dict(cols=1 << 31), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(out=a + 1), dict(rstd=None), dict(rstd=a + 2), dict(r_codes=None), dict(r_scales=None),
                dict(r_codes=a + 8), dict(c_codes=a + 8), dict(c_scales=None), dict(c_scales=a + 4),
                dict(out=None, r_codes=None, r_scales=None, c_codes=None, c_scales=None)):
        call("zs_rms_norm", *dict(good, **bad).values())
    back = dict(dy=a, lddy=64, x=a, ldx=64, weight=a, weight_dtype=0, rstd=a, residual=a, ldr=64, rows=4, cols=64, dtype=0, dx=a, lddx=64, dw=a,
                dw_dtype=2, scratch=a, r_codes=a, r_scales=a, c_codes=a, c_scales=a, stream=None)
    for bad in (dict(dy=None), dict(dy=a + 1), dict(lddy=63), dict(x=None), dict(ldx=63), dict(weight=None), dict(weight_dtype=-1), dict(rstd=None),
                dict(rstd=a + 1), dict(ldr=63), dict(rows=1 << 31), dict(cols=-1), dict(dtype=3), dict(dx=None), dict(lddx=63), dict(dw=a + 2),
                dict(dw_dtype=3), dict(scratch=None), dict(scratch=a + 8), dict(r_scales=None), dict(c_codes=None), dict(c_codes=a + 1)):
        call("zs_rms_norm_backward", *dict(back, **bad).values())
    refuses(zs.zs_rms_norm_scratch, -1, 4)
    refuses(zs.zs_rms_norm_scratch, 4, 1 << 31)
    assert zs.zs_rms_norm_scratch(0, 64) == 0 and zs.zs_rms_norm_scratch(64, 0) == 0
    # a float a row, and no more than a few hundred parts of the weight's gradient
    for rows, cols in ((1, 1), (33, 100), (5000, 4096), (1 << 20, 8192), (1 << 20, 20000)):
        assert 4 * (rows + cols) <= zs.zs_rms_norm_scratch(rows, cols) <= 4 * (rows + 304 * (cols + 511))


def test_matvec_refusals():
    a = A16
    good = dict(m=3, n=40, k=64, x=a, ldx=64, dtype=0, codes=a, scales=a, out=a, ldo=40, out_dtype=2, stream=None)
    for bad in (dict(m=-1), dict(m=zs.ZS_MATVEC_MAX_TOKENS + 1), dict(n=-1), dict(n=1 << 31), dict(k=1 << 31), dict(x=None), dict(x=a + 1), dict(ldx=63),
                dict(dtype=3), dict(dtype=2, x=a + 2), dict(codes=None), dict(codes=a + 8), dict(scales=None), dict(scales=a + 1), dict(out=None),
                dict(out=a + 2), dict(ldo=39), dict(out_dtype=-1)):
        call("zs_mx4_matvec", *dict(good, **bad).values())


def test_scratch_of_a_larger_matrix_does_for_a_smaller_one():
    rows = [1, 2, 7, 8, 9, 31, 33, 151, 152, 153, 303, 304, 305, 607, 608, 609, 2432, 8191, 8192, 8193, 1 << 20]
    cols = [1, 511, 512, 513, 1024, 2047, 2048, 2049, 4095, 4096, 4097, 4608, 4609, 8191, 8192, 8193, 8705, 16384, 32768, 1 << 18]
    need = [[zs.zs_rms_norm_scratch(r, c) for c in cols] for r in rows]
    for i in range(len(rows)):
        for j in range(len(cols)):
            assert i == 0 or need[i - 1][j] <= need[i][j], (rows[i], cols[j])
            assert j == 0 or need[i][j - 1] <= need[i][j], (rows[i], cols[j])


def test_clipping_of_gradients_that_overlap_is_refused():
    """A gradient that is in the list twice would be multiplied once or twice, as its chunks happen to meet."""
    for grads in ((A16, A16), (A16 + 2000, A16, A16 + 3998), (A16 + 1998, A16), (A16, A16 + 40000, A16 + 40016)):
        lst = zs.zs_build_tensors([tensor(grad=g) for g in grads], state_bits=8)
        refuses(zs.zs_clip_tensors, lst, A16)
    for grads in ((A16,), (A16 + 2000, A16, A16 + 4000), (A16 + 2002, A16)):
        lst = zs.zs_build_tensors([tensor(grad=g) for g in grads], state_bits=8)
        refuses(zs.zs_clip_tensors, lst, A16, status=zs.ZS_ESTATE)       # as far as the upload
    lst = zs.zs_build_tensors([tensor(), tensor(numel=0)], state_bits=8)
    refuses(zs.zs_clip_tensors, lst, A16, status=zs.ZS_ESTATE)
