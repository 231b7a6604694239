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
