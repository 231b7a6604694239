"""Where the tensors of the low-memory calls may be: on the current device, or in pinned host memory, which it reaches."""
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs

pytestmark = pytest.mark.gpu
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def room(rows, cols, device="cuda"):
    size = zs.zs_mx4_sizes(rows, cols)
    return dict(codes=torch.empty(size["code_bytes"], dtype=torch.uint8, device=device),
                scales=torch.empty(size["scale_bytes"], dtype=torch.uint8, device=device))


def test_host_memory():
    x = torch.randn(130, 96)
    on, pinned = room(130, 96), room(130, 96)
    zs.zs_mx4_quantize(x.cuda(), rows=on)
    zs.zs_mx4_quantize(x.pin_memory(), rows=pinned)
    torch.cuda.synchronize()
    assert torch.equal(on["codes"], pinned["codes"]) and torch.equal(on["scales"], pinned["scales"])
    for call in (lambda: zs.zs_mx4_quantize(x, rows=on), lambda: zs.zs_mx4_quantize(x.cuda(), rows=room(130, 96, "cpu")),
                 lambda: zs.zs_mx4_dequantize(on, x), lambda: zs.zs_mx4_matmul(on, room(130, 96, "cpu"), 96, torch.empty(130, 130, device="cuda"))):
        with pytest.raises(ValueError, match="got cpu"):
            call()


def test_lists():
    t = {k: torch.randn(300, device="cuda") for k in ("grad", "master", "exp_avg")}
    t["exp_avg_sq"] = torch.rand(300, device="cuda")
    table = torch.empty(1 << 12, dtype=torch.uint8, device="cuda")
    for name in t:
        lst = zs.zs_build_tensors([dict(t, **{name: t[name].cpu()})])
        with pytest.raises(ValueError, match="got cpu"):
            zs.zs_tensors_upload(lst, table, table.numel())
    want = None
    for grad in (t["grad"], t["grad"].cpu().pin_memory()):
        own = dict({k: v.clone() for k, v in t.items()}, grad=grad)
        lst = zs.zs_build_tensors([own])
        zs.zs_tensors_upload(lst, table, table.numel())
        with pytest.raises(ValueError, match="got cpu"):
            zs.zs_adam_tensors(lst, HP, 1, torch.ones(1))
        zs.zs_adam_tensors(lst, HP, 1, torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        want = own["master"] if want is None else want
        assert torch.equal(own["master"], want) and not torch.equal(want, t["master"])
