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


def test_larger_buffers():
    """More room than a matrix needs: flat, or more rows of the same width."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = torch.randn(40, 200, device="cuda", generator=g), torch.randn(50, 200, device="cuda", generator=g)
    size = zs.zs_mx4_sizes(64, 200)
    want = None
    for shape in ((40 * size["row_bytes"],), (40, size["row_bytes"]), (64, size["row_bytes"]), (1 << 16,)):
        a = dict(codes=torch.zeros(shape, dtype=torch.uint8, device="cuda"), scales=torch.zeros(1 << 13, dtype=torch.uint8, device="cuda"))
        b = room(50, 200)
        zs.zs_mx4_quantize(x, rows=a)
        zs.zs_mx4_quantize(w, rows=b)
        got = zs.zs_mx4_matmul(a, b, 200, torch.empty(40, 50, device="cuda"))
        want = got if want is None else want
        assert torch.equal(got, want) and bool(want.any())


@pytest.mark.parametrize("k", [1, 32, 96, 480])
def test_another_k_is_refused(k):
    """A matrix held with 512 columns is not one of fewer: its rows are farther apart."""
    def held(rows, cols):
        size = zs.zs_mx4_sizes(rows, cols)
        return dict(codes=torch.zeros(rows, size["row_bytes"], dtype=torch.uint8, device="cuda"),
                    scales=torch.zeros(size["scale_bytes"], dtype=torch.uint8, device="cuda"))

    out = torch.full((8, 16), 7.0, device="cuda")
    for a, b in ((held(8, 512), held(16, 512)), (held(8, 512), held(16, k)), (held(8, k), held(16, 512))):
        with pytest.raises(ValueError, match="bytes a row expected"):
            zs.zs_mx4_matmul(a, b, k, out)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
