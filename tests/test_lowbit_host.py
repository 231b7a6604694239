"""The low-bit calls' refusals and host-side layout (no GPU: argument errors enqueue nothing), and the references' own pins."""
import numpy as np
import pytest

import zero_sharded_optimizer_bucket_gb300 as zs
from synth import philox as sphilox
from tests import lowbit_ref as ref

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
A16 = 1 << 20        # an address that no call follows


def tensor(**kw):
    t = dict(numel=1000, grad=A16, master=A16, exp_avg=A16, exp_avg_sq=A16, exp_avg_scale=A16, exp_avg_sq_scale=A16, param=A16)
    t.update(kw)
    return t


def refuses(fn, *a, status=zs.ZS_EINVAL, **kw):
    with pytest.raises(zs.ZsError) as e:
        fn(*a, **kw)
    assert e.value.status == status
    assert zs.zs_last_error() != ""


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [dict(numel=-1), dict(grad=None), dict(grad=A16 + 1), dict(master=None), dict(master=A16 + 2), dict(exp_avg=None),
                                 dict(exp_avg_sq=None), dict(param=A16 + 1)])
def test_tensor_refusals(bits, bad):
    refuses(zs.zs_build_tensors, [tensor(), tensor(**bad)], state_bits=bits)


def test_list_refusals():
    refuses(zs.zs_build_tensors, [tensor()], state_bits=16)
    refuses(zs.zs_build_tensors, [tensor()], state_bits=8, grad_dtype=3)
    refuses(zs.zs_build_tensors, [tensor()], state_bits=8, param_dtype=zs.ZS_DTYPE_FP32)
    refuses(zs.zs_build_tensors, [tensor(exp_avg_scale=None)], state_bits=8)
    refuses(zs.zs_build_tensors, [tensor(exp_avg_sq_scale=A16 + 2)], state_bits=8)
    refuses(zs.zs_build_tensors, [tensor(exp_avg=A16 + 2)], state_bits=32)
    zs.zs_build_tensors([tensor(exp_avg=A16 + 1, param=None)], state_bits=8)         # bytes have no alignment
    zs.zs_build_tensors([tensor(exp_avg_scale=None, exp_avg_sq_scale=None)], state_bits=32)
    with pytest.raises(TypeError):
        zs.zs_build_tensors([tensor(moment=A16)])


def test_list_info_and_upload():
    sizes = [1, 255, 256, 257, 8192, 8193, 0, 100_000]
    lst = zs.zs_build_tensors([tensor(numel=n) for n in sizes], state_bits=8)
    info = zs.zs_tensors_info(lst)
    assert info["numel"] == sum(sizes) and info["n_tensors"] == len(sizes) and info["state_bits"] == 8
    assert info["n_blocks"] == sum(-(-n // 256) for n in sizes)
    assert info["n_chunks"] >= sum(n > 0 for n in sizes)
    need = info["device_table_bytes"]
    refuses(zs.zs_tensors_upload, lst, None, need)
    refuses(zs.zs_tensors_upload, lst, A16 + 8, need)
    refuses(zs.zs_tensors_upload, lst, A16, need - 1)
    refuses(zs.zs_adam_tensors, lst, HP, 1, status=zs.ZS_ESTATE)
    empty = zs.zs_build_tensors([])
    assert zs.zs_tensors_info(empty)["device_table_bytes"] == 0
    zs.zs_tensors_upload(empty, None, 0)
    zs.zs_adam_tensors(empty, HP, 1)                                                 # nothing to do, no launch


def test_step_refusals():
    for bits in (8, 32):
        lst = zs.zs_build_tensors([tensor()], state_bits=bits)
        refuses(zs.zs_adam_tensors, lst, HP, 0)
        refuses(zs.zs_adam_tensors, lst, dict(HP, beta1=1.0), 1)
        refuses(zs.zs_adam_tensors, lst, dict(HP, lr=float("nan")), 1)
        refuses(zs.zs_adam_tensors, lst, HP, 1, rounding=2)
        refuses(zs.zs_adam_tensors, lst, HP, 1, d_clip_coef=A16 + 2)
        refuses(zs.zs_adam_tensors, lst, HP, 1, d_flags=A16 + 1)
    refuses(zs.zs_adam_tensors, zs.zs_build_tensors([tensor()]), HP, 1, rounding="stochastic")


def test_mx4_sizes():
    for rows, cols in [(0, 0), (1, 1), (128, 32), (129, 33), (7, 256), (7, 257), (1000, 4096)]:
        s = zs.zs_mx4_sizes(rows, cols)
        groups = -(-cols // 32)
        assert s["row_bytes"] == 16 * groups and s["code_bytes"] == rows * 16 * groups
        assert s["scale_bytes"] == len(ref.tile_scales(np.zeros((rows, groups), np.uint8)))
    refuses(zs.zs_mx4_sizes, -1, 4)
    refuses(zs.zs_mx4_sizes, 4, 1 << 31)


def call(name, *a):
    got = getattr(zs._lib, name)(*a)
    assert got == zs.ZS_EINVAL, (name, a, got)
    assert zs.zs_last_error() != ""


def test_mx4_refusals():
    a, odd = A16, A16 + 8
    q = "zs_mx4_quantize"
    call(q, a, 4, 64, 63, 0, a, a, None, None, None)             # rows overlap
    call(q, a, -1, 64, 64, 0, a, a, None, None, None)
    call(q, a, 4, 1 << 31, 1 << 31, 0, a, a, None, None, None)
    call(q, a, 4, 64, 64, 3, a, a, None, None, None)
    call(q, a, 4, 64, 64, 0, None, None, None, None, None)
    call(q, None, 4, 64, 64, 0, a, a, None, None, None)
    call(q, a + 1, 4, 64, 64, 0, a, a, None, None, None)
    call(q, a + 2, 4, 64, 64, 2, a, a, None, None, None)
    call(q, a, 4, 64, 64, 0, a, None, None, None, None)
    call(q, a, 4, 64, 64, 0, None, a, None, None, None)
    call(q, a, 4, 64, 64, 0, a, a, odd, a, None)
    call(q, a, 4, 64, 64, 0, a, a, a, odd, None)
    d = "zs_mx4_dequantize"
    call(d, None, a, 4, 64, a, 64, 0, None)
    call(d, a, None, 4, 64, a, 64, 0, None)
    call(d, a, a, 4, 64, None, 64, 0, None)
    call(d, a, a, 4, 64, a, 63, 0, None)
    call(d, a, a, 4, 64, a, 64, -1, None)
    m = "zs_mx4_matmul"
    call(m, -1, 4, 64, a, a, a, a, a, 4, 0, None)
    call(m, 4, 4, 1 << 31, a, a, a, a, a, 4, 0, None)
    call(m, 4, 4, 64, a, a, a, a, a, 3, 0, None)
    call(m, 4, 4, 64, a, a, a, a, a, 4, 7, None)
    call(m, 4, 4, 64, None, a, a, a, a, 4, 0, None)
    call(m, 4, 4, 64, a, a, a, None, a, 4, 0, None)
    call(m, 4, 4, 64, a, odd, a, a, a, 4, 0, None)
    call(m, 4, 4, 64, a, a, a, a, None, 4, 0, None)
    call(m, 4, 4, 64, a, a, a, a, a + 1, 4, 0, None)
    call(m, 4, 4, 64, a, a, a, a, a + 2, 4, 2, None)


def test_binding_refusals():
    import torch
    held = dict(codes=torch.zeros(4, 16, dtype=torch.uint8), scales=torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):
        zs.zs_mx4_quantize(torch.zeros(4, 64).t(), rows=held)                 # columns first
    with pytest.raises(ValueError):
        zs.zs_mx4_quantize(torch.zeros(4, 64), rows=held)                     # too small
    with pytest.raises(TypeError):
        zs.zs_mx4_quantize(torch.zeros(4, 32, dtype=torch.float64), rows=held)
    t = dict(grad=torch.zeros(300), master=torch.zeros(300), exp_avg=torch.zeros(300, dtype=torch.uint8),
             exp_avg_sq=torch.zeros(300, dtype=torch.uint8), exp_avg_scale=torch.zeros(2), exp_avg_sq_scale=torch.zeros(2))
    zs.zs_build_tensors([t], state_bits=8)
    for bad in (dict(exp_avg=torch.zeros(300)), dict(master=torch.zeros(300, dtype=torch.float64))):
        with pytest.raises(TypeError):
            zs.zs_build_tensors([dict(t, **bad)], state_bits=8)
    for bad in (dict(exp_avg_scale=torch.zeros(1)), dict(grad=torch.zeros(299)), dict(grad=torch.zeros(600)[::2])):
        with pytest.raises(ValueError):
            zs.zs_build_tensors([dict(t, **bad)], state_bits=8)
    with pytest.raises(TypeError):
        zs.zs_build_tensors([t, dict(t, grad=torch.zeros(300, dtype=torch.bfloat16))], state_bits=8)


# ------------------------------------------------- pins of the references --

def test_reference_philox():
    """Ten rounds are the generator's, which its published vectors pin."""
    idx = np.arange(64, dtype=np.uint64)
    seed = 0x0123456789ABCDEF
    got = ref.philox([idx & np.uint64(0xFFFFFFFF), idx >> np.uint64(32), idx * np.uint64(0) + np.uint64(3), idx * np.uint64(0) + np.uint64(2)], seed, 10)
    z = np.zeros_like(idx)
    want = sphilox.philox4x32_10(idx, z, z + np.uint64(3), z + np.uint64(2), seed & 0xFFFFFFFF, seed >> 32)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def test_reference_formats():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)
    # a group's values by hand: max 5 -> scale 2^(2-2) = 1; 5 ties to 4, 0.25 to 0, -2.5 to -2
    x = np.zeros((1, 32))
    x[0, :5] = [5.0, 0.25, -2.5, 0.75, 3.0]
    code, byte = ref.mx4(x)
    assert byte[0, 0] == 127
    assert list(ref.mx4_values(code, byte)[0, :5]) == [4.0, 0.0, -2.0, 1.0, 3.0]
    assert list(ref.unpack(ref.pack(code))[0, :5]) == list(code[0, :5])
    # 0.15 -> floor(log2) = -3: scale 2^-5, 0.15 * 32 = 4.8 -> 4: 0.125
    code, byte = ref.mx4(np.full((1, 32), 0.15))
    assert byte[0, 0] == 122 and ref.mx4_values(code, byte)[0, 0] == 0.125


def test_reference_adam():
    import torch
    rng = np.random.default_rng(0)
    p = torch.nn.Parameter(torch.from_numpy(rng.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=float(np.float32(1e-3)), betas=(float(np.float32(0.9)), float(np.float32(0.999))), eps=float(np.float32(1e-8)),
                            weight_decay=float(np.float32(0.01)))
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in (1, 2, 3):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g * 0.5)
        opt.step()
        q, m, v = ref.adam64(q, m, v, g, HP, step, 0.5)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-15)


def test_list_keeps_its_tensors():
    """The list holds addresses, so it keeps the tensors themselves, whatever becomes of the caller's dicts."""
    import gc
    import weakref

    import torch
    t = dict(grad=torch.zeros(300), master=torch.zeros(300), exp_avg=torch.zeros(300), exp_avg_sq=torch.zeros(300))
    alive = [weakref.ref(x) for x in t.values()]
    lst = zs.zs_build_tensors([t], state_bits=32)
    t["grad"] = torch.zeros(300)                     # a training loop's next gradient
    t.clear()
    gc.collect()
    assert all(r() is not None for r in alive)
    del lst
    gc.collect()
    assert all(r() is None for r in alive)


def test_tensors_of_another_device_are_refused():
    """A CPU tensor's address never reaches a kernel: refused before the C call, with its name."""
    import torch
    x = torch.zeros(4, 32)
    size = zs.zs_mx4_sizes(4, 32)
    held = dict(codes=torch.zeros(size["code_bytes"], dtype=torch.uint8), scales=torch.zeros(size["scale_bytes"], dtype=torch.uint8))
    for call in (lambda: zs.zs_mx4_quantize(x, rows=held), lambda: zs.zs_mx4_dequantize(held, x), lambda: zs.zs_mx4_matmul(held, held, 32, torch.zeros(4, 4))):
        with pytest.raises(ValueError, match="got cpu"):
            call()
    t = dict(grad=torch.zeros(300), master=torch.zeros(300), exp_avg=torch.zeros(300), exp_avg_sq=torch.zeros(300))
    lst = zs.zs_build_tensors([t], state_bits=32)                                    # host only
    with pytest.raises(ValueError, match="got cpu"):
        zs.zs_tensors_upload(lst, A16, 1 << 20)
    with pytest.raises(ValueError, match="got cpu"):
        zs.zs_tensors_upload(zs.zs_build_tensors([tensor()]), torch.zeros(1 << 12, dtype=torch.uint8), 1 << 12)


@pytest.mark.parametrize("k", [1, 32, 96, 480])
def test_another_k_is_refused(k):
    """A matrix held with 512 columns is not one of fewer: its rows are farther apart."""
    import torch

    def held(rows, cols):
        size = zs.zs_mx4_sizes(rows, cols)
        return dict(codes=torch.zeros(rows, size["row_bytes"], dtype=torch.uint8), scales=torch.zeros(size["scale_bytes"], dtype=torch.uint8))

    out = torch.empty(8, 16)
    for a, b in ((held(8, 512), held(16, 512)), (held(8, 512), held(16, k))):
        with pytest.raises(ValueError, match="bytes a row expected"):
            zs.zs_mx4_matmul(a, b, k, out)
    for call in (lambda: zs.zs_mx4_dequantize(held(8, 512), torch.empty(8, k)), lambda: zs.zs_mx4_quantize(torch.empty(8, k), rows=held(8, 512)),
                 lambda: zs.zs_mx4_quantize(torch.empty(k, 8), cols=held(8, 512))):
        with pytest.raises(ValueError, match="bytes a row expected"):
            call()
