"""zs_adam_tensors on lists long enough for the long chunks (6144 elements with 8-bit moments, three rounds of stages of 8
blocks; 8192 with 32-bit ones), within the same derived bounds as short lists; and the two ways of taking a block, by whole
vectors and element by element, which have to give the same bits."""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests import lowbit_ref as ref
from tests.test_gpu_tensors import HP, bounds, check_codes, check_param, held, make, rand_state

pytestmark = pytest.mark.gpu
SIZES = [2_000_003, 257, 12_288, 20_481]
CHUNK = {8: 6144, 32: 8192}


@pytest.mark.parametrize("bits,rounding", [(32, "nearest"), (8, "nearest"), (8, "stochastic")])
@pytest.mark.parametrize("grad_kind,param_kind,shift", [("bf16", "bf16", 0), ("fp16", "fp16", 0), ("fp32", None, 0), ("fp32", "bf16", 0),
                                                        ("bf16", None, 0), ("bf16", "bf16", 1), ("fp32", "fp16", 1)])
def test_step(bits, rounding, grad_kind, param_kind, shift):
    rng = np.random.default_rng(bits + 7 * shift)
    states = [rand_state(n, bits, rng, grad_kind) for n in SIZES]
    bufs, lst = make(states, bits, grad_kind, param_kind, shift)
    assert zs.zs_tensors_info(lst)["n_chunks"] == sum(-(-n // CHUNK[bits]) for n in SIZES)
    coef = torch.full((1,), 0.625, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    step, seed = 5, 0x1234567890ABCDEF
    zs.zs_adam_tensors(lst, HP, step, coef, flags, rounding=rounding, seed=seed)
    torch.cuda.synchronize()
    for i, (s, b) in enumerate(zip(states, bufs)):
        assert all(x.guards_ok() for x in b.values())
        m0, v0 = (s["m"].astype(np.float64), s["v"].astype(np.float64)) if bits == 32 else \
            (held(s["m_code"], s["m_scale"]), held(s["r_code"], s["r_scale"]) ** 2)
        p, m, r, dp, dm, dr = bounds(s, m0, v0, HP, step, 0.625)
        got = {k: x.t.cpu().numpy() for k, x in b.items() if k not in ("grad", "param")}
        assert np.all(np.abs(got["master"] - p) <= dp)
        if param_kind:
            check_param(b)
        if bits == 32:
            assert np.all(np.abs(got["exp_avg"] - m) <= dm)
            assert np.all(np.abs(np.sqrt(got["exp_avg_sq"].astype(np.float64)) - r) <= dr)
            continue
        a, c = ref.random16(len(s["p"]), i, step, seed) if rounding == "stochastic" else (None, None)
        check_codes(got["exp_avg"], got["exp_avg_scale"], m, dm, a)
        check_codes(got["exp_avg_sq"], got["exp_avg_sq_scale"], r, dr, c, least=True)
    assert zs.zs_device_wait_timeouts() == 0


def wide_state(n, rng):
    """Blocks all over the range of float32, gradients spread over 20 octaves in each; some blocks of zeros, some with
    infinities and NaN, some whose squares pass 2^64."""
    blocks = -(-n // 256)
    top = np.repeat(rng.integers(-120, 28, blocks), 256)[:n]
    g = np.ldexp(rng.uniform(1, 2, n) * rng.choice([-1, 1], n), top - rng.integers(0, 20, n)).astype(np.float32)
    g[np.repeat(rng.random(blocks) < 0.05, 256)[:n]] = 0.0
    for at, x in ((3000, np.inf), (70_000, np.nan), (500_000, 1e15), (900_001, -1e25)):
        g[at] = x
    scale = lambda: np.ldexp(1.0, np.clip(rng.integers(-130, 20, blocks), -126, 127)).astype(np.float32) * (rng.random(blocks) > 0.1)  # noqa: E731
    code = lambda: rng.integers(0, 0x7F, n).astype(np.uint8)  # noqa: E731
    return dict(grad=torch.from_numpy(g), p=(rng.standard_normal(n) * 0.02).astype(np.float32), m_code=code() | rng.choice([0, 0x80], n).astype(np.uint8),
                r_code=code(), m_scale=scale().astype(np.float32), r_scale=scale().astype(np.float32))


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("hp", [HP, dict(HP, adamw=0), dict(HP, eps=0.0, beta2=0.5, weight_decay=0.0), dict(HP, beta1=0.0, beta2=0.0, bias_correction=0)])
def test_both_ways_give_the_same_bits(rounding, hp):
    """A list at vector addresses and the same one element further: whole blocks go one way in the first, every block the
    other way in the second (paired arithmetic and another root, against one operation at a time)."""
    state = wide_state(2_000_003, np.random.default_rng(17))
    out = []
    for shift in (0, 1):
        bufs, lst = make([state], 8, "fp32", "bf16", shift)
        for step in (1, 2):
            zs.zs_adam_tensors(lst, hp, step, rounding=rounding, seed=3)
        torch.cuda.synchronize()
        out.append({k: b.t.cpu() for k, b in bufs[0].items()})
    for k in out[0]:
        a, b = (o[k].contiguous().view(torch.uint8).numpy() for o in out)
        if k == "master":              # a NaN is a NaN
            a, b = (np.where(np.isnan(x.view(np.float32)), np.float32(np.nan), x.view(np.float32)).view(np.uint32) for x in (a, b))
        if k == "param":
            nan = torch.isnan(out[0][k]).numpy()
            assert np.array_equal(nan, torch.isnan(out[1][k]).numpy())
            a, b = (np.where(nan, 0, x.view(np.uint16)) for x in (a, b))
        assert np.array_equal(a, b), k


def test_root():
    """The vector path's root is the correctly rounded one, for every float below 2^64."""
    count = torch.full((1,), -1, dtype=torch.int64, device="cuda")
    zs.zs_test_root(count)
    assert count.item() == 0
