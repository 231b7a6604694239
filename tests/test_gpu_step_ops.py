"""The calls around the 4-bit products, run together as a training step and a few generated tokens use them.

A block is y = h + W2 relu(W1 norm(h)): two residual blocks in a row, their
forward and backward passes on 4-bit matrices, the gradients' norm, the
clipped update, and then single tokens through the held weights.  Every stage is
compared with the same stage in 64 bits on the values that the stage before it
left, so that one rounding of bf16 (2^-8 of a value), of fp32 and the products'
bound (include/zs.h) are all that may come between.
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs

pytestmark = pytest.mark.gpu
ROWS, DIM, HIDDEN = 160, 192, 320
EPS = 1e-5
HP = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
H16 = 2.0 ** -8


def room(rows, cols):
    size = zs.zs_mx4_sizes(rows, cols)
    return dict(codes=torch.empty(size["code_bytes"], dtype=torch.uint8, device="cuda"), scales=torch.empty(size["scale_bytes"], dtype=torch.uint8, device="cuda"))


def both(rows, cols):
    return dict(rows=room(rows, cols), cols=room(cols, rows))


def values(held, rows, cols):
    return zs.zs_mx4_dequantize(held, torch.empty(rows, cols, device="cuda")).double()


def e(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def product(a, b, m, n, k, out):
    zs.zs_mx4_matmul(a, b, k, out)
    va, vb = values(a, m, k), values(b, n, k)
    want = va @ vb.t()
    tol = (-(-k // 64) + 8) * 2.0 ** -22 * (va.abs() @ vb.abs().t()) * (1 + H16) + H16 * want.abs() + 2.0 ** -134
    assert bool(((out.double() - want).abs() <= tol).all())
    return out


def norm64(h, w):
    return h.double() / torch.sqrt(h.double().square().mean(1, keepdim=True) + float(np.float32(EPS))) * w.double()


def test_a_step_and_tokens():
    g = torch.Generator(device="cuda").manual_seed(7)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    params = []                                             # (name, master): norm, W1, W2 of each block
    for _ in range(2):
        params += [1 + 0.1 * normal(DIM), normal(HIDDEN, DIM) / DIM ** 0.5, normal(DIM, HIDDEN) / HIDDEN ** 0.5]
    items = [dict(master=p.clone().view(-1), param=p.bfloat16().view(-1), grad=torch.zeros(p.numel(), dtype=torch.bfloat16, device="cuda"),
                  exp_avg=torch.zeros(p.numel(), dtype=torch.uint8, device="cuda"), exp_avg_sq=torch.zeros(p.numel(), dtype=torch.uint8, device="cuda"),
                  exp_avg_scale=torch.zeros(-(-p.numel() // 256), device="cuda"), exp_avg_sq_scale=torch.zeros(-(-p.numel() // 256), device="cuda"))
             for p in params]
    lst = zs.zs_build_tensors(items, state_bits=8)
    info = zs.zs_tensors_info(lst)
    table = e(info["device_table_bytes"], dtype=torch.uint8)
    zs.zs_tensors_upload(lst, table, table.numel())
    view = lambda i, what: items[i][what].view(params[i].shape)  # noqa: E731
    norm, coef, flags = e(1, dtype=torch.float32), e(1, dtype=torch.float32), e(1, dtype=torch.int32)
    scratch, back_scratch = e(info["n_chunks"], dtype=torch.float64), e(zs.zs_rms_norm_scratch(ROWS, DIM), dtype=torch.uint8)

    for step in (1, 2):
        held = {}
        for i in (1, 2, 4, 5):
            held[i] = both(*params[i].shape)
            zs.zs_mx4_quantize(view(i, "param"), **held[i])
        # forward: the second block's norm adds the first one's output to the stream
        x0 = normal(ROWS, DIM).bfloat16()
        saved, stream, delta = [], x0, None
        for b in range(2):
            w = view(3 * b, "param")
            a, s, rstd = both(ROWS, DIM), e(ROWS, DIM), e(ROWS, dtype=torch.float32)
            whole = e(ROWS, DIM)
            zs.zs_rms_norm(stream if delta is None else delta, w, EPS, rstd, residual=None if delta is None else stream, sum=None if delta is None else s,
                           out=whole, **a)
            h = stream if delta is None else s
            if delta is not None:
                assert torch.equal(s, (delta.float() + stream.float()).bfloat16())
            unrounded = stream.double() + (0 if delta is None else delta.double())
            want = norm64(unrounded, w)
            assert bool(((whole.double() - want).abs() <= (H16 + 4 * 2.0 ** -24) * (1 + H16) * want.abs()).all())
            y1 = product(a["rows"], held[3 * b + 1]["rows"], ROWS, HIDDEN, DIM, e(ROWS, HIDDEN))
            act = torch.relu(y1)
            r = both(ROWS, HIDDEN)
            zs.zs_mx4_quantize(act, **r)
            delta = product(r["rows"], held[3 * b + 2]["rows"], ROWS, DIM, HIDDEN, e(ROWS, DIM))
            saved.append((h, rstd, a, r, act))
            stream = h
        final = stream.float() + delta.float()
        # backward: d of the mean square of what comes out
        d, d_held = (2 * final / final.numel()).bfloat16(), both(ROWS, DIM)
        zs.zs_mx4_quantize(d, **d_held)
        for b in (1, 0):
            h, rstd, a, r, act = saved[b]
            product(d_held["cols"], r["cols"], DIM, HIDDEN, ROWS, view(3 * b + 2, "grad"))
            d1 = product(d_held["rows"], held[3 * b + 2]["cols"], ROWS, HIDDEN, DIM, e(ROWS, HIDDEN)) * (act > 0)
            d1_held = both(ROWS, HIDDEN)
            zs.zs_mx4_quantize(d1, **d1_held)
            product(d1_held["cols"], a["cols"], HIDDEN, DIM, ROWS, view(3 * b + 1, "grad"))
            dn = product(d1_held["rows"], held[3 * b + 1]["cols"], ROWS, DIM, HIDDEN, e(ROWS, DIM))
            w, dx, dx_held = view(3 * b, "param"), e(ROWS, DIM), both(ROWS, DIM)
            zs.zs_rms_norm_backward(dn, h, w, rstd, dx, residual=d, dw=view(3 * b, "grad"), scratch=back_scratch, **dx_held)
            r64, g64, h64 = rstd.double()[:, None], dn.double() * w.double(), h.double()
            want = (g64 - h64 * r64 * r64 * (g64 * h64).mean(1, keepdim=True)) * r64 + d.double()
            size = r64 * (g64.abs() + h64.abs() * r64 * r64 * (g64 * h64).abs().mean(1, keepdim=True)) + d.double().abs()
            assert bool(((dx.double() - want).abs() <= H16 * want.abs() + 6 * 2.0 ** -24 * size).all())
            dw = (dn.double() * h64 * r64).sum(0)
            assert bool(((view(3 * b, "grad").double() - dw).abs() <= H16 * dw.abs() + (ROWS + 3) * 2.0 ** -24 * (dn.double() * h64 * r64).abs().sum(0)).all())
            d, d_held = dx, dx_held
        # norm, clip, update
        zs.zs_norm_tensors(lst, scratch, 0.5 * step, norm, coef, flags)
        want = torch.sqrt(sum(t["grad"].double().square().sum() for t in items))
        assert abs(float(norm) - float(want)) <= 2.0 ** -23 * float(want) and int(flags) == 0
        assert float(coef) == min(np.float32(1), np.float32(0.5 * step) / (np.float32(float(norm)) + np.float32(1e-6)))
        before = [t["master"].clone() for t in items]
        zs.zs_adam_tensors(lst, HP, step, coef, flags, rounding="stochastic", seed=3)
        for t, old in zip(items, before):
            assert torch.equal(t["param"], t["master"].bfloat16())
            moved = (t["master"] - old).abs().max()
            assert 0 < float(moved) <= 10 * HP["lr"]        # a few lr at most: |m| / sqrt(v) of two steps
    # tokens through the weights as they are held now, as one and as three
    for i in (1, 2, 4, 5):
        zs.zs_mx4_quantize(view(i, "param"), **held[i])
    for m in (1, 3):
        tokens, rstd, y = normal(m, DIM).bfloat16(), e(m, dtype=torch.float32), e(m, DIM)
        zs.zs_rms_norm(tokens, view(0, "param"), EPS, rstd, out=y)
        up = zs.zs_mx4_matvec(y, held[1]["rows"], e(m, HIDDEN))
        w = values(held[1]["rows"], HIDDEN, DIM)
        want = y.double() @ w.t()
        tol = (DIM // 32 + 24) * 2.0 ** -22 * (y.double().abs() @ w.abs().t()) + 2.0 ** -39 * y.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
        assert bool(((up.double() - want).abs() <= tol * (1 + H16) + H16 * want.abs()).all())
