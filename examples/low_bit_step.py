"""Training with little memory: 4-bit products, 8-bit moments, a sharded step.

A two-layer network learns a fixed random one.  N virtual ranks each see their
own batch; the parameters are sharded by a plan.  A step:

  gather   the 16-bit shards into whole parameters     zs_all_gather_coalesced
  hold     the weights in 4 bits, along both dimensions  zs_mx4_quantize
  forward  y = x w^T on 4-bit matrices                 zs_mx4_quantize, zs_mx4_matmul
  backward dx, and dw straight into the rank's bucket    zs_mx4_quantize, zs_mx4_matmul
  reduce   the ranks' gradients to the owners          zs_reduce_scatter_all
  norm     and clip coefficient                        zs_grad_norm
  update   every shard, moments in 8 bits or 32        zs_adam_tensors

  python examples/low_bit_step.py [--steps 200] [--bits 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_sharded_optimizer_bucket_gb300 as zs  # noqa: E402

N, BATCH, INPUTS, HIDDEN, OUTPUTS = 4, 256, 192, 512, 64
HP = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
SHAPES = [(HIDDEN, INPUTS), (OUTPUTS, HIDDEN)]          # the two weights
DEV = "cuda"


def room(rows, cols):
    """Buffers of a 4-bit matrix."""
    size = zs.zs_mx4_sizes(rows, cols)
    return dict(codes=torch.empty(size["code_bytes"], dtype=torch.uint8, device=DEV),
                scales=torch.empty(size["scale_bytes"], dtype=torch.uint8, device=DEV))


class Held:
    """A 16-bit matrix in 4 bits along its rows and along its columns."""

    def __init__(self, rows, cols):
        self.shape, self.rows, self.cols = (rows, cols), room(rows, cols), room(cols, rows)

    def take(self, x):
        zs.zs_mx4_quantize(x, rows=self.rows, cols=self.cols)
        return self


class Sharded:
    """Plan, buffers and optimizer state of the two weights over N ranks."""

    def __init__(self, weights, bits):
        cfg = zs.zs_default_config(N)
        cfg.param_persistence_threshold = 0
        self.plan = zs.zs_build_partition(cfg, [w.numel() for w in weights])
        info = zs.zs_plan_info(self.plan)
        S = info["shard_elems"]
        b16 = lambda n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        f32 = lambda n: torch.zeros(n, device=DEV)  # noqa: E731
        self.table = torch.empty(info["device_table_bytes"], dtype=torch.uint8, device=DEV)
        zs.zs_plan_upload(self.plan, self.table, self.table.numel())
        self.grad_shards, self.param_shards, self.master = b16(N * S), b16(N * S), f32(N * S)
        m0, v0 = f32(N * S), f32(N * S)                 # zs_partition zeroes 32-bit moments
        state = zs.make_state(param_shards=self.param_shards, master=self.master, exp_avg=m0, exp_avg_sq=v0)
        zs.zs_partition(self.plan, torch.cat([w.reshape(-1) for w in weights]), state)
        # one rank's gradient buffers, bucket by bucket, and where each weight lies in them
        self.grads, self.place, ptrs = [], {}, []
        for b in range(info["n_reduce_buckets"]):
            entry = zs.zs_bucket_info(self.plan, b)
            bufs = [b16(entry["buf_elems"]) for _ in range(N)]
            for q in range(entry["n_entries"]):
                p, lo, hi, off = zs.zs_bucket_entry(self.plan, b, q)
                self.place[p] = (b, off)
            self.grads.append(bufs)
            ptrs += [t.data_ptr() for t in bufs]
        self.rank_grads = torch.tensor(ptrs, dtype=torch.int64, device=DEV)
        # the optimizer's list: a shard row of each rank
        per = -(-S // zs.ZS_STATE_BLOCK)
        tensors = []
        for r in range(N):
            row = slice(r * S, (r + 1) * S)
            t = dict(grad=self.grad_shards[row], param=self.param_shards[row], master=self.master[row])
            if bits == 8:
                t.update(exp_avg=torch.zeros(S, dtype=torch.uint8, device=DEV), exp_avg_scale=f32(per),
                         exp_avg_sq=torch.zeros(S, dtype=torch.uint8, device=DEV), exp_avg_sq_scale=f32(per))
            else:
                t.update(exp_avg=m0[row], exp_avg_sq=v0[row])
            tensors.append(t)
        self.list = zs.zs_build_tensors(tensors, state_bits=bits)
        self.list_table = torch.empty(zs.zs_tensors_info(self.list)["device_table_bytes"], dtype=torch.uint8, device=DEV)
        zs.zs_tensors_upload(self.list, self.list_table, self.list_table.numel())
        self.bits = bits
        self.flat = b16(info["flat_elems"])
        self.scratch = torch.zeros(info["norm_scratch_elems"], dtype=torch.float64, device=DEV)
        self.norm, self.coef = f32(1), f32(1)
        self.flags = torch.zeros(1, dtype=torch.int32, device=DEV)

    def gather(self):
        offs = zs.zs_all_gather_coalesced(self.plan, list(range(len(SHAPES))), self.param_shards, self.flat, self.flat.numel())
        return [self.flat[o:o + r * c].view(r, c) for o, (r, c) in zip(offs, SHAPES)]

    def grad_of(self, rank, p):
        b, off = self.place[p]
        r, c = SHAPES[p]
        return self.grads[b][rank][off:off + r * c].view(r, c)

    def step(self, t):
        zs.zs_reduce_scatter_all(self.plan, self.rank_grads, self.grad_shards, None, self.scratch)
        zs.zs_grad_norm(self.plan, self.grad_shards, None, self.scratch, False, 1.0, self.norm, self.coef, self.flags)
        zs.zs_adam_tensors(self.list, HP, t, self.coef, self.flags,
                           rounding="stochastic" if self.bits == 8 else "nearest", seed=2026)


def train(steps=200, bits=8, seed=0):
    """The mean loss over the ranks at every step, and the trained state."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device=DEV, generator=gen)  # noqa: E731
    teacher = [normal(r, c) / c ** 0.5 for r, c in SHAPES]
    model = Sharded([normal(r, c) / c ** 0.5 for r, c in SHAPES], bits)
    w = [Held(*s) for s in SHAPES]
    x, h, dy, dh = Held(BATCH, INPUTS), Held(BATCH, HIDDEN), Held(BATCH, OUTPUTS), Held(BATCH, HIDDEN)
    out = lambda a, b: torch.empty(a, b, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h_out, y_out, dh_out = out(BATCH, HIDDEN), out(BATCH, OUTPUTS), out(BATCH, HIDDEN)
    losses = []
    for t in range(1, steps + 1):
        for held, weight in zip(w, model.gather()):
            held.take(weight)
        loss = 0.0
        for rank in range(N):
            data = normal(BATCH, INPUTS)
            want = torch.relu(data @ teacher[0].t()) @ teacher[1].t()
            x.take(data.bfloat16())
            hidden = torch.relu(zs.zs_mx4_matmul(x.rows, w[0].rows, INPUTS, h_out))
            h.take(hidden)
            error = zs.zs_mx4_matmul(h.rows, w[1].rows, HIDDEN, y_out).float() - want
            loss = loss + error.square().mean()
            dy.take((2 * error / OUTPUTS).bfloat16())
            zs.zs_mx4_matmul(dy.cols, h.cols, BATCH, model.grad_of(rank, 1))
            back = zs.zs_mx4_matmul(dy.rows, w[1].cols, OUTPUTS, dh_out) * (hidden > 0)
            dh.take(back)
            zs.zs_mx4_matmul(dh.cols, x.cols, BATCH, model.grad_of(rank, 0))
        model.step(t)
        losses.append(loss / N)
    return torch.stack(losses).tolist(), model


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    losses, _ = train(a.steps, a.bits)
    for t in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {t + 1:4d}  loss {losses[t]:.4f}")
    print(f"step {a.steps:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
