"""The low-bit training operators, as cases that can be measured.

Three operators that belong together, since one step of training with little
memory goes through all of them:

adam    an AdamW step over a list of tensors, its moments held in 32 bits or
        in 8 (a scale for each block of 256 elements);
quant   a matrix to microscaled 4-bit floating point (blocks of 32, an
        8-bit power of two for each), along its rows, its columns or both,
        and back to values;
matmul  the product of two 4-bit matrices, out[M, N] = A[M, K] B[N, K]^T;
linear  both together: the three products of a linear layer's training step
        (its output, and the gradients of its input and weight) from 16-bit
        matrices.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256                 # elements that share the scales of the 8-bit moments
GROUP = 32                  # elements that share the scale of a 4-bit group
ROUNDS = 7                  # Philox rounds of the stochastic rounding
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
SEED = 0x5EED00C0FFEE
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LAYER = (4096, 11008, 4096)     # hidden, ffn, key/value width of the decoder layer
LAYER_GQA = (4096, 14336, 1024)
MOST_ELEMENTS = 202_383_360     # of the largest listed optimizer step
MOST_FLOPS = 2.0 * 8192 * 14336 * 4096


def listed():
    return [
        # the smallest model's six tensors: a step that is all latency
        dict(name="adam32_tiny", op="adam", shapes="tiny", bits=32, dtype="bf16", rounding="nearest"),
        # one decoder layer, moments in 32 bits: bandwidth
        dict(name="adam32_layer", op="adam", shapes="layer", hidden=LAYER[0], ffn=LAYER[1], kv=LAYER[2], bits=32,
             dtype="bf16", rounding="nearest"),
        # the six tensors with moments in 8 bits and fp32 gradients, no 16-bit copy
        dict(name="adam8_tiny", op="adam", shapes="tiny", bits=8, dtype="fp32", rounding="stochastic"),
        # the decoder layer, moments in 8 bits, rounded stochastically: long runs
        dict(name="adam8_layer", op="adam", shapes="layer", hidden=LAYER[0], ffn=LAYER[1], kv=LAYER[2], bits=8,
             dtype="bf16", rounding="stochastic"),
        # many small tensors of ragged sizes, fp16
        dict(name="adam8_many", op="adam", shapes="many", count=2000, shape_seed=7, bits=8, dtype="fp16",
             rounding="nearest"),
        # activations of a few decoding tokens
        dict(name="quant_tokens", op="quant", rows=24, cols=4096, dtype="bf16", along="rows"),
        # a weight for the forward and the backward pass at once
        dict(name="quant_weight", op="quant", rows=14336, cols=4096, dtype="bf16", along="both"),
        # one token through the down projection: the weight's bytes
        dict(name="matmul_token", op="matmul", m=1, n=4096, k=14336, dtype="bf16"),
        # a batch of decoding tokens through the grouped key projection
        dict(name="matmul_batch", op="matmul", m=48, n=1024, k=4096, dtype="fp16"),
        # nothing a multiple of a tile, 32-bit output
        dict(name="matmul_odd", op="matmul", m=1001, n=777, k=1490, dtype="fp32"),
        # a long prompt through the up projection: the tensor cores
        dict(name="matmul_prompt", op="matmul", m=8192, n=14336, k=4096, dtype="bf16"),
        # a linear layer's training step from 16-bit matrices
        dict(name="linear_train", op="linear", m=4096, n=11008, k=4096, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adam", "adam", "quant", "matmul", "matmul", "linear"])
    if op == "adam":
        bits = rng.choice([8, 8, 32])
        c = dict(op=op, bits=bits, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 rounding=rng.choice(["nearest", "stochastic"]) if bits == 8 else "nearest")
        if rng.random() < 0.5:
            return dict(c, shapes="many", count=_spread(rng, 1, 1800), shape_seed=rng.randrange(1 << 30))
        hidden, ffn, kv = (_spread(rng, 64, 4096), _spread(rng, 64, 11008), _spread(rng, 32, 4096))
        return dict(c, shapes="layer", hidden=hidden, ffn=ffn, kv=min(kv, hidden))
    if op == "quant":
        return dict(op=op, rows=_spread(rng, 1, 14336), cols=_spread(rng, 32, 4096), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    along=rng.choice(["rows", "cols", "both"]))
    m, n, k = _spread(rng, 1, 8192), _spread(rng, 64, 14336), _spread(rng, 32, 14336)
    if op == "linear":
        m, n, k = max(m, 16), min(n, 11008), min(k, 4096)
        m = min(m, max(16, int(MOST_FLOPS / (6.0 * n * k))))
        return dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "fp16"]))
    m = min(m, max(1, int(MOST_FLOPS / (2.0 * n * k))))
    return dict(op=op, m=m, n=n, k=k, dtype=rng.choice(["bf16", "fp16", "fp32"]))


# ---------------------------------------------------------------- sizes --

def _numels(case):
    if case["shapes"] == "tiny":
        return [64 * 64, 64, 256 * 64, 256, 64 * 256, 64]
    if case["shapes"] == "layer":
        h, f, kv = case["hidden"], case["ffn"], case["kv"]
        return [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f, h, h]
    r = np.random.RandomState(case["shape_seed"] % (1 << 31))
    got = np.floor(10.0 ** r.uniform(2.0, 6.0, case["count"]) + 0.5).astype(np.int64)
    total = np.cumsum(got)
    return [int(x) for x in got[total <= MOST_ELEMENTS]] or [int(got[0])]


def _padded(n, to):
    return -(-n // to) * to


def work(case):
    if case["op"] == "adam":
        n = sum(_numels(case))
        size = 4 if case["dtype"] == "fp32" else 2
        # gradient, master read and written, the 16-bit copy, both moments read and written
        each = size + 8 + (0 if case["dtype"] == "fp32" else 2) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": n * each, "flops": 16.0 * n}
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        ways = 2 if case["along"] == "both" else 1
        # the matrix once, and for each way its codes, scales and values
        return {"bytes": n * (size + ways * (0.5 + 1 / GROUP + size)), "flops": 4.0 * n * ways}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "matmul":
        return {"bytes": (m + n) * k * (0.5 + 1 / GROUP) + size * m * n, "flops": 2.0 * m * n * k}
    return {"bytes": 2.0 * size * (m * k + n * k + m * n), "flops": 6.0 * m * n * k}


# --------------------------------------------------------------- inputs --

def _quantize(x):
    """(4-bit codes [R, Kp], scale bytes [R, Kp/32]) of a float matrix, Kp = its columns padded to 32."""
    r, k = x.shape
    kp = _padded(k, GROUP)
    x = torch.nn.functional.pad(x.float(), (0, kp - k)).view(r, kp // GROUP, GROUP)
    top = x.abs().amax(2)
    field = top.view(torch.int32) >> 23
    bad = field == 255
    byte = (field - 2).clamp(min=0)
    y = x * ((254 - byte) << 23).view(torch.float32).unsqueeze(2)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * (torch.signbit(y).to(torch.uint8))
    code = torch.where(bad.unsqueeze(2), torch.zeros_like(code), code)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return code.view(r, kp), byte.to(torch.uint8)


def _pack(code):
    """Two codes a byte, the even element in the low half."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _tile(scale):
    """Scale bytes [R, G] in the order the library holds them: tiles of 128 rows by 4 groups, 8 groups at least."""
    r, g = scale.shape
    s = torch.nn.functional.pad(scale, (0, _padded(g, 8) - g, 0, _padded(r, 128) - r))
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4)
    return s.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(tiles, r, g):
    s = tiles.view(_padded(r, 128) // 128, _padded(g, 8) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return s.reshape(_padded(r, 128), _padded(g, 8))[:r, :g]


def _moment8(x, least):
    """(e4m3 codes, scales) of rows of BLOCK floats, rounded to nearest; least: the code of a positive value is not zero."""
    scale, y = _scaled(x)
    q = y.to(torch.float8_e4m3fn).float()
    if least:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return q.to(torch.float8_e4m3fn), scale


def _scaled(x):
    """The block's scale, a power of two that takes its largest value to [128, 256), and the values over it."""
    field = (x.abs().amax(1).view(torch.int32) >> 23).clamp(min=8)
    return ((field - 7) << 23).view(torch.float32), x * ((261 - field) << 23).view(torch.float32).unsqueeze(1)


def _activations(gen, m, k, dtype):
    """Rows of unit scale with a few channels that are much larger, as residual streams have."""
    x = torch.randn(m, k, device="cuda", generator=gen)
    big = torch.rand(k, device="cuda", generator=gen) < 0.01
    return torch.where(big, 20 * x, x).to(TYPES[dtype])


def _codes(x):
    code, scale = _quantize(x)
    return _pack(code), _tile(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev, kind = "cuda", TYPES[case["dtype"]]
    if case["op"] == "adam":
        numel = _numels(case)
        blocks = [-(-n // BLOCK) for n in numel]
        start = np.concatenate([[0], np.cumsum(blocks)])[:-1] * BLOCK
        total = BLOCK * sum(blocks)
        tensor = torch.repeat_interleave(torch.arange(len(numel), device=dev), torch.tensor(blocks, device=dev))
        first = torch.from_numpy(start).to(dev)[tensor]        # of each block's tensor
        length = torch.tensor(numel, device=dev)[tensor]
        at = (torch.arange(len(tensor), device=dev) * BLOCK - first).unsqueeze(1) + torch.arange(BLOCK, device=dev)
        inside = at < length.unsqueeze(1)
        del at

        def normal(sigma):
            return torch.where(inside, torch.randn(total // BLOCK, BLOCK, device=dev, generator=gen) * sigma, 0.0)

        grad = normal(1e-3)
        u = torch.rand(total // BLOCK, 1, device=dev, generator=gen)
        grad = grad * torch.where(u < 0.02, 0.0, torch.where(u > 0.99, 100.0, 1.0))    # rows not met, outliers
        s = dict(case=case, numel=numel, start=[int(x) for x in start], tensor=tensor, first=first, step=1000,
                 grad=grad.to(kind).view(-1))
        del grad
        s["master"] = normal(0.02).view(-1)
        s["param"] = None if case["dtype"] == "fp32" else s["master"].to(kind)
        m, r = normal(3e-4), normal(1e-3).abs()
        if case["bits"] == 8:
            for name, x, least in (("exp_avg", m, False), ("exp_avg_sq", r, True)):
                q, scale = _moment8(x, least)
                s[name], s[name + "_scale"] = q.view(-1), scale
        else:
            s["exp_avg"], s["exp_avg_sq"] = m.view(-1), (r * r).view(-1)
        s["coef"] = torch.full((1,), 0.73, device=dev)
        s["flags"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    if case["op"] == "quant":
        r, c = case["rows"], case["cols"]
        s = dict(case=case, x=_activations(gen, r, c, case["dtype"]))
        for way, (a, b) in (("rows", (r, c)), ("cols", (c, r))):
            if case["along"] in (way, "both"):
                s[way] = dict(_room(a, b), out=torch.empty(a, b, dtype=kind, device=dev))
        return s
    m, n, k = case["m"], case["n"], case["k"]
    x = _activations(gen, m, k, "bf16" if case["op"] == "matmul" else case["dtype"])
    w = (torch.randn(n, k, device=dev, generator=gen) * 0.02).to(x.dtype)
    if case["op"] == "matmul":
        (ac, asc), (bc, bsc) = _codes(x), _codes(w)
        return dict(case=case, a=ac, a_scale=asc, b=bc, b_scale=bsc, out=torch.empty(m, n, dtype=kind, device=dev))
    dy = (torch.randn(m, n, device=dev, generator=gen) * 1e-3).to(kind)
    s = dict(case=case, x=x, w=w, dy=dy, y=torch.empty(m, n, dtype=kind, device=dev),
             dx=torch.empty(m, k, dtype=kind, device=dev), dw=torch.empty(n, k, dtype=kind, device=dev))
    for name, (a, b) in (("x", (m, k)), ("w", (n, k)), ("dy", (m, n))):
        s[name + "_rows"], s[name + "_cols"] = _room(a, b), _room(b, a)
    return s


def _room(rows, cols):
    """The buffers of a 4-bit matrix."""
    return dict(codes=torch.empty(rows, _padded(cols, GROUP) // 2, dtype=torch.uint8, device="cuda"),
                scales=torch.empty(_padded(rows, 128) * _padded(cols, 8 * GROUP) // GROUP, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------- plain forms --

def _consts(step):
    """Hyper-parameters as the float32 numbers that the update works with."""
    f = lambda x: float(np.float32(x))  # noqa: E731
    lr, b1, b2, eps, wd = map(f, (LR, BETA1, BETA2, EPS, DECAY))
    bc1, bc2 = 1.0 - b1 ** step, 1.0 - b2 ** step
    return dict(lr=lr, b1=b1, b2=b2, eps=eps, omb1=f(1.0 - b1), omb2=f(1.0 - b2), lr_wd=f(lr * wd), bc1=f(bc1), bc2=f(bc2),
                step_size=f(lr / bc1), root=f(1.0 / math.sqrt(bc2)))


def _philox(q, tensor, step):
    """Philox4x32 with ROUNDS rounds: four 32-bit words for each counter (q, tensor, step), keyed by SEED."""
    low = 0xFFFFFFFF
    c = [q & low, q >> 32, tensor, torch.full_like(q, step & low)]
    k0, k1 = SEED & low, SEED >> 32
    for _ in range(ROUNDS):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57       # the low 64 bits, whatever the sign
        c = [((p1 >> 32) & low) ^ c[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, 1)


def _dithered(y, random16):
    """y rounded to e4m3 up or down, up as often as its place between the two says (16 random bits)."""
    a = y.abs()
    off = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)        # the range of equal spacing, as one binade
    bits = (a + off).view(torch.int32) + ((random16 << 4) | 8)
    z = (bits & ~0xFFFFF).view(torch.float32) - off
    return torch.copysign(z, y)


def _adam_plain(s):
    case, c = s["case"], _consts(s["step"])
    g, p = s["grad"].float() * s["coef"], s["master"]
    p = p - p * c["lr_wd"]
    if case["bits"] == 32:
        m = s["exp_avg"] * c["b1"] + g * c["omb1"]
        v = s["exp_avg_sq"] * c["b2"] + (g * g) * c["omb2"]
        one = torch.ones((), device="cuda")
        p = p - (m / (one * c["bc1"])) / ((v / (one * c["bc2"])).sqrt() + c["eps"]) * c["lr"]
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    else:
        m0 = (s["exp_avg"].float().view(-1, BLOCK) * s["exp_avg_scale"].unsqueeze(1)).view(-1)
        r0 = (s["exp_avg_sq"].float().view(-1, BLOCK) * s["exp_avg_sq_scale"].unsqueeze(1)).view(-1)
        m = m0 * c["b1"] + g * c["omb1"]
        r = ((r0 * r0) * c["b2"] + (g * g) * c["omb2"]).sqrt()
        p = p - m / (r * c["root"] + c["eps"]) * c["step_size"]
        if case["rounding"] == "nearest":
            (mq, ms), (rq, rs) = _moment8(m.view(-1, BLOCK), False), _moment8(r.view(-1, BLOCK), True)
        else:
            per = BLOCK // 4
            q = ((torch.arange(len(s["tensor"]), device="cuda") * BLOCK - s["first"]) >> 2).unsqueeze(1) + torch.arange(per, device="cuda")
            word = _philox(q.view(-1), s["tensor"].repeat_interleave(per), s["step"]).view(-1, BLOCK)
            ms, y = _scaled(m.view(-1, BLOCK))
            mq = _dithered(y, (word & 0xFFFF).to(torch.int32)).to(torch.float8_e4m3fn)
            rs, y = _scaled(r.view(-1, BLOCK))
            z = _dithered(y, (word >> 16).to(torch.int32))
            rq = torch.where((r.view(-1, BLOCK) > 0) & (z == 0), 2.0 ** -9, z).to(torch.float8_e4m3fn)
        s["exp_avg"].copy_(mq.view(-1))
        s["exp_avg_sq"].copy_(rq.view(-1))
        s["exp_avg_scale"].copy_(ms)
        s["exp_avg_sq_scale"].copy_(rs)
    s["master"].copy_(p)
    if s["param"] is not None:
        s["param"].copy_(p)


def _values(code, scale):
    """The numbers that codes and scale bytes stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    byte = scale.to(torch.int32)
    two = torch.where(byte == 0, torch.full_like(byte, 1 << 22), byte << 23).view(torch.float32)
    two = torch.where(byte == 255, math.nan, two)
    r, k = code.shape
    return (table[code.to(torch.int32)].view(r, k // GROUP, GROUP) * two.unsqueeze(2)).view(r, k)


def _held(codes, tiles):
    code = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    return _values(code, _untile(tiles, codes.shape[0], code.shape[1] // GROUP))


def _through(x):
    """A matrix's values after 4 bits, in its own shape."""
    return _values(*_quantize(x))[:, :x.shape[1]]


# ------------------------------------------------------------------ run --

def _zs():
    import zero_sharded_optimizer_bucket_gb300 as zs
    return zs


def run(s):
    case = s["case"]
    if case["op"] == "adam":
        if own:
            zs = _zs()
            if "list" not in s:
                s["list"] = _tensor_list(zs, s)
            zs.zs_adam_tensors(s["list"], dict(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY), s["step"],
                               s["coef"], s["flags"], rounding=case["rounding"], seed=SEED)
        else:
            _adam_plain(s)
        s["step"] += 1
        return {k: s[k] for k in ("master", "param", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
                if s.get(k) is not None}
    if case["op"] == "quant":
        x, r, c = s["x"], case["rows"], case["cols"]
        if not own:
            return {w: _through(x if w == "rows" else x.t()).to(x.dtype) for w in ("rows", "cols") if w in s}
        zs = _zs()
        zs.zs_mx4_quantize(x, rows=s.get("rows"), cols=s.get("cols"))
        return {w: zs.zs_mx4_dequantize(s[w], s[w]["out"]) for w in ("rows", "cols") if w in s}
    if case["op"] == "matmul":
        if not own:
            return (_held(s["a"], s["a_scale"]) @ _held(s["b"], s["b_scale"]).t()).to(s["out"].dtype)
        return _zs().zs_mx4_matmul(dict(codes=s["a"], scales=s["a_scale"]), dict(codes=s["b"], scales=s["b_scale"]),
                                   case["k"], s["out"])
    x, w, dy = s["x"], s["w"], s["dy"]
    if not own:
        y = _through(x) @ _through(w).t()
        dx = _through(dy) @ _through(w.t()).t()
        dw = _through(dy.t()) @ _through(x.t()).t()
        return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.to(x.dtype)}
    zs = _zs()
    for name in ("x", "w", "dy"):
        zs.zs_mx4_quantize(s[name], rows=s[name + "_rows"], cols=s[name + "_cols"])
    return {"y": zs.zs_mx4_matmul(s["x_rows"], s["w_rows"], case["k"], s["y"]),
            "dx": zs.zs_mx4_matmul(s["dy_rows"], s["w_cols"], case["n"], s["dx"]),
            "dw": zs.zs_mx4_matmul(s["dy_cols"], s["x_cols"], case["m"], s["dw"])}


def _tensor_list(zs, s):
    """The library's handle of the tensors, each a run of the flat buffers, and its device table."""
    case, items = s["case"], []
    for n, at in zip(s["numel"], s["start"]):
        t = {k: s[k][at:at + n] for k in ("grad", "param", "master", "exp_avg", "exp_avg_sq") if s.get(k) is not None}
        if case["bits"] == 8:
            b, e = at // BLOCK, at // BLOCK - (-n // BLOCK)
            t.update(exp_avg_scale=s["exp_avg_scale"][b:e], exp_avg_sq_scale=s["exp_avg_sq_scale"][b:e])
        items.append(t)
    got = zs.zs_build_tensors(items, state_bits=case["bits"])
    table = torch.empty(zs.zs_tensors_info(got)["device_table_bytes"], dtype=torch.uint8, device="cuda")
    zs.zs_tensors_upload(got, table, table.numel())
    return got


# ---------------------------------------------------------- in 64 bits --

def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx4_64(x):
    """What a matrix holds after 4 bits, along its rows, from the definition: 2^(floor(log2 max) - 2) a group, the nearest of
    0, 1/2, 1, 3/2, 2, 3, 4, 6 times it, ties to the even one."""
    r, k = x.shape
    g = torch.nn.functional.pad(x.double(), (0, -k % GROUP)).view(r, -1, GROUP)
    top = g.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, torch.full_like(top, -126).to(torch.int32)).clamp(min=-125) - 2
    y = g * _two(-e)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).to(torch.float64)
    q = (torch.round(y / step) * step).clamp(-6, 6)
    return (q * _two(e)).view(r, -1)[:, :k]


def _e4m3_64(y):
    """The nearest number with three bits after the leading one, of 2^-9 at least apart."""
    e = torch.where(y == 0, torch.zeros_like(y, dtype=torch.int32), torch.frexp(y).exponent - 1).clamp(min=-6) - 3
    return torch.round(y * _two(-e)) * _two(e)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return {w: _mx4_64(s["x"] if w == "rows" else s["x"].t()) for w in ("rows", "cols") if w in s}
    if case["op"] == "matmul":
        def held(codes, tiles):
            code = torch.stack([codes % 16, codes // 16], 2).view(codes.shape[0], -1).long()
            mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")[code % 8]
            e = _untile(tiles, code.shape[0], code.shape[1] // GROUP).to(torch.int32) - 127
            return mag * (1 - 2 * (code // 8)) * _two(e).repeat_interleave(GROUP, 1)
        return held(s["a"], s["a_scale"]) @ held(s["b"], s["b_scale"]).t()
    if case["op"] == "linear":
        x, w, dy = s["x"], s["w"], s["dy"]
        return {"y": _mx4_64(x) @ _mx4_64(w).t(), "dx": _mx4_64(dy) @ _mx4_64(w.t()).t(),
                "dw": _mx4_64(dy.t()) @ _mx4_64(x.t()).t()}
    t = s["step"]
    b1, b2, lr, wd, eps = (float(np.float32(v)) for v in (BETA1, BETA2, LR, DECAY, EPS))
    g = s["grad"].double() * float(s["coef"])
    m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * s["exp_avg_scale"].double()[:, None]).view(-1)
        v = ((v.view(-1, BLOCK) * s["exp_avg_sq_scale"].double()[:, None]) ** 2).view(-1)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    p = s["master"].double()
    p = p - lr * wd * p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
    out = {"master": p, "param": None if s["param"] is None else p}
    if case["bits"] == 32:
        return dict(out, exp_avg=m, exp_avg_sq=v)
    for name, x in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1)
        e = torch.where(top > 0, torch.frexp(top).exponent - 1, torch.full_like(top, -127).to(torch.int32)).clamp(min=-119) - 7
        scale = _two(e)
        out[name + "_scale"] = scale
        q = None
        if case["rounding"] == "nearest":
            q = _e4m3_64(x / scale[:, None])
            q = (torch.where((x > 0) & (q == 0), 2.0 ** -9, q) if name == "exp_avg_sq" else q).view(-1)
        out[name] = q
    return out
