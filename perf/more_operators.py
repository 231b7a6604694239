"""The operators around the 4-bit products of a training step, as cases that can be measured.

norm    the global gradient norm over a list of tensors, its clip coefficient
        and overflow flag, and with `clip` the gradients scaled in place;
rms     the root-mean-square norm in front of a linear layer, with the
        residual's addition, its result in 16 or 32 bits and / or held in
        microscaled 4-bit form along its rows and its columns, as the
        products of the layer's training step read it;
back    its backward pass: the gradient of the residual stream, whole and in
        both 4-bit forms, and the gradient of the norm's weight;
matvec  a few tokens in 16 or 32 bits through a weight held in 4 bits, for
        generating from the weights that training holds.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256                 # elements that share the scales of the 8-bit moments
GROUP = 32                  # elements that share the scale of a 4-bit group
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LAYER = (4096, 11008, 4096)     # hidden, ffn, key/value width of the decoder layer
MOST_ELEMENTS = 202_383_360     # of the largest listed list of gradients
MOST_VALUES = 4096 * 4096       # of the largest listed matrix of tokens
MOST_WEIGHT = 14336 * 4096


def listed():
    return [
        # the smallest model's six gradients in fp32: all latency
        dict(name="norm_tiny", op="norm", shapes="tiny", dtype="fp32", clip=False, scaled=False),
        # one decoder layer's gradients, whose coefficient the update applies: one read
        dict(name="norm_layer", op="norm", shapes="layer", hidden=LAYER[0], ffn=LAYER[1], kv=LAYER[2], dtype="bf16",
             clip=False, scaled=False),
        # many small fp16 tensors of ragged sizes, clipped in place for an update that takes no coefficient
        dict(name="clip_many", op="norm", shapes="many", count=2000, shape_seed=7, dtype="fp16", clip=True, scaled=False),
        # a few decoding tokens: residual added, normalised for a product with 16-bit tokens
        dict(name="rms_tokens", op="rms", rows=24, cols=4096, dtype="bf16", weight="bf16", residual=True, out=True, held="none"),
        # a training step's tokens, held in both forms for the layer's three products
        dict(name="rms_train", op="rms", rows=4096, cols=4096, dtype="bf16", weight="bf16", residual=True, out=False, held="both"),
        # nothing a multiple of a tile or vector, 32 bits, no residual (the first norm), along the rows
        dict(name="rms_odd", op="rms", rows=1001, cols=777, dtype="fp32", weight="fp32", residual=False, out=True, held="rows"),
        # a training step's backward pass: the stream's gradient whole and held, the weight's
        dict(name="back_train", op="back", rows=4096, cols=4096, dtype="bf16", weight="bf16", residual=True, held="both"),
        # a ragged batch in fp16 with a 32-bit weight, 16-bit products before it
        dict(name="back_odd", op="back", rows=1333, cols=1490, dtype="fp16", weight="fp32", residual=True, held="none"),
        # one token through the down projection: the weight's bytes
        dict(name="matvec_token", op="matvec", m=1, n=4096, k=14336, dtype="bf16"),
        # some sequences decoding together through the up projection
        dict(name="matvec_batch", op="matvec", m=32, n=14336, k=4096, dtype="fp16"),
        # nothing a multiple of a tile, 32 bits
        dict(name="matvec_odd", op="matvec", m=5, n=777, k=1490, dtype="fp32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rms", "rms", "back", "matvec", "matvec"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op == "norm":
        clip = rng.random() < 0.5
        c = dict(op=op, dtype=dtype, clip=clip, scaled=not clip and rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(c, shapes="many", count=_spread(rng, 1, 1800), shape_seed=rng.randrange(1 << 30))
        # in place a pass reads twice and writes: smaller layers keep it below the largest case
        hidden, ffn, kv = (_spread(rng, 64, 2048 if clip else 4096), _spread(rng, 64, 5504 if clip else 11008), _spread(rng, 32, 4096))
        if dtype == "fp32":
            hidden, ffn = min(hidden, 2048), min(ffn, 5504)
        return dict(c, shapes="layer", hidden=hidden, ffn=ffn, kv=min(kv, hidden))
    if op == "matvec":
        n, k = _spread(rng, 32, 14336), _spread(rng, 32, 14336)
        return dict(op=op, m=_spread(rng, 1, 64), n=min(n, MOST_WEIGHT // k), k=k, dtype=dtype)
    rows, cols = _spread(rng, 1, 8192), _spread(rng, 32, 8192)
    c = dict(op=op, rows=min(rows, MOST_VALUES // cols), cols=cols, dtype=dtype, weight=rng.choice([dtype, "fp32"]),
             residual=rng.random() < 0.8, held=rng.choice(["none", "rows", "cols", "both"]))
    return c if op == "back" else dict(c, out=c["held"] == "none" or rng.random() < 0.5)


# ---------------------------------------------------------------- sizes --

def _numels(case):
    if case["shapes"] == "tiny":
        return [64 * 64, 64, 256 * 64, 256, 64 * 256, 64]
    if case["shapes"] == "layer":
        h, f, kv = case["hidden"], case["ffn"], case["kv"]
        return [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f, h, h]
    r = np.random.RandomState(case["shape_seed"] % (1 << 31))
    most = MOST_ELEMENTS // (4 if case["dtype"] == "fp32" else 2)
    got = np.floor(10.0 ** r.uniform(2.0, 6.0, case["count"]) + 0.5).astype(np.int64)
    total = np.cumsum(got)
    return [int(x) for x in got[total <= most]] or [int(got[0])]


def _padded(n, to):
    return -(-n // to) * to


def _size(kind):
    return 4 if kind == "fp32" else 2


def _ways(case):
    return {"none": (), "rows": ("rows",), "cols": ("cols",), "both": ("rows", "cols")}[case["held"]]


def work(case):
    if case["op"] == "norm":
        n = sum(_numels(case))
        # every gradient read; in place it is read again, and written
        return {"bytes": n * _size(case["dtype"]) * (3 if case["clip"] else 1) + 12, "flops": n * (3.0 if case["clip"] else 2.0)}
    if case["op"] == "matvec":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * (0.5 + 1 / GROUP) + _size(case["dtype"]) * m * (n + k), "flops": 2.0 * m * n * k}
    r, c, size = case["rows"], case["cols"], _size(case["dtype"])
    held = r * c * len(_ways(case)) * (0.5 + 1 / GROUP + 2)         # codes, scales, and the values that come back
    if case["op"] == "rms":
        whole = 1 + 2 * case["residual"] + case["out"]              # x, the residual and the sum, the result
        return {"bytes": r * c * size * whole + held + c * _size(case["weight"]) + 4 * r, "flops": 6.0 * r * c}
    # the result's gradient, the input and the gradient of the sum read; the input's gradient written
    return {"bytes": r * c * size * (3 + case["residual"]) + held + 2 * c * _size(case["weight"]) + 4 * r, "flops": 11.0 * r * c}


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


def _stream(gen, m, k):
    """Rows of a residual stream: unit scale, a few channels that are much larger."""
    x = torch.randn(m, k, device="cuda", generator=gen)
    big = torch.rand(k, device="cuda", generator=gen) < 0.01
    return torch.where(big, 20 * x, x)


def _room(rows, cols):
    """The buffers of a 4-bit matrix, and of its values."""
    return dict(codes=torch.empty(rows, _padded(cols, GROUP) // 2, dtype=torch.uint8, device="cuda"),
                scales=torch.empty(_padded(rows, 128) * _padded(cols, 8 * GROUP) // GROUP, dtype=torch.uint8, device="cuda"),
                out=torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev, kind = "cuda", TYPES[case["dtype"]]
    if case["op"] == "norm":
        numel = _numels(case)
        blocks = [-(-n // BLOCK) for n in numel]
        start = np.concatenate([[0], np.cumsum(blocks)])[:-1] * BLOCK
        total = BLOCK * sum(blocks)
        tensor = torch.repeat_interleave(torch.arange(len(numel), device=dev), torch.tensor(blocks, device=dev))
        first, length = torch.from_numpy(start).to(dev)[tensor], torch.tensor(numel, device=dev)[tensor]
        at = (torch.arange(len(tensor), device=dev) * BLOCK - first).unsqueeze(1) + torch.arange(BLOCK, device=dev)
        sigma = 1.0 if case["dtype"] == "fp16" else 1e-3       # fp16 gradients carry a loss scale
        grad = torch.where(at < length.unsqueeze(1), torch.randn(total // BLOCK, BLOCK, device=dev, generator=gen) * sigma, 0.0)
        del at
        u = torch.rand(total // BLOCK, 1, device=dev, generator=gen)
        grad = grad * torch.where(u < 0.02, 0.0, torch.where(u > 0.99, 100.0, 1.0))    # rows not met, outliers
        s = dict(case=case, numel=numel, start=[int(x) for x in start], grad=grad.to(kind).view(-1),
                 max_norm=0.5 * sigma * math.sqrt(sum(numel)))
        # what the optimizer's list has beside the gradients
        s["master"] = torch.empty(total, device=dev)
        s["exp_avg"], s["exp_avg_sq"] = (torch.empty(total, dtype=torch.uint8, device=dev) for _ in range(2))
        s["exp_avg_scale"], s["exp_avg_sq_scale"] = (torch.empty(total // BLOCK, device=dev) for _ in range(2))
        s["norm"], s["coef"] = torch.empty(1, device=dev), torch.empty(1, device=dev)
        s["flags"] = torch.empty(1, dtype=torch.int32, device=dev)
        s["scale"] = torch.full((1,), 1024.0, device=dev) if case["scaled"] else None
        if own:             # made once, for gradients that stay where they are
            s["list"] = _tensor_list(_zs(), s)
        return s
    if case["op"] == "matvec":
        m, n, k = case["m"], case["n"], case["k"]
        x = _stream(gen, m, k).to(kind)
        code, scale = _quantize((torch.randn(n, k, device=dev, generator=gen) * 0.02).bfloat16())
        return dict(case=case, x=x, w=dict(codes=_pack(code), scales=_tile(scale)), out=torch.empty(m, n, dtype=kind, device=dev))
    r, c = case["rows"], case["cols"]
    x = _stream(gen, r, c).to(kind)
    w = (1 + 0.1 * torch.randn(c, device=dev, generator=gen)).to(TYPES[case["weight"]])
    s = dict(case=case, x=x, w=w, residual=None, rstd=torch.empty(r, device=dev))
    for way in _ways(case):
        s[way] = _room(r, c) if way == "rows" else _room(c, r)
    if case["op"] == "rms":
        if case["residual"]:
            s["residual"], s["sum"] = _stream(gen, r, c).to(kind), torch.empty(r, c, dtype=kind, device=dev)
        if case["out"]:
            s["out"] = torch.empty(r, c, dtype=kind, device=dev)
        return s
    s["dy"] = (torch.randn(r, c, device=dev, generator=gen) * 1e-3).to(kind)
    if case["residual"]:
        s["residual"] = (torch.randn(r, c, device=dev, generator=gen) * 1e-3).to(kind)
    s["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
    s["dx"], s["dw"] = torch.empty(r, c, dtype=kind, device=dev), torch.empty(c, dtype=w.dtype, device=dev)
    if own:
        s["scratch"] = torch.empty(_zs().zs_rms_norm_scratch(r, c), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------- plain forms --

def _norm_plain(s):
    g = s["grad"].float()
    norm = g.square().sum().sqrt()
    scale = torch.ones((), device="cuda") if s["scale"] is None else s["scale"]
    norm = norm / scale
    fine = torch.isfinite(norm)
    coef = torch.where(fine, (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0) / scale, 1.0)
    s["norm"].copy_(norm)
    s["coef"].copy_(coef)
    s["flags"].copy_(torch.where(fine, 0, 1))
    if s["case"]["clip"]:
        s["grad"].copy_(torch.where(fine, g * s["coef"], g))


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
    return _values(*_quantize(x))[:, :x.shape[1]].bfloat16()


def _forms(y, case):
    return {way: _through(y if way == "rows" else y.t()) for way in _ways(case)}


def _rms_plain(s):
    case, h = s["case"], s["x"].float()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        got["sum"] = h.to(s["x"].dtype)
    # the mean in 64 bits: results lie next to the borders of 4 bits
    rstd = (1 / (h.double().square().sum(1) / h.shape[1] + float(np.float32(EPS))).sqrt()).float()
    y = (h * rstd.unsqueeze(1) * s["w"].float()).to(s["x"].dtype)
    got["rstd"] = rstd
    if case["out"]:
        got["out"] = y
    return dict(got, **_forms(y, case))


def _back_plain(s):
    case, x, dy, rstd = s["case"], s["x"].float(), s["dy"].float(), s["rstd"]
    g = dy * s["w"].float()
    # the mean in 64 bits: results lie next to the borders of 4 bits
    mean = (g.double() * x.double()).sum(1) / x.shape[1]
    part = (mean * rstd.double().square()).float()
    dx = (g - x * part.unsqueeze(1)) * rstd.unsqueeze(1)
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    dx = dx.to(s["x"].dtype)
    dw = (dy * (x * rstd.unsqueeze(1))).sum(0).to(s["w"].dtype)
    return dict(dx=dx, dw=dw, **_forms(dx, case))


# ------------------------------------------------------------------ run --

def _zs():
    import zero_sharded_optimizer_bucket_gb300 as zs
    return zs


def run(s):
    case = s["case"]
    if case["op"] == "norm":
        if own:
            zs = _zs()
            scaler = None if s["scale"] is None else zs.make_loss_scaler(s["scale"], scale_window=0)
            zs.zs_norm_tensors(s["list"], s["scratch"], s["max_norm"], s["norm"], s["coef"], s["flags"], scaler=scaler)
            if case["clip"]:
                zs.zs_clip_tensors(s["list"], s["coef"], s["flags"])
        else:
            _norm_plain(s)
        got = dict(norm=s["norm"], coef=s["coef"], flags=s["flags"])
        if case["clip"]:
            s["max_norm"] *= 0.97           # a threshold that follows the norm down: every pass clips
            got["grad"] = s["grad"]
        return got
    if case["op"] == "matvec":
        if own:
            return _zs().zs_mx4_matvec(s["x"], s["w"], s["out"])
        return (s["x"].float() @ _held(s["w"]["codes"], s["w"]["scales"])[:, :case["k"]].t()).to(s["x"].dtype)
    if case["op"] == "rms":
        if not own:
            return _rms_plain(s)
        zs = _zs()
        zs.zs_rms_norm(s["x"], s["w"], EPS, residual=s["residual"], sum=s.get("sum"), out=s.get("out"), rstd=s["rstd"],
                       rows=s.get("rows"), cols=s.get("cols"))
        got = {k: s[k] for k in ("sum", "rstd", "out") if k in s}
    else:
        if not own:
            return _back_plain(s)
        zs = _zs()
        zs.zs_rms_norm_backward(s["dy"], s["x"], s["w"], s["rstd"], residual=s["residual"], dx=s["dx"], dw=s["dw"],
                                scratch=s["scratch"], rows=s.get("rows"), cols=s.get("cols"))
        got = dict(dx=s["dx"], dw=s["dw"])
    for way in _ways(case):
        got[way] = zs.zs_mx4_dequantize(s[way], s[way]["out"])
    return got


def _tensor_list(zs, s):
    """The library's handle of the tensors, each a run of the flat buffers, its device table and the norm's scratch."""
    items = []
    for n, at in zip(s["numel"], s["start"]):
        t = {k: s[k][at:at + n] for k in ("grad", "master", "exp_avg", "exp_avg_sq")}
        b, e = at // BLOCK, at // BLOCK - (-n // BLOCK)
        t.update(exp_avg_scale=s["exp_avg_scale"][b:e], exp_avg_sq_scale=s["exp_avg_sq_scale"][b:e])
        items.append(t)
    got = zs.zs_build_tensors(items, state_bits=8)
    info = zs.zs_tensors_info(got)
    table = torch.empty(info["device_table_bytes"], dtype=torch.uint8, device="cuda")
    zs.zs_tensors_upload(got, table, table.numel())
    s["scratch"] = torch.empty(info["n_chunks"], dtype=torch.float64, device="cuda")
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        g = s["grad"].double()
        scale = 1024.0 if case["scaled"] else 1.0
        norm = g.norm() / scale
        clip = min(1.0, s["max_norm"] / (float(norm) + float(np.float32(1e-6))))
        got = dict(norm=norm.view(1), coef=torch.full((1,), clip / scale, dtype=torch.float64, device="cuda"),
                   flags=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return dict(got, grad=g * clip) if case["clip"] else got
    if case["op"] == "matvec":
        codes, tiles, k = s["w"]["codes"], s["w"]["scales"], case["k"]
        code = torch.stack([codes % 16, codes // 16], 2).view(codes.shape[0], -1).long()
        mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")[code % 8]
        e = _untile(tiles, code.shape[0], code.shape[1] // GROUP).to(torch.int32) - 127
        w = mag * (1 - 2 * (code // 8)) * _two(e).repeat_interleave(GROUP, 1)
        return s["x"].double() @ w[:, :k].t()
    x, w = s["x"].double(), s["w"].double()
    n = x.shape[1]
    kind = TYPES[case["dtype"]]
    if case["op"] == "rms":
        if case["residual"]:
            x = x + s["residual"].double()
        root = torch.sqrt(torch.einsum("ij,ij->i", x, x) / n + float(np.float32(EPS)))
        y = x / root[:, None] * w
        got = dict(sum=x if case["residual"] else None, rstd=1 / root, out=y if case["out"] else None)
    else:
        r, dy = s["rstd"].double()[:, None], s["dy"].double()
        z = x * r
        y = r * (w * dy - z * torch.einsum("ij,ij->i", w * dy, z)[:, None] / n)
        if case["residual"]:
            y = y + s["residual"].double()
        got = dict(dx=y, dw=torch.einsum("ij,ij->j", dy, z))
    for way in _ways(case):         # 4 bits of the result in its own type
        got[way] = _mx4_64(y.to(kind) if way == "rows" else y.to(kind).t())
    return {k: v for k, v in got.items() if v is not None}
