"""The waits of the low-memory kernels: their limits begin when the previous
kernel has completed.  A kernel that lets its dependents begin at once works
on past the limit and only then writes what the call behind it reads.
Nothing faults, traps or hangs."""
import time

import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs

pytestmark = pytest.mark.gpu
LIMIT = 1.0                            # s, of one wait


def held(rows, cols, seed):
    """A random 4-bit matrix with scales of 1."""
    size = zs.zs_mx4_sizes(rows, cols)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dict(codes=torch.randint(0, 256, (size["code_bytes"],), dtype=torch.uint8, device="cuda", generator=g),
                scales=torch.full((size["scale_bytes"],), 127, dtype=torch.uint8, device="cuda"))


# Each maker gives what is written late, and a function of it that prepares a
# call, stops before it (the call alone has to come behind the late copy: a
# fill in between would wait for it) and then makes it and gives its result.

def product(m, n, k):
    a, b = held(m, k, 1), held(n, k, 2)

    def run(codes):
        out = torch.full((m, n), 77.0, device="cuda")
        torch.cuda.synchronize()
        yield
        yield zs.zs_mx4_matmul(dict(a, codes=codes), b, k, out)
    return a["codes"], run


def quantiser(ld):
    x = torch.randn(300 * ld, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))

    def run(x):
        size = zs.zs_mx4_sizes(300, 999)
        room = torch.zeros(size["code_bytes"] + size["scale_bytes"], dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        yield
        zs.zs_mx4_quantize(x.view(300, ld)[:, :999], rows=dict(codes=room[:size["code_bytes"]], scales=room[size["code_bytes"]:]))
        yield room
    return x, run


def update(bits):
    n = 4096 * 5
    g = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    kind = torch.uint8 if bits == 8 else torch.float32

    def run(grad):
        t = dict(grad=grad, master=torch.zeros(n, device="cuda"), exp_avg=torch.zeros(n, dtype=kind, device="cuda"),
                 exp_avg_sq=torch.zeros(n, dtype=kind, device="cuda"))
        if bits == 8:
            t.update(exp_avg_scale=torch.zeros(n // 256, device="cuda"), exp_avg_sq_scale=torch.zeros(n // 256, device="cuda"))
        lst = zs.zs_build_tensors([t], state_bits=bits)
        table = torch.empty(zs.zs_tensors_info(lst)["device_table_bytes"], dtype=torch.uint8, device="cuda")
        zs.zs_tensors_upload(lst, table, table.numel())
        torch.cuda.synchronize()
        yield
        zs.zs_adam_tensors(lst, dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0), 1)
        yield t["master"]
    return g, run


CALLS = {"pair of SMs": lambda: product(1290, 1801, 704), "pair of SMs, many stages": lambda: product(1290, 1801, 33024),
         "split": lambda: product(200, 300, 8192), "few tokens": lambda: product(5, 300, 8192),
         "quantiser": lambda: quantiser(1000), "quantiser, ragged": lambda: quantiser(1001),
         "8-bit update": lambda: update(8), "32-bit update": lambda: update(32)}


@pytest.mark.parametrize("name", list(CALLS))
def test_previous_kernel_past_the_limit(name):
    late, run = CALLS[name]()
    early = torch.zeros_like(late)
    results = []
    for codes in (late, early):        # the second time without the copy: the kernel is loaded, the result another
        call = run(codes)
        next(call)
        results.append(next(call))
    call = run(early)
    next(call)
    t0 = time.perf_counter()
    zs.zs_test_late_copy(early, late, late.numel() * late.itemsize, int(1.5e9 * LIMIT))
    got = next(call)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 > 1.4 * LIMIT
    assert torch.equal(early, late) and torch.equal(got, results[0]) and not torch.equal(got, results[1])
    assert zs.zs_device_wait_timeouts(reset=True) == 0


@pytest.fixture
def give_up():
    zs.zs_device_wait_timeouts(reset=True)
    yield zs.zs_test_give_up
    zs.zs_test_give_up(-1)
    torch.cuda.synchronize()
    zs.zs_device_wait_timeouts(reset=True)


# sizes, the stage whose wait runs out, and how many tiles of 256 x 256 a pair has finished before (None: not the pairs' kernel)
KINDS = {20: torch.bfloat16, 64: torch.float16, 1290: torch.bfloat16}      # by m; else fp32
GIVE_UP = [(5, 300, 8192, 0, None), (5, 300, 8192, 1, None), (20, 300, 8192, 1, None), (64, 300, 8192, 0, None), (200, 300, 8192, 0, None),
           (200, 300, 8192, 3, None), (100, 9900, 512, 1, None), (5, 40000, 8192, 7, None), (1290, 1801, 704, 0, 0), (1290, 1801, 704, 2, 0),
           (1290, 1801, 4096, 9, 0), (1290, 1801, 33024, 100, 0), (4096, 5120, 512, 3, 1), (4096, 5120, 512, 4, 2)]


@pytest.mark.parametrize("m,n,k,at,finished", GIVE_UP)
def test_product_gives_up(m, n, k, at, finished, give_up):
    """A wait for operands that gives up: no CTA of its tile stores a sum of some parts (pairs leave the tile as it was, the other
    kernel writes NaN); it is counted; the next call is right."""
    a, b = held(m, k, 1), held(n, k, 2)
    launch = zs.zs_test_mx4_launch(m, n, k)
    assert (launch["tmem_columns"] == 512) == (finished is not None)
    out = torch.full((m, n), 77.0, device="cuda", dtype=KINDS.get(m, torch.float32))
    want = zs.zs_mx4_matmul(a, b, k, torch.empty_like(out))
    give_up(at)
    zs.zs_mx4_matmul(a, b, k, out)
    give_up(-1)
    torch.cuda.synchronize()
    assert zs.zs_device_wait_timeouts(reset=True) > 0
    kept = out == 77.0
    if finished is None:
        assert bool(out.isnan().all())
    else:                              # tiles go down the columns of tiles, the pairs one after the other
        tiles = -(-m // 256)
        order = (torch.arange(m, device="cuda") // 256)[:, None] + tiles * (torch.arange(n, device="cuda") // 256)[None, :]
        done = order < finished * (torch.cuda.get_device_properties(0).multi_processor_count // 2)
        assert torch.equal(out[done], want[done]) and bool(kept[~done].all())
    zs.zs_mx4_matmul(a, b, k, out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and zs.zs_device_wait_timeouts() == 0


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_quantiser_gives_up(kind, at, give_up):
    """A CTA whose wait for its unit `at` gives up writes nothing from there on: tiles go row by row, the CTAs one after the other."""
    rows, cols = 20000, 1100
    x = torch.randn(rows, cols + 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(kind)[:, :cols]
    size = zs.zs_mx4_sizes(rows, cols)

    def run():
        h = dict(codes=torch.full((rows, size["row_bytes"]), 0xA5, dtype=torch.uint8, device="cuda"),
                 scales=torch.full((size["scale_bytes"],), 0xA5, dtype=torch.uint8, device="cuda"))
        zs.zs_mx4_quantize(x, rows=h)
        torch.cuda.synchronize()
        return h

    want = run()
    give_up(at)
    got = run()
    give_up(-1)
    assert zs.zs_device_wait_timeouts(reset=True) > 0
    ctas = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    tiles_c = size["scale_bytes"] // 512 // -(-rows // 128)
    # the units of a tile are its columns 0..127, or (fp32) 0..63 and 64..127; 64 bytes a row of a tile
    units = 2 if kind == torch.float32 else 1
    row, byte = torch.meshgrid(torch.arange(rows, device="cuda"), torch.arange(size["row_bytes"], device="cuda"), indexing="ij")
    tile = row // 128 * tiles_c + byte // 64
    unit = tile // ctas * units + (byte % 64) // (64 // units)
    done = unit < at
    assert torch.equal(got["codes"][done], want["codes"][done]) and bool((got["codes"][~done] == 0xA5).all())
    tile = torch.arange(size["scale_bytes"], device="cuda") // 512
    done = tile // ctas * units + units - 1 < at       # a tile's scales come with its last unit
    assert torch.equal(got["scales"][done], want["scales"][done]) and bool((got["scales"][~done] == 0xA5).all())
    for name, t in run().items():
        assert torch.equal(t, want[name])
    assert zs.zs_device_wait_timeouts() == 0


@pytest.mark.parametrize("at", [0, 2])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_update_gives_up(at, kind, rounding, give_up):
    """The blocks of the stage whose wait gives up (8 blocks of 256 of each chunk of 6144) stay as they were, the others are updated."""
    n = 2_000_128                                       # a last block of 256
    g = torch.Generator(device="cuda").manual_seed(5)
    first = dict(grad=(torch.randn(n, device="cuda", generator=g) * 1e-3).to(kind), param=torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
                 master=torch.randn(n, device="cuda", generator=g), exp_avg=torch.full((n,), 0x30, dtype=torch.uint8, device="cuda"),
                 exp_avg_sq=torch.full((n,), 0x31, dtype=torch.uint8, device="cuda"), exp_avg_scale=torch.full((n // 256,), 1e-5, device="cuda"),
                 exp_avg_sq_scale=torch.full((n // 256,), 1e-5, device="cuda"))

    def run():
        t = {k: v.clone() for k, v in first.items()}
        lst = zs.zs_build_tensors([t], state_bits=8)
        info = zs.zs_tensors_info(lst)
        assert info["n_chunks"] == -(-n // 6144)
        table = torch.empty(info["device_table_bytes"], dtype=torch.uint8, device="cuda")
        zs.zs_tensors_upload(lst, table, table.numel())
        zs.zs_adam_tensors(lst, dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01), 2, rounding=rounding, seed=7)
        torch.cuda.synchronize()
        return t

    want = run()
    give_up(at)
    got = run()
    give_up(-1)
    assert zs.zs_device_wait_timeouts(reset=True) > 0
    kept = torch.arange(n, device="cuda") % 6144 // 2048 == at
    for name, t in got.items():
        held_up = kept[::256] if name.endswith("scale") else kept
        assert torch.equal(t[held_up], first[name][held_up]), name
        assert torch.equal(t[~held_up], want[name][~held_up]), name
    for name, t in run().items():
        assert torch.equal(t, want[name])
    assert zs.zs_device_wait_timeouts() == 0
