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
