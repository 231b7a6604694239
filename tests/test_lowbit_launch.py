"""What the 4-bit product's launches ask of an SM (host only): the CTAs that
fit one by their shared memory find all the tensor memory they allocate.

tcgen05.alloc waits without a bound, and a CTA of a split keeps its columns
until the other CTAs of its cluster have theirs; CTAs of any calls, on any
streams, may share an SM."""
import random

import pytest

import zero_sharded_optimizer_bucket_gb300 as zs

SHARED, COLUMNS, RESERVED = 228 * 1024, 512, 1024     # of an SM; of shared memory, per CTA, by the runtime


def shapes():
    """Each tile width and every number of stages, split or not, then sizes at random."""
    for m in (1, 16, 17, 32, 33, 64, 65, 128, 129, 300, 1024, 8192):
        for n in (1, 128, 129, 1024, 2432, 4096, 9800, 14336):
            for k in (1, 256, 257, 512, 1024, 2048, 4096, 4097, 14336, 32800):
                yield m, n, k
    rng = random.Random(1)
    for _ in range(2000):
        yield tuple(int(2 ** rng.uniform(0, 15)) for _ in range(3))


def test_tensor_memory_is_there():
    """A CTA's share of the SM's shared memory is at least a fifth for each 128 columns, and a little more: five such shares
    do not fit, so no mixture of CTAs wants more than 512 columns."""
    seen = set()
    for shape in shapes():
        got = zs.zs_test_mx4_launch(*shape)
        assert got["tmem_columns"] in (128, 256, 512)
        assert got["shared_bytes"] <= 227 * 1024
        parts = got["tmem_columns"] // 128
        assert 5 * got["shared_bytes"] > parts * SHARED, (shape, got)
        assert SHARED // (got["shared_bytes"] + RESERVED) * got["tmem_columns"] <= COLUMNS, (shape, got)
        seen.add((got["tmem_columns"], got["split"] > 1, got["stages"] == 1))
    assert {(128, True, True), (128, False, True), (256, True, False), (256, False, True), (512, False, False)} <= seen


def test_launch_refusals():
    for bad in ((0, 1, 1), (1, -1, 1), (1, 1, 1 << 31)):
        with pytest.raises(zs.ZsError):
            zs.zs_test_mx4_launch(*bad)
