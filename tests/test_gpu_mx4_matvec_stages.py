"""zs_mx4_matvec where a CTA's tokens do not lie in shared memory at once: stage
after stage of k, the next one's on their way while one is multiplied.
Tolerances as in test_gpu_mx4_matvec.py.
"""
import numpy as np
import pytest
import torch

import zero_sharded_optimizer_bucket_gb300 as zs
from tests import lowbit_ref as ref
from tests.test_gpu_mx4_matvec import check
from tests.test_gpu_rms_norm import Mat, same
from tests.test_gpu_tensors import KINDS

pytestmark = pytest.mark.gpu
DTYPE = {"bf16": zs.ZS_DTYPE_BF16, "fp16": zs.ZS_DTYPE_FP16, "fp32": zs.ZS_DTYPE_FP32}
# tokens that fill each width of the kernel, and some less (one 16-bit token of 65536 values fits at once)
TOKENS = {"bf16": (8, 7, 16, 13, 32, 23, 64), "fp16": (8, 16, 11, 32, 64, 50), "fp32": (4, 3, 8, 16, 11, 64)}
# the smallest weight of these that is taken in stages
WEIGHTS = [(n, k) for k in (4096, 8200, 14336, 28672, 70000) for n in (1500, 4096, 14336)]


def stages(m, n, k, kind):
    got = zs.zs_test_mx4_matvec_launch(m, n, k, DTYPE[kind])
    return -(-got["units"] // got["stage"])


def weight(n, k, seed):
    """test_gpu_mx4_matvec's, decoded on the GPU: n k is large here."""
    kp = -(-k // 32) * 32
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = torch.randint(0, 16, (n, kp), dtype=torch.uint8, device="cuda", generator=g)
    code[:, k:] = 0
    byte = torch.randint(114, 127, (n, kp // 32), device="cuda", generator=g)
    held = dict(codes=(code[:, 0::2] | code[:, 1::2] << 4).contiguous(), scales=torch.from_numpy(ref.tile_scales(byte.cpu().numpy().astype(np.uint8))).cuda())
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    w = table[code.int()].view(n, -1, 32) * torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), byte - 127)[:, :, None]
    return held, w.view(n, kp)[:, :k]


CASES = [(kind, m) for kind in TOKENS for m in TOKENS[kind]]


@pytest.mark.parametrize("kind,m", CASES)
@pytest.mark.parametrize("less", [0, 1, 6])
def test_stages(kind, m, less):
    """less: k is not whole pieces, nor the last stage full."""
    found = [(n, k - less) for n, k in WEIGHTS if stages(m, n, k - less, kind) > 1]
    assert found, (kind, m)
    n, k = found[0]
    held, w = weight(n, k, m + less)
    g = torch.Generator(device="cuda").manual_seed(m)
    x = (torch.randn(m, k, device="cuda", generator=g) * 10.0 ** (2 * torch.rand(m, 1, device="cuda", generator=g) - 1)).to(KINDS[kind])
    first = check(x, held, w, "fp32")
    # rows of x that are not aligned go another way, to the same bits
    again = check(Mat(m, k, kind, x, 3, 1).t, held, w, "fp32")
    assert same(first, again)


def test_every_width_in_many_stages():
    """Rings that go around over the stages, and stages of each width of the kernel."""
    seen = set()
    for kind, m in CASES:
        for n, k in WEIGHTS:
            got = zs.zs_test_mx4_matvec_launch(m, n, k, DTYPE[kind])
            assert got["stage"] % got["warps_k"] == 0 and 2 <= got["depth"] <= 4 and got["shared_bytes"] <= 227 * 1024
            if -(-got["units"] // got["stage"]) > 2:
                seen.add((kind, min(got["tokens"], 32)))
    assert {("bf16", 8), ("bf16", 16), ("bf16", 32), ("fp16", 8), ("fp16", 16), ("fp16", 32), ("fp32", 4), ("fp32", 8), ("fp32", 16)} <= seen


@pytest.mark.parametrize("bad", [(0, 1, 1, 0), (1025, 1, 1, 0), (1, 0, 1, 0), (1, 1, 1 << 31, 0), (1, 1, 1, 3)])
def test_launch_refusals(bad):
    with pytest.raises(zs.ZsError):
        zs.zs_test_mx4_matvec_launch(*bad)
