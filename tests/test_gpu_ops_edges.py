"""The decoding operators at the ends of their ranges, against their plain 64-bit forms."""
import math

import pytest
import torch

import ops_plain as R
from sync_protocols_amd import ops
from test_gpu_ops import check_norm, check_route, dev, run_moe, run_w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


# ----------------------------------------------------------------- products
# Every sum of a group is at most 15 sum |x| s and is rounded once an element, the one of x as often; then the groups'.
@pytest.mark.parametrize("rows", [1, 5, 20, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_group", [0, 128])
def test_w4_small_elements_beside_a_large_one(rows, group, x_group):
    """One element of 448 where the weight is its zero point, 2^-5 elsewhere: what is left is the small elements' sum."""
    k, n = 256, 48
    x = torch.full((rows, k), 2.0 ** -5)
    q = torch.full((n, k), 1, dtype=torch.uint8)
    for t in range(rows):
        x[t, 17 + t % 3] = 448.0
        x[t, 140 + t % 3] = -448.0
    q[:, 17:20] = q[:, 140:143] = 15
    packed = q[:, 0::2] | q[:, 1::2] << 4
    s, z = torch.ones(n, k // group).bfloat16(), torch.full((n, k // group), 15, dtype=torch.uint8)
    x = x.to(torch.float8_e4m3fn)
    xs = torch.ones((rows, k // 128) if x_group else rows)
    got = ops.w4_linear(dev(x), ops.W4Weight(*dev(packed, s, z)), x_scale=dev(xs))
    want = x.double() @ R.w4_values(packed, s, z).t()
    tol = (2 * group + 8) * R.U * 15 * x.double().abs().sum(1, keepdim=True)
    R.close(got, want, tol + R.BF16_HALF * (want.abs() + tol), "out")
