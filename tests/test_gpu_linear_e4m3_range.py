"""gdn_linear_act of e4m3 codes that differ by many powers of two, and of sums that cancel: how far the 8-bit matrix
instructions may be off for a bf16 out, and that an fp32 out does not have their error.

Eight neighbouring k are added at a time, each product cut toward zero at 2^-13 of the largest one's power of two, so a group is off
by less than 7 2^-13 of its largest product."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests import test_gpu_linear_act as lin

pytestmark = pytest.mark.gpu


def codes(kind, n, K, g):
    t = torch.randn(n, K, generator=g)
    if kind == "binades":
        t = t * torch.exp2(torch.randint(-8, 1, (n, K), generator=g).float())
    elif kind == "outliers":  # a few channels that are 200 times the others
        t[:, 5::64] *= 200
        t = t / 60
    elif kind == "cancel":    # a pair of large products of either sign in each group
        t = t / 100
        t[:, 0::8], t[:, 1::8] = 3.2, 3.2
    elif kind == "small":     # among the subnormal codes
        t = t / 4096
    return (t * 140).clamp(-448, 448).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("kind", ["binades", "outliers", "cancel", "small"])
@pytest.mark.parametrize("M,N,K", [(3, 96, 64), (16, 96, 4096), (40, 64, 1040), (100, 96, 272), (700, 40, 144)])
def test_codes_of_different_size(M, N, K, kind):
    g = torch.Generator().manual_seed(K)
    s = lin.make(M, N, K, "e4m3", False, False, "", "f32")
    s["x"], s["w"] = codes(kind, M, K, g).cuda(), codes(kind, N, K, g).cuda()
    if kind == "cancel":
        s["x"][:, 1::8] = (-s["x"][:, 1::8].float()).to(torch.float8_e4m3fn)
    y, sums, near = lin.want(s, "none", False)
    full = lin.host(lin.call(s, M, N, K))
    assert (np.abs(full - y) <= sums + near + ref.U32 * np.abs(y) + 2.0 ** -126).all()
    s["out"] = s["out"].to(torch.bfloat16)
    got = lin.host(lin.call(s, M, N, K))
    x, w = np.abs(lin.host(s["x"])).reshape(M, K // 8, 8), np.abs(lin.host(s["w"])).reshape(N, K // 8, 8)
    largest = np.zeros((M, N))
    for c in range(0, K // 8, 32):
        largest += (x[:, None, c:c + 32] * w[None, :, c:c + 32]).max(-1).sum(-1)
    cut = 7 * 2.0 ** -13 * largest * lin.host(s["x_scale"])[:, None] * lin.host(s["w_scale"])
    # sums in fp32: of K / 8 groups, of which each may round twice
    bound = cut + 2 * sums + near
    assert (np.abs(got - y) <= bound + ref.HALF["bf16"] * (np.abs(y) + bound) + 2.0 ** -126).all()
    size = np.abs(lin.host(s["x"])) @ np.abs(lin.host(s["w"])).T * lin.host(s["x_scale"])[:, None] * lin.host(s["w_scale"])
    assert (cut < 2.0 ** -10 * size).all()  # never half of what bf16 rounds off a sum of that size
