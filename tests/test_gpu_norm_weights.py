"""gdn_norm with weights that take s * weight past fp32's range."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.test_gpu_norm import call, check, host, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["f32", "e4m3", "i8"])
@pytest.mark.parametrize("d", [8, 64, 100, 5120])
def test_weights_of_any_size(d, out):
    """s * weight passes fp32's range where the norm does not; every finite row has its norm."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn(6, 1, d, generator=g)
    w = 1 + 0.2 * torch.randn(d, generator=g)
    x[1] *= 1e15
    x[2] *= 1e30
    x[3] *= 1e18
    x[4] *= 1e-10
    x[5] = x[5].clamp(-3, 3) * 1e38
    for f in (1e25, 3e35, 1e37):
        s = make(6, 1, d, "f32", "", out)
        s["x"], s["weight"] = x.cuda(), (w * f).cuda()
        call(s, 6, eps=1e-30)
        want_s, y = ref.norm(x.double().numpy(), host(s["weight"]), eps=1e-30)
        assert np.abs(y).max() < 3.4e38
        check(s, out, want_s, y)
