"""gdn_norm takes a weight of exactly one head."""

import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu


def test_a_weight_is_of_one_head():
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    out = torch.empty_like(x)
    for n in (63, 65, 128):
        with pytest.raises(gdn.GdnError, match="weight has shape"):
            gdn.gdn_norm(x, torch.ones(n, device="cuda"), out, 3)
    with pytest.raises(gdn.GdnError, match="weight has shape"):
        gdn.gdn_norm(x, torch.ones(2, 64, device="cuda"), out, 3)
    gdn.gdn_norm(x, torch.ones(64, device="cuda"), out, 3)
    torch.cuda.synchronize()
