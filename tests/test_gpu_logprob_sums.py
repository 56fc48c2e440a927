"""gdn_logprob over very long rows of equal logits, where every addition of one long chain would round the same way."""

import math

import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v", [(1, 1 << 24), (600, 131_071), (600, 1 << 22), (520, 1 << 24)])
def test_long_rows_of_equal_logits(n, v, dtype):
    for value in (0.0, 0.3, 0.61, 1.7, 2.9):
        x = torch.full((1, v), value, dtype=dtype, device="cuda").expand(n, v)
        lse, entropy = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        need = gdn.gdn_logprob_workspace_bytes(n, v, dtype, 0, 0)
        gdn.gdn_logprob(x, n, v, lse=lse, entropy=entropy, workspace=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"))
        # a thread adds up to 64 logits a batch, its batches of 32 KiB, and 16 sums meet; the slices' sums (64) besides
        rel = (64 + v * x.element_size() / 32768 + 16 + 64) * ref.U32
        got = x[0, 0].item()
        assert (lse.double() - (got + math.log(v))).abs().max().item() <= rel + 8 * ref.U32 * 20
        assert (entropy.double() - math.log(v)).abs().max().item() <= 3 * rel + 8 * ref.U32 * 20
