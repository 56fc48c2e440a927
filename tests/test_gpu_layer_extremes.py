"""gdn_norm, gdn_linear_act and gdn_logprob at the largest numbers of rows and columns that they take, and at the smallest K."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import test_gpu_linear_act as lin

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [8, 24, 56, 72])
@pytest.mark.parametrize("M", [1, 17, 40, 130, 1100])
def test_k_of_few_values(M, K):
    for gated, N in ((False, 100), (True, 33)):
        s = lin.make(M, N, K, "bf16", gated, True, "f32", "f32", seed=K)
        lin.check(s, lin.call(s, M, N, K, "silu", gated), M, N, "silu", gated)


@pytest.mark.parametrize("M,N", [((1 << 26) - 1, 1), (1, (1 << 26) - 1), (3, (1 << 25) + 5)])
def test_products_of_the_most_rows_and_columns(M, N):
    K = 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-3, 4, (M, K), device="cuda", generator=g, dtype=torch.int8)
    w = torch.randint(-3, 4, (N, K), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.full((M,), 0.5, device="cuda"), torch.full((N,), 4.0, device="cuda")
    out = torch.empty((M, N), device="cuda")
    need = gdn.gdn_linear_act_workspace_bytes(M, N, K, torch.int8)
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    gdn.gdn_linear_act(x, w, out, M, N, K, x_scale=xs, w_scale=ws, workspace=work)
    for i in range(M if N > M else N):  # whole numbers: exact
        if N > M:
            want = (w.float() * x[i].float()).sum(1)
            assert torch.equal(out[i], 2 * want)
        else:
            want = (x.float() * w[i].float()).sum(1)
            assert torch.equal(out[:, i], 2 * want)


def test_norms_of_the_most_rows():
    n, heads = 1 << 23, 8
    x = torch.randint(1, 5, (n, heads, 2), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    out = torch.empty((n, heads, 2), dtype=torch.int8, device="cuda")
    scale = torch.empty((n, heads), device="cuda")
    gdn.gdn_norm(x, None, out, n, scale=scale, mode=gdn.GDN_NORM_NONE)
    most = x.float().amax(-1)
    assert torch.equal(scale, most / 127)
    assert torch.equal(out, torch.round(x.float() * (1 / scale)[..., None]).to(torch.int8))


def test_log_probabilities_of_the_most_rows():
    n = 1 << 26
    x = torch.randn(n, 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    lse, lp = torch.empty(n, device="cuda"), torch.empty((n, 1), device="cuda")
    ids, rank = torch.zeros((n, 1), dtype=torch.int32, device="cuda"), torch.empty((n, 1), dtype=torch.int32, device="cuda")
    gdn.gdn_logprob(x, n, 1, ids=ids, lse=lse, logprob=lp, rank=rank)
    # (K + log2 s) ln 2 of one value: the factor, its power, the logarithm, their sum and the last product, half a step each or
    # a whole one, of it or of 1
    assert ((lse - x[:, 0]).abs() <= 8 * 2.0 ** -24 * (x[:, 0].abs() + 1)).all()
    assert (lp.abs() <= 8 * 2.0 ** -24).all() and not rank.any()


def test_the_longest_row():
    v = 1 << 24
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(1, v, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dtype)
        x[0, v - 1], x[0, 12345] = 20.0, 19.0
        ids = torch.tensor([[v - 1, 12345]], dtype=torch.int32, device="cuda")
        out = {"lse": torch.empty(1, device="cuda"), "logprob": torch.empty((1, 2), device="cuda"),
               "rank": torch.empty((1, 2), dtype=torch.int32, device="cuda"),
               "top_ids": torch.empty((1, 2), dtype=torch.int32, device="cuda"), "top_logprob": torch.empty((1, 2), device="cuda")}
        need = gdn.gdn_logprob_workspace_bytes(1, v, dtype, 2, 2)
        gdn.gdn_logprob(x, 1, v, ids=ids, workspace=torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), **out)
        want = torch.logsumexp(x.double(), 1)
        # a lane adds V / (64 slices x 256) values of one sign, 16 more sums meet
        tol = (16 + v / (64 * 256) + 16) * 2.0 ** -24 + 8 * 2.0 ** -24 * 40
        assert (out["lse"].double() - want).abs().item() <= tol
        assert out["rank"].tolist() == [[0, 1]] and out["top_ids"].tolist() == [[v - 1, 12345]]
        assert np.allclose(out["logprob"].cpu().numpy(), [[20 - want.item(), 19 - want.item()]], rtol=0, atol=2 * tol)
        assert torch.equal(out["logprob"], out["top_logprob"])
