"""gdn_logprob's alternatives where a finite value masks most of a row, so that few logits are above it and very many equal:
the equal ones come by their index, and the row costs what one masked by -infinity does."""

import pytest
import torch

from tests.test_gpu_logprob_far import run
from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu


def allowed(v, at, fill, seed=0):
    x = torch.full((v,), fill)
    at = torch.as_tensor(at) % v
    x[at] = 2.5 * torch.randn(len(at), generator=torch.Generator().manual_seed(seed))
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(1, 3), (1, 70), (1, 1601), (1, 9001), (2, 70_001), (600, 20_011)])
@pytest.mark.parametrize("top_k", [1, 20, 64])
def test_few_allowed_tokens(n, v, dtype, top_k):
    rows = []
    for i, fill in enumerate((-1e30, -1e10, -100.0, 0.0)):
        rows.append(allowed(v, [v - 1], fill))
        rows.append(allowed(v, [0, 1, v - 2], fill, i))
        rows.append(allowed(v, range(7, 15), fill, i))                       # a run of 16 bytes, and of the next
        rows.append(allowed(v, range(v // 2, v // 2 + 30), fill, i))
        rows.append(allowed(v, range(0, v, max(v // 19, 1)), fill, i))       # spread, in number next to top_k
        rows.append(allowed(v, range(v - 300, v), fill, i))                  # none before the last batch
        rows.append(allowed(v, range(3, 3 + 400), fill, i))
    x = torch.full((v,), 1.0)                                               # two and three values, in runs
    x[v // 3: v // 3 + 5], x[-7:] = 2.0, -3.0
    rows.append(x)
    y = torch.full((v,), -1e10)
    y[: v // 2] = -1e12
    y[v // 2 + 9: v // 2 + 12] = 4.0
    rows.append(y)
    z = torch.zeros(v)
    z[::2] = -0.0
    z[v // 4: v // 4 + 10] = -1.0
    rows.append(z)
    run(rows, dtype, n, top_k=top_k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_periods_that_meet_the_same_threads(dtype):
    """Allowed tokens 256 runs of 16 bytes apart, which one thread of a workgroup holds all of, and rising values."""
    v, per = 120_011, 4096
    t = torch.arange(v)
    rows = []
    for step in (per // 4, per // 2, per):
        rows.append(torch.where(t % step < 6, (t % 977).float() / 64, torch.tensor(-1e10)))
        rows.append(torch.where(t % step < 6, (t // step).float(), torch.tensor(-1e10)))
        rows.append(torch.where(t % step < 6, torch.tensor(1.0), torch.tensor(-1e10)))
    for n in (1, 600):
        run(rows, dtype, n, top_k=20)


@pytest.mark.parametrize("n,v", [(1, 131_072), (600, 32_768)])
def test_a_finite_mask_costs_what_an_infinite_one_does(n, v):
    def least(fill):
        x = allowed(v, range(9000, 9008), fill).to(torch.bfloat16).cuda().repeat(n, 1)
        k = 20
        out = {"lse": torch.empty(n, device="cuda"), "top_ids": torch.empty((n, k), dtype=torch.int32, device="cuda"),
               "top_logprob": torch.empty((n, k), device="cuda")}
        ws = torch.empty(max(16, gdn.gdn_logprob_workspace_bytes(n, v, x.dtype, 0, k)), dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(30):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                gdn.gdn_logprob(x, n, v, workspace=ws, **out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 100)
        return min(times)

    base = least(float("-inf"))
    got = {fill: least(fill) for fill in (-1e10, -1e30, torch.finfo(torch.bfloat16).min)}
    assert all(t <= 2 * base for t in got.values()), (base, got)  # us; one more pass at most, of which the first loads suffice here
