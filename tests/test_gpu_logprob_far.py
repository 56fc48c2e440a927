"""gdn_logprob where the logits, or what masks them, are large finite numbers: their powers of two, log2(e) / T times the
logit, pass the range in which fp32 still tells neighbouring whole numbers apart."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.test_gpu_logprob import call, make, some_ids

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FILLS = [-1e9, -5e9, -1e10, -1e11, -1e12, -1e15, -1e18, -1e30]
# one slice of one batch, one of several, several slices; (600, 40000) has one slice and several batches
SIZES = [(1, 50), (1, 9001), (1, 70_001), (600, 40_000)]


def near(logits, got, ids, temperature, top_k, copies=1):
    """check(), of rows that repeat as copies (at other places in 16 bytes, and so with other orders of their sums), with what large arguments add.  Sums are against a whole number of powers of two that is next to the maximum's
    own up to half a step of fp32 there: 2^-24 of it and 1/2, and at most 33 (from 2^30 on logits are counted).  A power's
    argument and log s are that much larger, and so are their roundings: two half steps each, and one for every addition of
    the terms that the entropy weighs by it."""
    x = logits.double().cpu().numpy()
    want = ref.logprob(x, None if ids is None else ids.cpu().numpy(), temperature, top_k)
    want = {k: np.concatenate([w] * copies) for k, w in want.items()}
    for k in ("rank", "top_ids"):
        if k in got:
            assert np.array_equal(got[k], want[k]), (k, np.argwhere(got[k] != want[k])[:5])
    top = np.where(np.isfinite(x), x, -np.inf).max(1)
    size = np.concatenate([np.abs(np.where(np.isfinite(top), top, 0)) / temperature] * copies)
    beside = np.minimum(2.0 ** -24 * 1.4427 * size + 0.5, 33)
    rel = (16 + x.shape[1] / 64 + 16) * ref.U32
    for k in ("lse", "logprob", "top_logprob", "entropy"):
        if k not in got:
            continue
        g, w = got[k].astype(np.float64), want[k]
        w = np.where(w < -3.4028235677973366e38, -np.inf, w)
        assert np.array_equal(np.isnan(g), np.isnan(w)), (k, g[np.isnan(g) != np.isnan(w)][:5])
        f = np.isfinite(w)
        assert np.array_equal(g[~f & ~np.isnan(w)], w[~f & ~np.isnan(w)]), k
        by_row = lambda a: a if w.ndim == 1 else a[:, None]  # noqa: E731
        if k == "entropy":
            tol = 3 * rel * (1 + np.abs(w) + beside)
        else:  # a log probability is a difference of logits, whatever their size
            tol = rel + 8 * ref.U32 * (np.abs(w) + by_row(beside) + (by_row(size) if k == "lse" else 0))
        assert (np.abs(g - w)[f] <= np.broadcast_to(tol, w.shape)[f]).all(), (k, np.abs(g - w)[f].max())


def run(rows, dtype, n, temperature=1.0, top_k=10):
    """rows repeated to n of them."""
    x = torch.stack(rows).to(TYPES[dtype]).cuda()
    m, v = x.shape
    ids = some_ids(m, v, 2)
    ids[:, 1] = v - 1
    more = max(1, -(-n // m))
    k = min(top_k, v)
    got = call(x.repeat(more, 1), ids.repeat(more, 1), temperature, k)
    near(x, got, ids, temperature, k, more)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", SIZES)
def test_masks_of_large_finite_values(n, v, dtype):
    """The first half, the second, all but nine tokens, a run of 16 bytes, and one batch's worth of every row masked."""
    rows = []
    for i, fill in enumerate(FILLS):
        x = make(1, v, "f32", seed=i)[0].cpu()
        x[[slice(0, v // 2), slice(v // 2, v), slice(0, max(v - 9, 1)), slice(16, 24), slice(0, 16384)][i % 5]] = fill
        if i % 5 == 4:
            x[-20:] = torch.arange(20.0)
        rows.append(x)
        y = make(1, v, "f32", seed=i + 50)[0].cpu()
        y[torch.arange(v) % 3 > 0] = fill
        rows.append(y)
    run(rows, dtype, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", SIZES)
def test_rows_of_a_mask_alone(n, v, dtype):
    """Every logit masked by the same value, and by two."""
    rows = [torch.full((v,), f) for f in FILLS]
    rows.append(torch.where(torch.arange(v) < v // 3, torch.tensor(-1e12), torch.tensor(-1e10)))
    rows.append(torch.where(torch.arange(v) % 7 == 2, torch.tensor(-2.0 ** 30), torch.tensor(-1e18)))
    run(rows, dtype, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", SIZES)
def test_large_logits(n, v, dtype):
    """Tops from 2^24 to 10^18, alone, several alike, and among others of either size."""
    rows = []
    g = torch.Generator().manual_seed(v)
    for i, top in enumerate([2.0 ** 24 + 6, 3e8, 6.2e8, 7.4e8, 7.5e8, 1.5e9, 3e9, 5e9, 1.2e10, 1e12, 1e15, 1e17, 1e18]):
        x = 2.5 * torch.randn(v, generator=g)
        at = torch.randint(0, v, (3,), generator=g)
        x[at[:1 + i % 3]] = top
        rows.append(x)
        rows.append(torch.rand(v, generator=g) * top)
        rows.append(-top * (1 + torch.rand(v, generator=g)))
    run(rows, dtype, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.6, 0.1, 2.0 ** -10, 2.0 ** -20, 2.0 ** 20])
def test_temperatures(temperature, dtype):
    for n, v in ((1, 50), (1, 70_001), (600, 9001)):
        rows = [s * make(1, v, "f32", seed=i)[0].cpu() for i, s in enumerate((1.0, 30.0, 400.0, 2000.0, -2000.0, 1e9, 1e12))]
        for fill in (-1e9, -1e10, -3e18):
            x = make(1, v, "f32", seed=9)[0].cpu()
            x[: v - 20] = fill
            rows.append(x)
        run(rows, dtype, n, temperature)


def test_entropy_is_never_negative():
    """Rows that are sure of a token: log s and u / s are equal up to their roundings."""
    n, v = 4000, 300
    x = torch.full((n, v), -60.0)
    x[torch.arange(n), torch.arange(n) % v] = 37.0 * torch.rand(n, generator=torch.Generator().manual_seed(1))
    for t in (1.0, 0.7, 3.0):
        for rows in (x, x.to(torch.bfloat16)):
            assert (call(rows.cuda(), temperature=t)["entropy"] >= 0).all()


def test_log_probabilities_beside_a_maximum_of_the_other_sign():
    """The difference of two logits passes fp32's range, and divided by T it does not."""
    x = torch.zeros((3, 40))
    x[0, 3], x[0, 5] = 3e38, -3e38
    x[1, 3], x[1, 5] = 1e38, -3.3e38
    x[2, 3], x[2, 5] = 3.4e38, -3.4e38
    for t in (4.0, 1000.0):
        run(list(x), "f32", 1, t)
        run(list(x), "bf16", 1, t)
