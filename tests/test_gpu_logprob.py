"""gdn_logprob against its formulas in 64 bits; ranks and alternatives are whole numbers and have to be equal."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu
INF = float("inf")


def call(logits, ids=None, temperature=1.0, top_k=0, stats=True, n=None, rank=True, logprob=True):
    n, v = logits.shape[0] if n is None else n, logits.shape[1]
    m = 0 if ids is None else ids.shape[1]
    out = {}
    if stats:
        out.update(lse=torch.full((n,), 7.0, device="cuda"), entropy=torch.full((n,), 7.0, device="cuda"))
    if m and logprob:
        out["logprob"] = torch.full((n, m), 7.0, device="cuda")
    if m and rank:
        out["rank"] = torch.full((n, m), 77, dtype=torch.int32, device="cuda")
    if top_k:
        out["top_ids"] = torch.full((n, top_k), 77, dtype=torch.int32, device="cuda")
        out["top_logprob"] = torch.full((n, top_k), 7.0, device="cuda")
    need = gdn.gdn_logprob_workspace_bytes(n, v, logits.dtype, m, top_k)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda") if need else None
    gdn.gdn_logprob(logits, n, v, ids=ids, temperature=temperature, workspace=ws, **out)
    torch.cuda.synchronize()
    if need:
        assert (ws[need:] == 255).all()
    return {k: t.cpu().numpy() for k, t in out.items()}


def check(logits, got, ids=None, temperature=1.0, top_k=0):
    x = logits.double().cpu().numpy()
    want = ref.logprob(x, None if ids is None else ids.cpu().numpy(), temperature, top_k)
    for k in ("rank", "top_ids"):
        if k in got:
            assert np.array_equal(got[k], want[k]), (k, np.argwhere(got[k] != want[k])[:5])
    # e^d for d = (l - max) is off by |d| + 6 half steps (the difference, the factor log2(e) / T and the power), which
    # e^d |d| <= 1/e keeps to 7 of the sum of them all; a lane adds up to V / 64 values of one sign, and 16 sums meet
    # behind it; log s and the sum with the maximum round once each
    rel = (16 + x.shape[1] / 64 + 16) * ref.U32
    top = np.where(np.isfinite(x), x, -np.inf).max(1)
    size = np.abs(np.where(np.isfinite(top), top, 0)) / temperature
    for k in ("lse", "logprob", "top_logprob", "entropy"):
        if k not in got:
            continue
        g, w = got[k].astype(np.float64), want[k]
        w = np.where(w < -3.4028235677973366e38, -INF, w)  # what rounds to -infinity in fp32: below -(2 - 2^-24) 2^127
        assert np.array_equal(np.isnan(g), np.isnan(w)), k
        f = np.isfinite(w)
        assert np.array_equal(g[~f & ~np.isnan(w)], w[~f & ~np.isnan(w)]), k
        if k == "entropy":  # log s - u / s, and |u| / s is the entropy's size
            tol = 3 * rel * (1 + np.abs(w))
        else:
            tol = rel + 8 * ref.U32 * (np.abs(w) + (size if w.ndim == 1 else size[:, None]))
        assert (np.abs(g - w)[f] <= np.broadcast_to(tol, w.shape)[f]).all(), (k, np.abs(g - w)[f].max())


def make(n, v, dtype="bf16", seed=0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(n, v, generator=g)
    x[torch.arange(n), torch.randint(0, v, (n,), generator=g)] += 10 * torch.rand(n, generator=g)
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def some_ids(n, v, m, seed=1):
    ids = torch.randint(0, v, (n, m), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    if m > 1:
        ids[:, 1] = -1
    if m > 2:
        ids[:, 2] = v
    if m > 3:
        ids[:, 3] = ids[:, 0]  # the same token twice
    return ids.cuda()


SIZES = [(1, 1), (1, 2), (3, 7), (2, 64), (5, 100), (4, 511), (3, 1000), (2, 4096), (2, 8191), (3, 8193), (1, 16385), (2, 32001),
         (300, 257), (1, 131072), (3, 131071), (2, 200003)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", SIZES)
def test_sizes(n, v, dtype):
    x = make(n, v, dtype, seed=v)
    for m, k, t in ((1, min(5, v), 1.0), (4, min(64, v), 0.7), (0, min(20, v), 1.3), (2, 0, 1.0)):
        ids = some_ids(n, v, m) if m else None
        check(x, call(x, ids, t, k), ids, t, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_drafted_token_is_the_argmax_or_near(dtype):
    x = make(40, 5000, dtype)
    ids = torch.stack([x.argmax(1), x.argmin(1), x.float().topk(3, 1).indices[:, 2]], 1).to(torch.int32)
    got = call(x, ids, 1.0, 10)
    check(x, got, ids, 1.0, 10)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [50, 1000, 9001, 70000])
def test_ties(v, dtype):
    """Equal logits: a row of one value, of two, of few; the lower index comes first."""
    g = torch.Generator().manual_seed(v)
    x = torch.stack([torch.full((v,), 1.5), torch.randint(0, 2, (v,), generator=g).float(),
                     torch.randint(-3, 4, (v,), generator=g).float(), torch.zeros(v) * -torch.randint(0, 2, (v,), generator=g),
                     torch.arange(v).float() // 8, -(torch.arange(v).float() // 8)])
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    ids = some_ids(len(x), v, 5)
    for k in (1, min(40, v), min(64, v)):
        check(x, call(x, ids, 1.0, k), ids, 1.0, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [3, 700, 20000])
def test_masked_rows(v, dtype):
    x = make(7, v, dtype).float()
    lowest = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min
    x[0] = -INF                       # nothing is left
    x[1, : v - 1] = -INF              # one token is left
    x[2, torch.arange(v) % 3 > 0] = -INF
    x[3] = lowest                     # a mask of the type's lowest value everywhere
    x[4, 1:] = lowest
    x[5, ::2] = lowest
    x[6, 0], x[6, 1] = -lowest, lowest
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    ids = some_ids(7, v, 2)
    ids[:, 1] = v - 1
    k = min(10, v)
    check(x, call(x, ids, 1.0, k), ids, 1.0, k)


@pytest.mark.parametrize("v", [40, 3000, 50001])
def test_nan_and_infinity(v):
    x = make(6, v, "f32")
    x[0, v // 2] = float("nan")
    x[1, 7] = INF
    x[2, 7], x[2, 9] = INF, INF
    x[3, 5], x[3, 6] = -INF, float("nan")
    x[4] = float("nan")
    ids = some_ids(6, v, 3)
    ids[:, 2] = 7
    for x in (x, x.to(torch.bfloat16)):
        check(x, call(x, ids, 1.0, 12), ids, 1.0, 12)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (0, 1), (8, 8), (4, 2)])
def test_rows_at_any_place(offset, pad, dtype):
    """Rows that start and end inside a run of 16 bytes, with NaN around them."""
    n, v = 5, 4099
    x = make(n, v, dtype)
    wide = torch.full((offset + n * (v + pad),), float("nan"), dtype=x.dtype, device="cuda")
    rows = wide[offset:].view(n, v + pad)[:, :v]
    rows.copy_(x)
    ids = some_ids(n, v, 2)
    check(x, call(rows, ids, 1.0, 8), ids, 1.0, 8)


def test_few_outputs_fewer_rows_and_none():
    x = make(9, 3001)
    ids = some_ids(9, 3001, 2)
    full = call(x, ids, 1.0, 6)
    assert np.array_equal(call(x, ids, stats=False, logprob=False)["rank"], full["rank"])
    assert np.array_equal(call(x, ids, stats=False, rank=False)["logprob"], full["logprob"])
    assert np.array_equal(call(x, top_k=6, stats=False)["top_ids"], full["top_ids"])
    part = call(x, ids, 1.0, 6, n=4)
    assert all(np.array_equal(part[k], full[k][:4]) for k in full)
    lse = torch.full((9,), 7.0, device="cuda")
    gdn.gdn_logprob(x, 0, 3001, lse=lse)
    need = gdn.gdn_logprob_workspace_bytes(4, 3001, x.dtype)
    gdn.gdn_logprob(x, 4, 3001, lse=lse, workspace=torch.empty(max(16, need), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert (lse[4:] == 7).all() and np.array_equal(lse[:4].cpu().numpy(), full["lse"][:4])


@pytest.mark.parametrize("n,v", [(1, 131072), (64, 32001)])
def test_another_stream_a_graph_and_the_same_bits(n, v):
    x, ids = make(n, v), some_ids(n, v, 3)
    first = call(x, ids, 1.0, 20)
    out = {k: torch.from_numpy(t).cuda() for k, t in first.items()}
    ws = torch.empty(max(16, gdn.gdn_logprob_workspace_bytes(n, v, x.dtype, 3, 20)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_logprob(x, n, v, ids=ids, workspace=ws, **out)
    for _ in range(3):
        for t in out.values():
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(t.cpu().numpy(), first[k]) for k, t in out.items())
        again = call(x, ids, 1.0, 20)
        assert all(np.array_equal(again[k], first[k]) for k in first)
