"""gdn_norm, gdn_linear_act and gdn_logprob at the ends of what a call may be: offsets past 2^31, rows that repeat, two
calls at once, more slices than one, and logits whose order is the worst for the list of candidates."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import layer_ref as ref
from tests import test_gpu_linear_act as lin
from tests import test_gpu_logprob as logp
from tests import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


def test_norm_rows_past_2_31_elements():
    n, d = 270_000, 8192
    x = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, 1, d, device="cuda").bfloat16()
    s = {"x": x, "weight": None, "residual": None, "total": None, "scale": torch.empty((n, 1), device="cuda"),
         "out": torch.empty((n, 1, d), dtype=torch.int8, device="cuda")}
    norm.call(s, n)
    tail = {"total": None, "out": s["out"][-3:], "scale": s["scale"][-3:]}
    norm.check(tail, "i8", *ref.norm(norm.host(x[-3:])))
    assert not s["scale"][:-3].any()


@pytest.mark.parametrize("M", [3, 70])
def test_product_of_rows_far_apart(M):
    """w with a stride that puts its last rows past 2^31 elements."""
    N, K, far = 4, 128, (1 << 30) + 64
    s = lin.make(M, N, K, "bf16", False, False, "f32", "f32")
    base = torch.zeros(3 * far + K, dtype=torch.bfloat16, device="cuda")
    w = torch.as_strided(base, (4, K), (far, 1))
    w.copy_(s["w"])
    s["w"] = w
    lin.check(s, lin.call(s, M, N, K), M, N)


def test_logits_past_2_31_elements():
    n, v = 17_000, 131_071
    x = torch.full((n, v), -1.0, dtype=torch.bfloat16, device="cuda")
    x[-2:] = logp.make(2, v)
    ids = torch.randint(0, v, (n, 1), dtype=torch.int32, device="cuda")
    got = logp.call(x, ids, 1.0, 3)
    logp.check(x[-2:], {k: t[-2:] for k, t in got.items()}, ids[-2:], 1.0, 3)
    # equal logits everywhere: the first three, and a token's rank is its index
    assert (got["top_ids"][:-2] == np.arange(3)).all()
    assert np.array_equal(got["rank"][:-2], ids[:-2].cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(1, 50_001), (40, 131_072), (600, 40_000)])
def test_logits_in_order(n, v, dtype):
    """Logits that rise or fall with their index, in steps that bf16 holds and in runs of equal ones: every batch brings
    more candidates than the one before."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    i = torch.arange(v, device="cuda")
    rows = torch.stack([i.float() / 64, -i.float() / 64, (i // 3000).float(), (i % 97).float(), (i >= v - 9).float(), (i < 9).float()])
    x = rows.repeat(-(-n // 6), 1)[:n].to(t)
    ids = logp.some_ids(n, v, 2)
    for k in (1, 20, 64):
        few = slice(0, 6)
        got = logp.call(x, ids, 1.0, k)
        logp.check(x[few], {a: b[few] for a, b in got.items()}, ids[few], 1.0, k)
        for r in range(6, n):  # the others repeat them
            assert np.array_equal(got["top_ids"][r], got["top_ids"][r % 6])


@pytest.mark.parametrize("n", [1, 3, 20, 100, 700, 1500])
def test_every_division_into_slices(n):
    v = 20_011
    x, ids = logp.make(n, v, seed=n), logp.some_ids(n, v, 1)
    got = logp.call(x, ids, 1.0, 7)
    few = np.unique(np.linspace(0, n - 1, 5).astype(int))
    at = torch.from_numpy(few).cuda()
    logp.check(x[at], {k: t[few] for k, t in got.items()}, ids[at], 1.0, 7)


def test_rows_that_repeat():
    s = lin.make(40, 30, 256, "bf16", False, True, "", "f32")
    s["x"] = s["x"][:1].expand(40, 256)
    out = lin.call(s, 40, 30, 256)
    lin.check(s, out, 40, 30)
    assert (out == out[:1]).all()
    x = logp.make(1, 3000).expand(5, 3000)
    got = logp.call(x, top_k=4)
    assert all((t == t[:1]).all() for t in got.values())


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    prods = [lin.make(16, 512, 4096, "bf16", False, False, "", "bf16", whole=False, seed=i) for i in range(2)]
    logits = [logp.make(2, 131072, seed=i) for i in range(2)]
    want_p = [lin.call(s, 16, 512, 4096).clone() for s in prods]
    want_l = [logp.call(x, top_k=5) for x in logits]
    ws = [torch.empty(1 << 22, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert gdn.gdn_linear_act_workspace_bytes(16, 512, 4096, torch.bfloat16) > 0
    outs = [{"lse": torch.empty(2, device="cuda"), "top_ids": torch.empty((2, 5), dtype=torch.int32, device="cuda"),
             "top_logprob": torch.empty((2, 5), device="cuda")} for _ in range(2)]
    for s in prods:
        s["out"].fill_(77)
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            s = prods[i]
            gdn.gdn_linear_act(s["x"], s["w"], s["out"][:16, :512], 16, 512, 4096, workspace=ws[i], stream=st)
            gdn.gdn_logprob(logits[i], 2, 131072, workspace=ws[i], stream=st, **outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(prods[i]["out"][:16, :512], want_p[i])
        assert all(np.array_equal(outs[i][k].cpu().numpy(), want_l[i][k]) for k in outs[i])


def test_tensors_elsewhere_are_refused():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    out = torch.zeros((2, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gdn.GdnError, match="device"):
        gdn.gdn_linear_act(x, w, out, 2, 8, 64)
    with pytest.raises(gdn.GdnError, match="device"):
        gdn.gdn_norm(x[:, None], None, x[:, None], 2)
    with pytest.raises(gdn.GdnError, match="device"):
        gdn.gdn_logprob(x, 2, 64, lse=torch.zeros(2, device="cuda"))
    with pytest.raises(gdn.GdnError, match="shape"):
        gdn.gdn_logprob(x.cuda(), 2, 64, lse=torch.zeros(1, device="cuda"))
    with pytest.raises(gdn.GdnError, match="columns"):
        gdn.gdn_linear_act(w[:2].t().contiguous().t(), w, out, 2, 8, 64)


def test_e4m3_into_bf16_and_into_fp32():
    """Random codes: the 8-bit products' 16 bits stay far below bf16's rounding, and an fp32 out does not have them."""
    for M, K in ((5, 4096), (100, 2048), (700, 1024)):
        s = lin.make(M, 96, K, "e4m3", False, False, "", "f32", whole=False, seed=M)
        want, sums, near = lin.want(s, "none", False)
        full = lin.host(lin.call(s, M, 96, K))
        assert (np.abs(full - want) <= sums + near + ref.U32 * np.abs(want)).all()
        assert np.linalg.norm(full - want) <= 2.0 ** -21 * np.linalg.norm(want)  # K = 4096 sums of random sign: a few 2^-24
        s["out"] = s["out"].to(torch.bfloat16)
        got = lin.host(lin.call(s, M, 96, K))
        exact_rounding = np.linalg.norm(lin.host(torch.from_numpy(want).to(torch.bfloat16)) - want)
        assert np.linalg.norm(got - want) <= 1.01 * exact_rounding  # 1.4e-5 beside 1.7e-3, added in squares
