"""gdn_norm against its formula in 64 bits."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
U = ref.U32
# r = 1 / sqrt(mean + eps): the sum of squares is off by half a step for each addition on a value's way (up to 16 in its
# lane, 10 between the lanes), its root by half of that, and four operations round; the products by w and r two more
Y = 24 * U


def host(t):
    return t.double().cpu().numpy()


def make(n, heads, d, x="bf16", residual="", out="bf16", extra=0, seed=0, weight=True, offset=0):
    """Device tensors; extra: heads beside these in the same rows, offset: elements before the first row."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(n * (heads + extra) * d + offset, generator=g).to(TYPES[x]).cuda()
    s = {"x": wide[offset:].view(n, heads + extra, d)[:, extra:]}
    s["weight"] = (1 + 0.2 * torch.randn(d, generator=g)).cuda() if weight else None
    s["residual"] = (2 * torch.randn(n, heads, d, generator=g)).to(TYPES[residual]).cuda() if residual else None
    s["total"] = torch.full_like(s["residual"], 7) if residual else None
    s["out"] = torch.zeros((n, heads, d), dtype=torch.uint8 if out in ref.FULL else TYPES[out], device="cuda")
    if out in ref.FULL:
        s["out"] = s["out"].view(TYPES[out])
    s["scale"] = torch.full((n, heads), -1.0, device="cuda") if out in ref.FULL else None
    return s


def call(s, n, **kw):
    gdn.gdn_norm(s["x"], s["weight"], s["out"], n, residual=s["residual"], total=s["total"], scale=s["scale"], **kw)
    torch.cuda.synchronize()


def check(s, out, want_s, y):
    """out's values, codes and scale against the exact s and y."""
    if s["total"] is not None:
        half = ref.HALF["bf16" if s["total"].dtype == torch.bfloat16 else "f32"]
        err = np.abs(host(s["total"]) - want_s)
        assert (err <= (half + 2 * U) * np.abs(want_s)).all(), err.max()
    if out not in ref.FULL:
        assert (np.abs(host(s["out"]) - y) <= (ref.HALF[out] + Y) * np.abs(y) * (1 + 2 * Y) + 1e-40).all()
        return
    scale = host(s["scale"])
    most = np.abs(y).max(-1)
    assert (np.abs(scale - most / ref.FULL[out]) <= (Y + 2 * U) * most / ref.FULL[out]).all()
    unit = (most / ref.FULL[out])[..., None]
    codes, c = host(s["out"]), np.where(unit > 0, y / np.where(unit > 0, unit, 1), 0)
    # the code's own value is off by the product's errors, and then rounded: whole numbers by half of one, e4m3 by half a
    # step of three bits, at least half of the smallest one's 2^-9
    off = (2 * Y + 4 * U) * np.abs(c)
    rounding = 0.5 if out == "i8" else np.maximum(2.0 ** -4 * (np.abs(c) + off), 2.0 ** -10)
    assert (np.abs(codes - c) <= rounding + off).all(), np.abs(codes - c).max()
    assert np.abs(codes).max() <= ref.FULL[out]


@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("n,heads,d", [(1, 1, 1), (3, 1, 7), (1, 1, 64), (5, 3, 63), (9, 2, 64), (33, 4, 128), (7, 5, 136),
                                       (6, 2, 256), (4, 3, 257), (5, 1, 512), (3, 1, 520), (2, 1, 1000), (3, 1, 1025), (2, 1, 4097),
                                       (5, 1, 5120), (2, 1, 8192), (3, 1, 8200), (1, 1, 9999), (2, 1, 16384), (300, 1, 96)])
def test_sizes(n, heads, d, out):
    for seed, (x, residual) in enumerate([("bf16", ""), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")]):
        s = make(n, heads, d, x, residual, out, seed=seed + d)
        call(s, n)
        check(s, out, *ref.norm(host(s["x"]), host(s["weight"]), None if not residual else host(s["residual"])))


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("extra,offset,d", [(2, 0, 128), (1, 1, 128), (3, 4, 256), (1, 8, 72), (0, 3, 5120), (2, 2, 33)])
def test_rows_inside_others(extra, offset, d, out):
    s = make(11, 3, d, "bf16", "f32", out, extra=extra, offset=offset)
    call(s, 11)
    check(s, out, *ref.norm(host(s["x"]), host(s["weight"]), host(s["residual"])))


@pytest.mark.parametrize("d", [96, 1000, 5120])
def test_the_sum_alone_and_without_weight(d):
    s = make(5, 2, d, "bf16", "bf16", "i8", weight=False)
    call(s, 5, mode=gdn.GDN_NORM_NONE, eps=0.0)
    want_s, y = ref.norm(host(s["x"]), None, host(s["residual"]), rms=False)
    check(s, "i8", want_s, y)
    s = make(5, 2, d, "f32", "", "f32", weight=False)
    call(s, 5, mode=gdn.GDN_NORM_NONE)
    assert torch.equal(s["out"], s["x"])


@pytest.mark.parametrize("d", [128, 5120])
def test_in_place(d):
    a = make(6, 1, d, "bf16", "bf16", "bf16", seed=3)
    b = {k: None if v is None else v.clone() for k, v in a.items()}
    call(a, 6)
    b["total"], b["out"] = b["residual"], b["x"]  # the stream takes the sum, x its norm
    call(b, 6)
    assert torch.equal(a["total"], b["total"]) and torch.equal(a["out"], b["out"])
    c = make(6, 1, d, "bf16", "bf16", "bf16", seed=3)
    c["total"], c["out"] = c["x"], c["residual"]
    call(c, 6)
    assert torch.equal(a["total"], c["total"]) and torch.equal(a["out"], c["out"])


def test_a_residual_that_repeats_and_rows_behind_the_last():
    s = make(9, 2, 640, "bf16", "bf16", "e4m3")
    s["residual"] = s["residual"][:1].expand(9, 2, 640)
    before = {k: s[k].clone() for k in ("total", "out", "scale")}
    call(s, 5)
    want_s, y = ref.norm(host(s["x"])[:5], host(s["weight"]), host(s["residual"])[:5])
    check({k: v if k in ("x", "weight") else v[:5] for k, v in s.items()}, "e4m3", want_s, y)
    for k, t in before.items():
        assert torch.equal(s[k][5:].view(torch.uint8), t[5:].view(torch.uint8)), k
    call(s, 0)


@pytest.mark.parametrize("d", [64, 100, 5120])
def test_rows_of_zeros_and_of_extreme_values(d):
    x = torch.randn(8, 1, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e30           # squares pass fp32's range
    x[3] = 3e38
    x[4] = 0
    x[4, 0, d // 2] = -3e38
    x[5] *= 1e19
    x[6] *= 1e-42          # subnormal
    for out in ("f32", "e4m3", "i8"):
        s = make(8, 1, d, "f32", "", out)
        s["x"] = x.cuda()
        call(s, 8, eps=1e-5)
        want_s, y = ref.norm(x.double().numpy(), host(s["weight"]), eps=1e-5)
        # subnormal inputs may count as zeros, and results below 2^-126 and codes of such rows may be zero
        if out == "f32":
            assert (np.abs(host(s["out"]) - y) <= (U + Y) * np.abs(y) + 2.0 ** -126).all()
            assert not host(s["out"])[0].any()
        else:
            keep = [2, 3, 4, 5, 7]
            check({k: v[keep] if k in ("out", "scale") else None for k, v in s.items()}, out, want_s[keep], y[keep])
            assert not host(s["out"])[0].any() and host(s["scale"])[0] == 0


@pytest.mark.parametrize("d", [64, 100, 5120])
def test_infinities_and_nan_stay_in_their_row(d):
    for bad in (float("inf"), float("-inf"), float("nan")):
        for out in ("bf16", "e4m3", "i8"):
            s = make(3, 2, d, "bf16", "bf16", out)
            s["x"][1, 0, d - 1] = bad
            call(s, 3)
            want_s, y = ref.norm(host(s["x"]), host(s["weight"]), host(s["residual"]))
            if out == "bf16":
                got = host(s["out"])
                assert np.isnan(got[1, 0, d - 1]) and (np.isnan(got[1, 0]) | (got[1, 0] == 0)).all()
            else:
                assert np.isnan(host(s["scale"])[1, 0]) and not host(s["out"])[1, 0].any()
            ok = np.ones((3, 2), bool)
            ok[1, 0] = False
            check({"total": None, "out": s["out"][torch.from_numpy(ok).cuda()],
                   "scale": None if s["scale"] is None else s["scale"][torch.from_numpy(ok).cuda()]}, out, want_s[ok], y[ok])


def test_values_of_one_size_round_to_even():
    """Rows whose scale is a power of two: codes at exact halves."""
    x = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5]).view(1, 1, 8)
    s = make(1, 1, 8, "f32", "", "i8", weight=False)
    s["x"] = x.cuda()
    call(s, 1, mode=gdn.GDN_NORM_NONE)
    assert s["out"].flatten().tolist() == [127, 0, 2, 2, 0, -2, -2, 64] and s["scale"].item() == 1.0


def test_another_stream_and_a_graph():
    s = make(40, 1, 5120, "bf16", "bf16", "e4m3")
    call(s, 40)
    want = {k: s[k].clone() for k in ("total", "out", "scale")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_norm(s["x"], s["weight"], s["out"], 40, residual=s["residual"], total=s["total"], scale=s["scale"])
    for _ in range(3):
        s["total"].zero_(), s["scale"].zero_(), s["out"].view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[k].view(torch.uint8), t.view(torch.uint8)) for k, t in want.items())
