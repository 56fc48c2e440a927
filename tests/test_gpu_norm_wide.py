"""gdn_norm without its division over rows past 16384 channels: the operands of a down product as wide as its FFN."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import device, gdn
from gated_deltanet_linear_verify_amd import workloads as W
from tests import layer_ref as ref
from tests.test_gpu_norm import call, check, host, make

pytestmark = pytest.mark.gpu


def weight_of(s):
    return None if s["weight"] is None else host(s["weight"])


@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("n,heads,d", [(3, 1, 16385), (2, 1, 16392), (5, 1, 17408), (3, 2, 25600), (2, 1, 27999), (1, 1, 65535), (2, 1, 65536)])
def test_long_rows_without_the_division(n, heads, d, out):
    for seed, (x, residual, weight) in enumerate([("bf16", "", False), ("bf16", "bf16", True), ("f32", "bf16", False), ("bf16", "f32", True)]):
        s = make(n, heads, d, x, residual, out, seed=seed + d, weight=weight)
        call(s, n, mode=gdn.GDN_NORM_NONE)
        check(s, out, *ref.norm(host(s["x"]), weight_of(s), None if not residual else host(s["residual"]), rms=False))


@pytest.mark.parametrize("d", [17408, 16401])
def test_long_rows_in_place_inside_others_and_behind_the_last(d):
    a = make(4, 1, d, "bf16", "bf16", "bf16", seed=3)
    b = {k: None if v is None else v.clone() for k, v in a.items()}
    call(a, 4, mode=gdn.GDN_NORM_NONE)
    b["total"], b["out"] = b["residual"], b["x"]
    call(b, 4, mode=gdn.GDN_NORM_NONE)
    assert torch.equal(a["total"], b["total"]) and torch.equal(a["out"], b["out"])
    s = make(5, 2, d, "bf16", "f32", "i8", extra=1, offset=3)
    before = {k: s[k].clone() for k in ("total", "out", "scale")}
    call(s, 3, mode=gdn.GDN_NORM_NONE)
    want_s, y = ref.norm(host(s["x"])[:3], weight_of(s), host(s["residual"])[:3], rms=False)
    check({k: v if k in ("x", "weight") else v[:3] for k, v in s.items()}, "i8", want_s, y)
    for k, t in before.items():
        assert torch.equal(s[k][3:].view(torch.uint8), t[3:].view(torch.uint8)), k


@pytest.mark.parametrize("d", [17408, 16385])
def test_long_rows_of_zeros_infinities_and_extremes(d):
    x = torch.randn(6, 1, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0
    x[1, 0, d - 1] = float("nan")
    x[2, 0, 7] = float("-inf")
    x[3] = 3e38
    x[4] *= 1e-44
    for out in ("e4m3", "i8"):
        s = make(6, 1, d, "f32", "", out, weight=False)
        s["x"] = x.cuda()
        call(s, 6, mode=gdn.GDN_NORM_NONE)
        codes, scale = host(s["out"]), host(s["scale"])
        assert not codes[[0, 1, 2, 4]].any() and scale[0, 0] == 0 and scale[4, 0] == 0 and np.isnan(scale[1:3]).all()
        keep = [3, 5]
        check({"total": None, "out": s["out"][keep], "scale": s["scale"][keep]}, out, None, host(s["x"])[keep])


def test_long_rows_with_the_division_are_refused():
    s = make(2, 1, 16392)
    with pytest.raises(gdn.GdnError, match="16384"):
        call(s, 2)
    s = make(1, 1, 65544, "bf16", "", "i8", weight=False)
    with pytest.raises(gdn.GdnError, match="65536"):
        call(s, 1, mode=gdn.GDN_NORM_NONE)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M,width", [(1, 17408), (5, 16400), (2, 25600)])
def test_ffn_step_of_wide_layers(fmt, M, width):
    hidden = 64
    inp = W.make_ffn_inputs(M, hidden, width, seed=M)
    d = device.upload_ffn(inp, fmt=fmt)
    device.ffn_step(d)
    torch.cuda.synchronize()
    total, _ = ref.norm(inp["x"], inp["norm_w"], inp["stream"])
    act = d["act"] if fmt == "bf16" else d["act8"]
    if fmt != "bf16":
        check({"total": None, "out": d["act8"], "scale": d["act_scale"]}, fmt, None, host(d["act"]))
        check({"total": None, "out": d["w_down"], "scale": d["down_scale"]}, fmt, None,
              host(torch.from_numpy(np.asarray(inp["w_down"], np.float32)).bfloat16()))
    scales = (None, None) if fmt == "bf16" else (host(d["act_scale"]), host(d["down_scale"]))
    want, sums, near = ref.linear(host(act), host(d["w_down"]), *scales, None, "none", False, total)
    err = np.abs(host(d["stream"]) - want)
    assert (err <= sums + 2 * ref.U32 * np.abs(total) + near + ref.U32 * np.abs(want)).all(), err.max()
