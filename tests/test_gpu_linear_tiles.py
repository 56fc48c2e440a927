"""gdn_linear_act in each of its tile shapes: sizes one past and one short of a tile, K that ends inside a step of 128 bytes,
columns that are and are not a multiple of 4, more than eight rows of tiles, and K in parts.  tests/test_linear_tiles.py holds that
these sizes reach every shape.

Rows of x repeat with a period that no tile has, so the rows of the result have to repeat bit for bit; those of one period are
compared with the formula in 64 bits, in all their columns."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests import test_gpu_linear_act as lin
from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu
PERIOD = 61
# (M, N, K, type, gated)
SIZES = [
    # 16 x 64, few and many workgroups, one part and several
    (16, 1001, 208, "bf16", False), (15, 300, 4112, "e4m3", True), (3, 77, 6992, "i8", False), (1, 131, 4112, "bf16", True),
    (16, 33_001, 144, "bf16", False), (15, 16_602, 208, "e4m3", True), (2, 33_004, 336, "i8", False),
    # 32 x 64
    (17, 333, 208, "bf16", True), (32, 500, 336, "e4m3", False), (31, 129, 4112, "i8", True), (31, 10_500, 144, "e4m3", True),
    # 64 x 64, up to 64 rows and more
    (33, 501, 208, "bf16", False), (64, 300, 4112, "i8", True), (63, 200, 336, "e4m3", True), (65, 68, 144, "bf16", True),
    (513, 63, 4112, "bf16", False), (65, 63, 5136, "e4m3", True), (513, 68, 336, "i8", False),
    # 64 x 128
    (65, 5119, 144, "bf16", True), (513, 2241, 336, "e4m3", False), (65, 1732, 4112, "bf16", False), (513, 1156, 336, "i8", True),
    (191, 3001, 208, "bf16", False),
    # 128 x 128, three buffers
    (129, 15_655, 144, "bf16", False), (2049, 641, 336, "e4m3", True), (2049, 1284, 336, "i8", False), (257, 580, 6992, "bf16", True),
    (1025, 257, 6992, "bf16", False), (257, 3457, 6992, "i8", False), (385, 1284, 6992, "e4m3", True),
    # 128 x 128, two buffers
    (2305, 833, 144, "bf16", True), (129, 21_804, 336, "e4m3", False), (2305, 1665, 336, "i8", False), (129, 11_047, 336, "e4m3", True),
    (2049, 257, 6992, "bf16", False), (129, 2180, 6992, "bf16", True),
    # 256 x 256
    (257, 32_039, 144, "bf16", False), (2049, 2756, 144, "bf16", True), (2049, 2753, 336, "e4m3", True), (257, 32_044, 336, "i8", False),
    (2305, 5505, 336, "e4m3", False), (769, 5121, 5136, "bf16", False), (769, 2564, 5136, "bf16", True), (1023, 5121, 13_840, "i8", False),
    (1025, 2564, 13_840, "e4m3", True),
]
# with an out in bf16, of eight neighbouring products all but the largest are cut at 2^-13 of it
E4M3_SUMS = 7 * 2.0 ** -13


def repeat(s, M):
    """The tensors of s with M rows, of which PERIOD are different."""
    at = torch.arange(M, device="cuda") % PERIOD
    for k in ("x", "x_scale", "residual"):
        if s[k] is not None:
            t = s[k]
            s[k] = t.view(torch.uint8)[at].view(t.dtype) if t.element_size() == 1 else t[at]
    return at


@pytest.mark.parametrize("M,N,K,dtype,gated", SIZES)
@pytest.mark.parametrize("whole", [True, False])
def test_every_tile(M, N, K, dtype, gated, whole):
    first = min(M, PERIOD)
    # small whole numbers, exact in any order of the sums, onto an fp32 result; random values into bf16 (e4m3: the 8-bit
    # matrix instructions)
    act, residual, out = ("gelu_tanh", "f32", "f32") if whole else ("silu", "bf16", "bf16")
    s = lin.make(first, N, K, dtype, gated, True, residual, out, whole=whole, seed=M + N)
    y, sums, near = lin.want(s, act, gated)
    if whole or dtype == "i8":
        sums = 0
    elif dtype == "e4m3":
        p = (lin.host(s["x"]) @ lin.host(s["w"]).T) * lin.host(s["x_scale"])[:, None] * lin.host(s["w_scale"]) + lin.host(s["bias"])
        size = (np.abs(lin.host(s["x"])) @ np.abs(lin.host(s["w"])).T) * lin.host(s["x_scale"])[:, None] * lin.host(s["w_scale"])
        if gated:
            sums = sums + E4M3_SUMS * (1.2 * size[:, :N] * np.abs(p[:, N:]) + size[:, N:] * np.abs(ref.activate(act, p[:, :N])))
        else:
            sums = sums + E4M3_SUMS * 1.2 * size
    at = repeat(s, M)
    s["out"] = torch.full((M + 2, N + 3), 77.0, dtype=s["out"].dtype, device="cuda")
    if N % 4 == 0:  # rows whose quads of columns are aligned, and, at other sizes, rows that are not
        s["out"] = torch.full((M + 2, N + 4), 77.0, dtype=s["out"].dtype, device="cuda")
    got = lin.call(s, M, N, K, act, gated)
    err = np.abs(lin.host(got[:first]) - y)
    bound = sums + near
    bad = err > bound + ref.HALF[out] * (np.abs(y) + bound) + 2.0 ** -126
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5])
    assert torch.equal(got, got[at])  # every other row is its first one again, bit for bit
    rest = s["out"].clone()
    rest[:M, :N] = 77.0
    assert (rest == 77.0).all()


@pytest.mark.parametrize("M,N,K,dtype,gated", [s for s in SIZES if s[0] > 64 and s[0] * s[1] < 3_000_000][::4])
def test_infinities_and_nan_stay_in_their_rows_and_columns(M, N, K, dtype, gated):
    if dtype == "i8":
        dtype = "bf16"
    s = lin.make(M, N, K, dtype, gated, False, "", "f32")
    rows = (0, M // 2, M - 1)
    cols = (1, N // 2 + 1, N - 1)
    for i, r in enumerate(rows):
        s["x"][r, (0, K // 2, K - 1)[i]] = float("nan")
    for i, c in enumerate(cols):
        s["w"][c, (K - 1, 3, K // 2)[i]] = float("nan")
    got = lin.host(lin.call(s, M, N, K, "relu", gated))
    bad = np.zeros((M, N), bool)
    bad[list(rows)], bad[:, list(cols)] = True, True
    assert (np.isnan(got) == bad).all()
