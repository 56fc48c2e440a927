"""gdn_linear_act against its formula in 64 bits."""

import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from gated_deltanet_linear_verify_amd import gdn

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
ACTS = {"none": gdn.GDN_ACT_NONE, "silu": gdn.GDN_ACT_SILU, "gelu": gdn.GDN_ACT_GELU, "gelu_tanh": gdn.GDN_ACT_GELU_TANH,
        "relu": gdn.GDN_ACT_RELU, "sigmoid": gdn.GDN_ACT_SIGMOID}


def host(t):
    return None if t is None else t.double().cpu().numpy()


def make(M, N, K, dtype="bf16", gated=False, bias=False, residual="", out="bf16", whole=True, seed=0, pad=0):
    """whole: operands are small whole numbers, so that every sum over K is exact in fp32.  pad: columns past K in x's and
    w's rows, which hold NaN (or 127)."""
    g = torch.Generator().manual_seed(seed)
    rows = 2 * N if gated else N

    def operand(n):
        t = torch.randint(-4, 5, (n, K), generator=g).float() if whole else torch.randn(n, K, generator=g) * (30 if dtype == "i8" else 1)
        if dtype == "i8" and not whole:
            t = t.round().clamp(-128, 127)
        full = torch.full((n, K + pad), 127.0 if dtype == "i8" else float("nan"))
        full[:, :K] = t
        return full.to(TYPES[dtype]).cuda()[:, :K]

    s = {"x": operand(M), "w": operand(rows), "x_scale": None, "w_scale": None}
    unit = (6.7 * K) ** -0.5 if whole else K ** -0.5 / (30 if dtype == "i8" else 1)
    if dtype != "bf16":
        s["x_scale"] = (torch.rand(M, generator=g) + 0.5).cuda()
        s["w_scale"] = ((torch.rand(rows, generator=g) + 0.5) * unit).cuda()
    s["bias"] = torch.randn(rows, generator=g).cuda() if bias else None
    s["residual"] = torch.randn(M, N, generator=g).to(TYPES[residual]).cuda() if residual else None
    s["out"] = torch.full((M + 2, N + 3), 77.0, dtype=TYPES[out], device="cuda")
    return s


def call(s, M, N, K, act="none", gated=False, **kw):
    need = gdn.gdn_linear_act_workspace_bytes(M, N, K, s["x"].dtype, gated)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda") if need else None
    out = s["out"][:M, :N]
    gdn.gdn_linear_act(s["x"], s["w"], out, M, N, K, x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"],
                       act=ACTS[act], gated=gated, residual=s["residual"], workspace=ws, **kw)
    torch.cuda.synchronize()
    if need:
        assert (ws[need:] == 255).all()  # nothing behind what was asked for
    return out


def want(s, act, gated):
    return ref.linear(host(s["x"]), host(s["w"]), host(s["x_scale"]), host(s["w_scale"]), host(s["bias"]), act, gated,
                      host(s["residual"]))


def check(s, out, M, N, act="none", gated=False, exact_sums=True):
    y, sums, near = want(s, act, gated)
    bound = near + (0 if exact_sums else sums)
    half = ref.HALF["bf16" if out.dtype == torch.bfloat16 else "f32"]
    err = np.abs(host(out) - y)
    bad = err > bound + half * (np.abs(y) + bound) + 2.0 ** -126
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5])
    rest = s["out"].clone()
    rest[:M, :N] = 77.0
    assert (rest == 77.0).all()  # nothing beside the result


SIZES = [(1, 1, 16), (1, 5, 32), (1, 512, 4096), (2, 33, 80), (7, 257, 144), (13, 100, 1040), (16, 64, 640), (17, 95, 272),
         (31, 130, 512), (32, 32, 128), (33, 48, 208), (48, 300, 1024), (64, 1000, 2048), (65, 129, 336), (100, 513, 256),
         (128, 128, 64), (129, 257, 4112), (200, 40, 5120), (256, 640, 768), (300, 300, 304), (513, 1031, 160), (1024, 96, 512)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dtype):
    for seed, (gated, act, bias, residual, out) in enumerate([(False, "none", False, "", "f32"), (True, "silu", True, "bf16", "bf16"),
                                                              (False, "gelu_tanh", True, "f32", "f32")]):
        s = make(M, N, K, dtype, gated, bias, residual, out, seed=seed + M)
        check(s, call(s, M, N, K, act, gated), M, N, act, gated)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M,N,K", [(1, 2048, 4096), (16, 1024, 5120), (40, 256, 8192), (160, 384, 2048), (640, 768, 1024)])
def test_random_values(M, N, K, dtype):
    for gated in (False, True):
        s = make(M, N, K, dtype, gated, True, "bf16", "f32", whole=False, seed=K)
        check(s, call(s, M, N, K, "silu", gated), M, N, "silu", gated, exact_sums=dtype == "i8")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
def test_activations(act, gated):
    for M in (3, 150):
        s = make(M, 70, 64, "bf16", gated, True, "", "f32")
        s["bias"] = s["bias"] * 8
        s["bias"][:6] = torch.tensor([0.0, 90.0, -90.0, 200.0, -200.0, 1e-6])
        check(s, call(s, M, 70, 64, act, gated), M, 70, act, gated)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M", [1, 20, 130])
def test_rows_inside_wider_ones(dtype, M):
    """Strides past K: what lies there (NaN) is not read into the result."""
    s = make(M, 77, 208, dtype, False, False, "f32", "bf16", pad=48)
    check(s, call(s, M, 77, 208), M, 77)
    s["residual"] = s["residual"][:1].expand(M, 77)
    check(s, call(s, M, 77, 208), M, 77)


@pytest.mark.parametrize("M,K", [(1, 1024), (24, 1024), (140, 256)])
def test_onto_the_residual(M, K):
    s = make(M, 90, K, "bf16", False, False, "f32", "f32")
    s["out"][:M, :90] = s["residual"]
    y = want(s, "none", False)
    s["residual"] = s["out"][:M, :90]
    out = call(s, M, 90, K)
    assert (np.abs(host(out) - y[0]) <= y[2] + ref.U32 * np.abs(y[0])).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [2, 40, 200])
def test_infinities_and_nan_stay_in_their_rows_and_columns(dtype, M):
    s = make(M, 100, 256, dtype, True, False, "", "f32")
    s["x"][1, 77] = float("nan")
    s["w"][42, 3] = float("nan")
    s["w"][100 + 17, 255] = float("nan")
    out = host(call(s, M, 100, 256, "silu", True))
    bad = np.zeros((M, 100), bool)
    bad[1], bad[:, 42], bad[:, 17] = True, True, True
    assert (np.isnan(out) == bad).all()
    y, _, near = want(s, "silu", True)
    assert (np.abs(out - y)[~bad] <= (near + ref.U32 * np.abs(y) + 1e-38)[~bad]).all()
    s = make(M, 100, 256, "i8", False, False, "", "f32")
    s["x_scale"][0] = float("nan")  # a row that gdn_norm found not finite
    out = host(call(s, M, 100, 256))
    assert np.isnan(out[0]).all() and np.isfinite(out[1:]).all()


def test_extreme_codes():
    """i8: every product 128^2, at the deepest K that int32 holds."""
    K = (1 << 17) - 16
    s = make(2, 3, K, "i8", out="f32")
    s["x"].fill_(-128), s["w"].fill_(-128)
    check(s, call(s, 2, 3, K), 2, 3)


def test_more_rows_are_left_alone_and_none_is_a_no_op():
    s = make(9, 20, 64, "bf16")
    gdn.gdn_linear_act(s["x"], s["w"], s["out"][:9, :20], 0, 20, 64)
    torch.cuda.synchronize()
    assert (s["out"] == 77).all()
    out = call(s, 4, 20, 64)
    y = want(s, "none", False)
    assert (np.abs(host(out) - y[0][:4]) <= 2.0 ** -8 * np.abs(y[0][:4])).all() and (s["out"][4:] == 77).all()


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (16, 640, 2048), (200, 256, 4096), (700, 512, 512)])
def test_another_stream_a_graph_and_the_same_bits(M, N, K):
    s = make(M, N, K, "bf16", True, False, "bf16", "bf16", whole=False)
    first = call(s, M, N, K, "silu", True).clone()
    need = gdn.gdn_linear_act_workspace_bytes(M, N, K, torch.bfloat16, True)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gdn.gdn_linear_act(s["x"], s["w"], s["out"][:M, :N], M, N, K, act=gdn.GDN_ACT_SILU, gated=True,
                           residual=s["residual"], workspace=ws)
    for _ in range(3):
        s["out"].fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["out"][:M, :N], first)
        s["out"].fill_(77)
        assert torch.equal(call(s, M, N, K, "silu", True), first)
