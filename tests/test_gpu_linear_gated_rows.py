"""A gated gdn_linear_act takes w, its scales and bias of exactly 2 N rows: of more, the up rows would not be the last N."""

import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import test_gpu_linear_act as lin

pytestmark = pytest.mark.gpu


def test_more_rows_are_refused_where_gated_and_left_alone_where_not():
    N, K = 20, 64
    s = lin.make(4, N, K, "e4m3", True, True, "", "f32")
    more = lin.make(4, N + 4, K, "e4m3", True, True, "", "f32")
    for name in ("w", "w_scale", "bias"):
        with pytest.raises(gdn.GdnError, match=f"{name} has 48 rows, a gated product of 20 columns takes 40"):
            lin.call(dict(s, **{name: more[name]}), 4, N, K, "silu", True)
    lin.check(s, lin.call(s, 4, N, K, "silu", True), 4, N, "silu", True)
    out = lin.call(dict(more, out=s["out"]), 4, N, K)  # the first 20 of 48
    cut = {k: more[k][:N] for k in ("w", "w_scale", "bias")}
    lin.check(dict(more, out=s["out"], **cut), out, 4, N)
