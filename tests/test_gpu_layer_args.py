"""What the layer's steps pass on to gdn_norm: the model's eps."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import device, gdn
from gated_deltanet_linear_verify_amd import workloads as W
from tests import layer_ref as ref
from tests import test_gpu_norm

pytestmark = pytest.mark.gpu


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("eps", [1e-5, 1e-2])
def test_the_steps_take_the_models_eps(eps):
    inp = W.make_ffn_inputs(5, 256, 512, seed=1)
    inp["stream"] *= 1e-3
    inp["x"] *= 2.0 ** -9
    d = device.upload_ffn(inp, eps=eps)
    device.ffn_step(d)
    torch.cuda.synchronize()
    _, y = ref.norm(inp["x"], inp["norm_w"], inp["stream"], eps=eps)
    test_gpu_norm.check({"total": None, "out": d["h"], "scale": None}, "bf16", None, y)
    inp = W.make_head_inputs(5, 256, 1000, seed=1)
    inp["stream"] *= 1e-3
    d = device.upload_head(inp, eps=eps)
    device.head_step(d)
    torch.cuda.synchronize()
    _, y = ref.norm(inp["stream"], inp["norm_w"], eps=eps)
    test_gpu_norm.check({"total": None, "out": d["h"], "scale": None}, "bf16", None, y)


def test_the_attention_step_takes_the_models_eps():
    B, T, hidden, n_q, n_kv, hd = 1, 3, 256, 2, 1, 128
    inp = W.make_attention_inputs(B, T, hidden, n_q, n_kv, hd, 3)
    rope = gdn.gdn_rope_init(64, theta=1e6)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for eps in (None, 1e-6, 10.0):
        kw = {} if eps is None else {"eps": eps}
        d = device.upload_attention(inp, rope, fmt=gdn.GDN_KV_BF16, page_size=16, n_pages=2, q_norm=np.ones(hd), k_norm=np.ones(hd), **kw)
        gdn.gdn_linear(d["x"], d["w_in"], B * T, d["w_in"].shape[0], hidden, [(0, d["w_in"].shape[0], d["qkv"], d["w_in"].shape[0], 0)])
        _, q = ref.norm(host(d["q"]), None, eps=1e-6 if eps is None else eps)
        device.attention_step(d, i32([[1]]), i32([0]), i32([list(range(T))]))
        torch.cuda.synchronize()
        # the rotation keeps the length of each pair of channels, up to the roundings of the norm and of its own
        pair = lambda a: np.hypot(a[..., :32], a[..., 32:64])  # noqa: E731
        assert (np.abs(pair(host(d["q"])) - pair(q)) <= 2.0 ** -6 * pair(q) + 1e-30).all()
        assert (np.abs(host(d["q"])[..., 64:] - q[..., 64:]) <= 2.0 ** -7 * np.abs(q[..., 64:])).all()
        got.append(d["y"].clone())
    assert torch.equal(got[0], got[1]) and not torch.equal(got[0], got[2])
