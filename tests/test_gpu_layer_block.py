"""GPU: a layer's FFN and the step's answer as a program runs them (norm with the residual, gated product, down product
onto the residual stream; final norm, logits, log probabilities), and the attention layer with norms of its heads.

Each stage is held to its own bar on the values that the stage before it stored."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import device, gdn
from gated_deltanet_linear_verify_amd import workloads as W
from tests import layer_ref as ref
from tests import test_gpu_logprob, test_gpu_norm

pytestmark = pytest.mark.gpu


def host(t):
    return None if t is None else t.double().cpu().numpy()


def beyond(got, want, sums, near, half):
    err = np.abs(host(got) - want)
    return (err > sums + near + half * (np.abs(want) + sums + near)).any()


# with an out in bf16 the 8-bit products of a sum are kept to about 16 bits of the largest beside them
E4M3_SUMS = 2.0 ** -15


def slack(fmt, x, w, xs, ws, sums):
    if fmt != "e4m3":
        return sums
    return sums + E4M3_SUMS * (np.abs(host(x)) @ np.abs(host(w)).T) * np.abs(host(xs))[:, None] * np.abs(host(ws))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M,hidden,width", [(1, 256, 512), (16, 512, 1040), (70, 256, 384), (200, 384, 640)])
def test_ffn_step(fmt, M, hidden, width):
    inp = W.make_ffn_inputs(M, hidden, width, seed=M)
    d = device.upload_ffn(inp, fmt=fmt)
    device.ffn_step(d)
    torch.cuda.synchronize()
    # the stream after the norm's addition, before the down product's
    total, y = ref.norm(inp["x"], inp["norm_w"], inp["stream"])
    shaped = {"total": None, "out": d["h"], "scale": d["h_scale"]}
    test_gpu_norm.check(shaped, fmt, total, y)
    want, sums, near = ref.linear(host(d["h"]), host(d["w_gate_up"]), host(d["h_scale"]), host(d["gate_up_scale"]), None, "silu", True)
    if fmt == "e4m3":  # of gate and up, through a slope of at most 1.2 and the other factor
        p = (host(d["h"]) @ host(d["w_gate_up"]).T) * host(d["h_scale"])[:, None] * host(d["gate_up_scale"])
        size = (np.abs(host(d["h"])) @ np.abs(host(d["w_gate_up"])).T) * host(d["h_scale"])[:, None] * host(d["gate_up_scale"])
        gate, up = p[:, :width], p[:, width:]
        sums = sums + E4M3_SUMS * (1.2 * size[:, :width] * np.abs(up) + size[:, width:] * np.abs(ref.activate("silu", gate)))
    assert not beyond(d["act"], want, sums, near, ref.HALF["bf16"])
    act = d["act"] if fmt == "bf16" else d["act8"]
    if fmt != "bf16":
        test_gpu_norm.check({"total": None, "out": d["act8"], "scale": d["act_scale"]}, fmt, None, host(d["act"]))
    want, sums, near = ref.linear(host(act), host(d["w_down"]), host(d["act_scale"]), host(d["down_scale"]), None, "none", False, total)
    # the stream is fp32, so e4m3's products are widened; the sum that was added to was rounded to fp32
    assert not beyond(d["stream"], want, sums + 2 * ref.U32 * np.abs(total), near, ref.HALF["f32"])


@pytest.mark.parametrize("fmt,dtype", [("bf16", torch.bfloat16), ("e4m3", torch.bfloat16), ("i8", torch.float32), ("e4m3", torch.float32)])
@pytest.mark.parametrize("M,hidden,vocab", [(1, 256, 5003), (24, 512, 2000), (80, 128, 9001)])
def test_head_step(fmt, dtype, M, hidden, vocab):
    inp = W.make_head_inputs(M, hidden, vocab, seed=M)
    d = device.upload_head(inp, fmt=fmt, n_ids=2, top_k=5, logits_dtype=dtype)
    d["ids"][:, 0] = torch.randint(0, vocab, (M,), device="cuda", dtype=torch.int32)
    got = {k: t.cpu().numpy() for k, t in device.head_step(d, temperature=0.8).items()}
    _, y = ref.norm(inp["stream"], inp["norm_w"])
    test_gpu_norm.check({"total": None, "out": d["h"], "scale": d["h_scale"]}, fmt, None, y)
    want, sums, near = ref.linear(host(d["h"]), host(d["w"]), host(d["h_scale"]), host(d["w_scale"]))
    if dtype == torch.bfloat16:
        sums = slack(fmt, d["h"], d["w"], d["h_scale"], d["w_scale"], sums)
    assert not beyond(d["logits"], want, sums, near, ref.HALF["bf16" if dtype == torch.bfloat16 else "f32"])
    test_gpu_logprob.check(d["logits"], got, d["ids"], 0.8, 5)


def test_a_step_in_a_graph():
    """FFN and head behind each other, captured once and replayed on changed inputs."""
    a = device.upload_ffn(W.make_ffn_inputs(16, 256, 512, 1), fmt="e4m3")
    b = device.upload_head(W.make_head_inputs(16, 256, 3001, 1), fmt="e4m3", top_k=4)
    b["stream"] = a["stream"]
    first = a["stream"].clone()

    def step():
        device.ffn_step(a)
        device.head_step(b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        a["stream"].copy_(first * (1 + i)), a["x"].copy_(torch.randn(16, 256, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = {k: t.clone() for k, t in b["answer"].items()}
        stream = a["stream"].clone()
        a["stream"].copy_(first * (1 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["stream"], stream) and all(torch.equal(b["answer"][k], t) for k, t in want.items())


def test_attention_step_with_norms_of_q_and_k():
    B, T, hidden, n_q, n_kv, hd = 2, 5, 256, 8, 2, 128
    inp = W.make_attention_inputs(B, T, hidden, n_q, n_kv, hd, 3)
    rng = np.random.default_rng(5)
    qw, kw = (1 + rng.normal(0, 0.2, hd) for _ in range(2))
    rope = gdn.gdn_rope_init(64, theta=1e6)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    table, start = i32([[1, 2], [3, 0]]), i32([0, 0])
    pos = i32([list(range(T)) * B])
    runs = []
    for norms in (False, True):
        d = device.upload_attention(inp, rope, fmt=gdn.GDN_KV_BF16, page_size=16, n_pages=4,
                                    q_norm=qw if norms else None, k_norm=kw if norms else None)
        device.attention_step(d, table, start, pos)
        torch.cuda.synchronize()
        runs.append(d)
    plain, normed = runs
    # by hand: the projection's rows, normed and rounded, then the calls behind them
    gdn.gdn_linear(plain["x"], plain["w_in"], B * T, plain["w_in"].shape[0], hidden, [(0, plain["w_in"].shape[0], plain["qkv"], plain["w_in"].shape[0], 0)])
    torch.cuda.synchronize()
    for n, w, heads in (("q", qw, n_q), ("k", kw, n_kv)):
        s = {"x": plain[n], "weight": torch.tensor(w, dtype=torch.float32, device="cuda"), "residual": None, "total": None,
             "out": torch.empty((B * T, heads, hd), dtype=torch.bfloat16, device="cuda"), "scale": None}
        test_gpu_norm.call(s, B * T)
        test_gpu_norm.check(s, "bf16", *ref.norm(host(s["x"]), host(s["weight"])))
        plain[n].copy_(s["out"])
    kv = plain["kv"]
    gdn.gdn_rope(rope, [(plain["q"], plain["q"])], pos, B * T)
    gdn.gdn_kv_write(kv, plain["k"], plain["v"], table, start, None, B, T, rope=rope, positions=pos)
    gdn.gdn_attn_verify(kv, plain["q"], table, start, None, None, None, None, plain["out"], B, T, plain["scale"], plain["workspace"])
    gdn.gdn_linear(plain["out"], plain["w_out"], B * T, hidden, n_q * hd, [(0, hidden, plain["y"], hidden, 0)])
    torch.cuda.synchronize()
    assert torch.equal(plain["y"], normed["y"]) and torch.isfinite(normed["y"].float()).all()
