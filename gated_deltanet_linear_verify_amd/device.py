"""Device buffers for the verify path: torch owns the memory, libgdn computes.

Plumbing only: uploads the seeded inputs of ``workloads`` in the storage dtypes of include/gdn.h
and allocates outputs, capture buffers and workspaces with the documented shapes.
"""

from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import gdn
from .workloads import BF16, Shape


def act_torch_dtype(code: int) -> torch.dtype:
    return torch.bfloat16 if code == BF16 else torch.float32


def upload(shape: Shape, inp: dict, *, device: str = "cuda", t_cap: Optional[int] = None,
           mode: int = gdn.GDN_CHAIN, capture: bool = True, fill_capture: float = float("nan"),
           flags: int = 0, eps: float = 1e-6) -> dict:
    """Device tensors for one call plus the ctypes dims / capture descriptors."""
    act = act_torch_dtype(shape.act_dtype)
    outd = act_torch_dtype(shape.out_dtype)
    B, T, P = shape.n_batch, shape.n_tok, shape.n_pool
    Hv, dv, dk, C = shape.n_vh, shape.d_v, shape.d_k, shape.conv_channels
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)
    d = {
        "qkv": f32(inp["qkv"]).to(act).contiguous(),
        "z": f32(inp["z"]).to(act).contiguous(),
        "alpha": f32(inp["alpha"]).to(act).contiguous(),
        "beta": f32(inp["beta"]).to(act).contiguous(),
        "A_log": f32(inp["A_log"]),
        "dt_bias": f32(inp["dt_bias"]),
        "conv_w": f32(inp["conv_w"]),
        "norm_w": f32(inp["norm_w"]),
        "state": f32(inp["state"]),
        "conv_state": f32(inp["conv_state"]),
        "slot_ids": torch.from_numpy(np.ascontiguousarray(inp["slot_ids"], dtype=np.int32)).to(device),
        # the prefill's slot, kept on the host so that a call does not read it back from the device
        "slot": int(np.asarray(inp["slot_ids"]).reshape(-1)[0]),
        "out": torch.empty((B, T, Hv, dv), dtype=outd, device=device),
    }
    if "parent" in inp:
        d["parent"] = torch.from_numpy(np.ascontiguousarray(inp["parent"], dtype=np.int32)).to(device)
    dims = gdn.make_dims(shape, flags=flags, eps=eps)
    d["dims"] = dims
    if capture:
        tc = T if t_cap is None else t_cap
        d["cap_ssm"] = torch.full((P, tc, Hv, dv, dk), fill_capture, dtype=torch.float32, device=device)
        conv_shape = (P, 3 + tc, C) if mode == gdn.GDN_CHAIN else (P, tc, 3, C)
        d["cap_conv"] = torch.full(conv_shape, fill_capture, dtype=torch.float32, device=device)
        d["capture"] = gdn.Capture(dims, d["cap_ssm"], d["cap_conv"], d["state"], d["conv_state"],
                                   tc, mode)
    return d


def verify(d: dict, n_batch: Optional[int] = None, stream=None, with_capture: bool = True) -> None:
    """gdn_verify over every token of the uploaded inputs (qkv is [B][T][C], so n_tok = T);
    ``n_batch`` may cut the batch to a prefix."""
    T = d["qkv"].shape[1]
    B = d["qkv"].shape[0] if n_batch is None else n_batch
    gdn.gdn_verify(d["dims"], d["state"], d["conv_state"], d["qkv"], d["z"], d["alpha"], d["beta"],
                   d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"],
                   d.get("capture") if with_capture else None, d["out"], T, d["slot_ids"], B,
                   stream)


def verify_resume(d: dict, resume_idx, n_batch: Optional[int] = None, stream=None, dims=None) -> None:
    """gdn_verify_resume over every token of the uploaded inputs: entry b starts from capture
    position resume_idx[b] (device int32) of the uploaded capture, or from its slot's state if < 0.
    ``dims`` replaces the uploaded dims (e.g. the same shape with other flags)."""
    T = d["qkv"].shape[1]
    B = d["qkv"].shape[0] if n_batch is None else n_batch
    gdn.gdn_verify_resume(d["dims"] if dims is None else dims, d["state"], d["conv_state"], d["qkv"], d["z"], d["alpha"],
                          d["beta"], d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"],
                          d["capture"], d["out"], T, d["slot_ids"], resume_idx, B, stream)


def verify_tree(d: dict, stream=None) -> None:
    B, T = d["parent"].shape
    gdn.gdn_verify_tree(d["dims"], d["state"], d["conv_state"], d["qkv"], d["z"], d["alpha"],
                        d["beta"], d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"], d["parent"],
                        d["capture"], d["out"], T, d["slot_ids"], B, stream)


def prefill(d: dict, stream=None) -> None:
    """gdn_prefill of every token of the uploaded single-entry inputs into slot slot_ids[0]."""
    T = d["qkv"].shape[1]
    need = gdn.gdn_prefill_workspace_bytes(d["dims"], T)
    ws = d.get("workspace")
    if ws is None or ws.numel() * 4 < need:
        ws = torch.empty((need + 3) // 4, dtype=torch.float32, device=d["qkv"].device)
        d["workspace"] = ws
    slot = d["slot"]
    gdn.gdn_prefill(d["dims"], d["state"], d["conv_state"], d["qkv"], d["z"], d["alpha"], d["beta"],
                    d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"], d["out"], T, slot, ws,
                    ws.numel() * 4, stream)


def snapshot_replay_round(d: dict, snap: dict, n_accept: int, stream=None) -> None:
    """One spec-decode round with snapshot-and-replay rollback on uploaded inputs (no capture):
    snapshot the batch's slots, verify all T tokens, and when n_accept < T restore the snapshot
    and verify the first n_accept tokens again.  snap holds pool-shaped "state" / "conv_state"."""
    B, T = d["qkv"].shape[0], d["qkv"].shape[1]
    gdn.gdn_snapshot(d["dims"], d["state"], d["conv_state"], snap["state"], snap["conv_state"], d["slot_ids"], B,
                     stream)
    verify(d, stream=stream, with_capture=False)
    if n_accept < T:
        gdn.gdn_restore(d["dims"], d["state"], d["conv_state"], snap["state"], snap["conv_state"], d["slot_ids"], B,
                        stream)
        rep = snap.get("replay")
        if rep is None or rep["n"] != n_accept:  # the accepted prefix of every input, contiguous
            rep = {"n": n_accept}
            for k in ("qkv", "z", "alpha", "beta"):
                rep[k] = d[k][:, :n_accept].contiguous()
            rep["out"] = d["out"][:, :n_accept].contiguous()
            snap["replay"] = rep
        gdn.gdn_verify(d["dims"], d["state"], d["conv_state"], rep["qkv"], rep["z"], rep["alpha"], rep["beta"],
                       d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"], None, rep["out"], n_accept,
                       d["slot_ids"], B, stream)


def layers_step(layers: list, slot_ids, accepted_idx, stream=None) -> None:
    """One spec-decode step over several layers, eagerly: gdn_verify of every layer (capture on,
    all uploaded tokens, every batch entry) with the shared slot_ids, then one
    gdn_rollback_layers to accepted_idx.  The launches a recorded gdn.Graph replays."""
    B, T = layers[0]["qkv"].shape[0], layers[0]["qkv"].shape[1]
    for d in layers:
        gdn.gdn_verify(d["dims"], d["state"], d["conv_state"], d["qkv"], d["z"], d["alpha"], d["beta"],
                       d["A_log"], d["dt_bias"], d["conv_w"], d["norm_w"], d["capture"], d["out"], T, slot_ids,
                       B, stream)
    gdn.gdn_rollback_layers([d["capture"] for d in layers], slot_ids, accepted_idx, B, stream)


def layers_graph(layers: list, slot_ids, accepted_idx,
                 phases: int = gdn.GDN_GRAPH_VERIFY | gdn.GDN_GRAPH_ROLLBACK) -> "gdn.Graph":
    """The same step recorded once (gdn_graph_create) over the uploaded layers' buffers."""
    B, T = layers[0]["qkv"].shape[0], layers[0]["qkv"].shape[1]
    return gdn.Graph(layers[0]["dims"], layers, layers[0]["capture"].t_cap, T, slot_ids, B, accepted_idx, phases)


def upload_block(shape: Shape, inp: dict, *, flags: int = gdn.GDN_F_QK_NORM_SILU) -> dict:
    """Device tensors of one GDN block call (workloads.make_block_inputs): the layer's buffers as
    upload() makes them (qkv, z, alpha, beta become outputs of the input projection), plus
    x [B*T][hidden], the concatenated input weight [C + H_v d_v + 2 H_v][hidden], w_out and
    y [B][T][hidden] (bf16)."""
    B, T, Hv, dv, C = shape.n_batch, shape.n_tok, shape.n_vh, shape.d_v, shape.conv_channels
    hidden = inp["x"].shape[-1]
    lay = dict(inp)
    lay.update(qkv=np.zeros((B, T, C), np.float32), z=np.zeros((B, T, Hv, dv), np.float32),
               alpha=np.zeros((B, T, Hv), np.float32), beta=np.zeros((B, T, Hv), np.float32))
    d = upload(shape, lay, flags=flags)
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16).contiguous()
    d["x"] = bf(inp["x"].reshape(B * T, hidden))
    d["w_in"] = bf(np.concatenate([inp["w_qkv"], inp["w_z"], inp["w_beta"], inp["w_alpha"]], axis=0))
    d["w_out"] = bf(inp["w_out"])
    d["y"] = torch.empty((B, T, hidden), dtype=torch.bfloat16, device="cuda")
    d["hidden"] = hidden
    return d


def block_step(d: dict, stream=None) -> None:
    """One GDN block call: the four input projections as one gdn_linear (beta through a sigmoid),
    gdn_verify with capture over every token, the output projection of the gated output."""
    B, T, C = d["qkv"].shape
    Hv, dv = d["z"].shape[2], d["z"].shape[3]
    Z, hidden, M = Hv * dv, d["hidden"], B * T
    segs = [(0, C, d["qkv"], C, 0), (C, C + Z, d["z"], Z, 0),
            (C + Z, C + Z + Hv, d["beta"], Hv, 1), (C + Z + Hv, C + Z + 2 * Hv, d["alpha"], Hv, 0)]
    gdn.gdn_linear(d["x"], d["w_in"], M, C + Z + 2 * Hv, hidden, segs, stream)
    verify(d, stream=stream)
    gdn.gdn_linear(d["out"], d["w_out"], M, hidden, Z, [(0, hidden, d["y"], hidden, 0)], stream)


def upload_attention(inp: dict, rope: "gdn.gdn_rope_table", *, fmt: int, page_size: int, n_pages: int,
                     prefix: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6) -> dict:
    """Device tensors of one attention_step (workloads.make_attention_inputs): x [B*T][hidden], the
    concatenated weight w_in [(n_q + 2 n_kv) d][hidden], the fused rows qkv [B*T][n_q + 2 n_kv][d] with the
    views q, k and v of them, w_out, y, an empty cache of n_pages pages and the workspace.  The round's lists
    (start, positions, parent, n_new, prefix_pages, prefix_len) are the caller's, as device tensors."""
    B, T, hidden = inp["x"].shape
    n_q, n_kv, hd = inp["n_q"], inp["n_kv"], inp["d"]
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16).contiguous()
    d = {"B": B, "T": T, "hidden": hidden, "rope": rope, "scale": hd ** -0.5}
    d["x"], d["w_in"], d["w_out"] = bf(inp["x"].reshape(B * T, hidden)), bf(inp["w_in"]), bf(inp["w_out"])
    d["qkv"] = torch.empty((B * T, n_q + 2 * n_kv, hd), dtype=torch.bfloat16, device="cuda")
    d["q"], d["k"], d["v"] = d["qkv"][:, :n_q], d["qkv"][:, n_q:n_q + n_kv], d["qkv"][:, n_q + n_kv:]
    d["out"] = torch.empty((B * T, n_q, hd), dtype=torch.bfloat16, device="cuda")
    d["y"] = torch.empty((B, T, hidden), dtype=torch.bfloat16, device="cuda")
    dtype = {gdn.GDN_KV_BF16: torch.bfloat16, gdn.GDN_KV_E4M3: torch.float8_e4m3fn, gdn.GDN_KV_I8: torch.int8}[fmt]
    k, v = (torch.zeros((n_pages, n_kv, page_size, hd), dtype=torch.uint8 if fmt else dtype, device="cuda").view(dtype)
            for _ in range(2))
    sc = [torch.zeros((n_pages, n_kv, page_size), dtype=torch.float32, device="cuda") for _ in range(2 if fmt else 0)]
    d["kv"] = gdn.KvCache(k, v, *sc)
    d["workspace"] = torch.empty(gdn.gdn_attn_workspace_bytes(d["kv"], n_q, B, T, prefix), dtype=torch.uint8, device="cuda")
    d["eps"] = eps  # of those norms (struct TargetWeights: rms_eps)
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):  # weights [d] of the heads' norms, where the layer has them
        d[name] = None if w is None else torch.from_numpy(np.ascontiguousarray(w, dtype=np.float32)).cuda()
    return d


def attention_step(d: dict, table, start, positions, n_new=None, parent=None, prefix_pages=None, prefix_len=None,
                   stream=None) -> None:
    """The attention of a layer over every drafted token: the q, k and v projections as one gdn_linear, the heads' norms
    where the layer has them (lucebox-hub internal.h, struct TargetWeights: q_norm, k_norm), q rotated in place, k rotated
    on its way into the cache, gdn_attn_verify of the chain or tree, the output projection."""
    B, T, kv, M = d["B"], d["T"], d["kv"], d["B"] * d["T"]
    N, Z = d["w_in"].shape[0], d["w_out"].shape[1]
    gdn.gdn_linear(d["x"], d["w_in"], M, N, d["hidden"], [(0, N, d["qkv"], N, 0)], stream)
    for name in ("q", "k"):
        if d.get(name + "_norm") is not None:
            gdn.gdn_norm(d[name], d[name + "_norm"], d[name], M, eps=d.get("eps", 1e-6), stream=stream)
    gdn.gdn_rope(d["rope"], [(d["q"], d["q"])], positions, M, stream=stream)
    gdn.gdn_kv_write(kv, d["k"], d["v"], table, start, n_new, B, T, rope=d["rope"], positions=positions, stream=stream)
    gdn.gdn_attn_verify(kv, d["q"], table, start, n_new, parent, prefix_pages, prefix_len, d["out"], B, T, d["scale"],
                        d["workspace"], stream=stream)
    gdn.gdn_linear(d["out"], d["w_out"], M, d["hidden"], Z, [(0, d["hidden"], d["y"], d["hidden"], 0)], stream)


CODES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def quantise_rows(x, fmt: str, out=None, scale=None, stream=None) -> tuple:
    """(codes [rows][K], scales [rows]) of a bf16 or fp32 matrix x in ``fmt`` (e4m3 or i8; K up to 65536); (x, None) for
    bf16."""
    if fmt == "bf16":
        return x, None
    rows, K = x.shape
    if out is None:
        out = torch.empty((rows, K), dtype=torch.uint8, device=x.device).view(CODES[fmt])
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    gdn.gdn_norm(x[:, None], None, out[:, None], rows, scale=scale[:, None], mode=gdn.GDN_NORM_NONE, stream=stream)
    return out, scale


def _scratch_bytes(M: int, fmt: str, *sizes) -> int:
    """Of the gdn_linear_act calls (N, K, gated) of a step, which run one after another."""
    return max([16] + [gdn.gdn_linear_act_workspace_bytes(M, N, K, CODES[fmt], gated) for N, K, gated in sizes])


def upload_ffn(inp: dict, *, fmt: str = "bf16", eps: float = 1e-6) -> dict:
    """Device tensors of one ffn_step (workloads.make_ffn_inputs): x [M][hidden] bf16 (the mixer's output), stream
    [M][hidden] fp32 (the residual stream), norm_w and the norm's eps, the weights gate_up [2 width][hidden] and down
    [hidden][width] in ``fmt`` (bf16, e4m3 or i8, the 8-bit ones with a scale per row), the buffers between them and the workspace."""
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    M, hidden = inp["x"].shape
    width = inp["w_down"].shape[1]
    d = {"M": M, "hidden": hidden, "width": width, "fmt": fmt, "x": f32(inp["x"]).bfloat16(), "stream": f32(inp["stream"]),
         "norm_w": f32(inp["norm_w"]), "eps": eps}
    for n in ("gate_up", "down"):
        d["w_" + n], d[n + "_scale"] = quantise_rows(f32(inp["w_" + n]).bfloat16(), fmt)
    new = lambda K: torch.empty((M, K), dtype=torch.uint8 if fmt != "bf16" else torch.bfloat16, device="cuda").view(CODES[fmt])
    d["h"], d["act8"] = new(hidden), new(width)
    d["act"] = torch.empty((M, width), dtype=torch.bfloat16, device="cuda")
    for n in ("h_scale", "act_scale"):
        d[n] = None if fmt == "bf16" else torch.empty(M, dtype=torch.float32, device="cuda")
    d["workspace"] = torch.empty(_scratch_bytes(M, fmt, (width, hidden, True), (hidden, width, False)), dtype=torch.uint8,
                                 device="cuda")
    return d


def ffn_step(d: dict, stream=None) -> None:
    """A layer's FFN behind its mixer: the mixer's output added to the residual stream and its norm (in the weights'
    type), SiLU(gate) * up as one product, its rows in 8 bits where the weights are, and the down product onto the
    residual stream."""
    M, K, F, ws = d["M"], d["hidden"], d["width"], d["workspace"]
    rows = lambda t: None if t is None else t[:, None]
    gdn.gdn_norm(rows(d["x"]), d["norm_w"], rows(d["h"]), M, residual=rows(d["stream"]), total=rows(d["stream"]),
                 scale=rows(d["h_scale"]), eps=d.get("eps", 1e-6), stream=stream)
    gdn.gdn_linear_act(d["h"], d["w_gate_up"], d["act"], M, F, K, x_scale=d["h_scale"], w_scale=d["gate_up_scale"],
                       act=gdn.GDN_ACT_SILU, gated=True, workspace=ws, stream=stream)
    act = quantise_rows(d["act"], d["fmt"], d["act8"], d["act_scale"], stream=stream)[0]
    gdn.gdn_linear_act(act, d["w_down"], d["stream"], M, K, F, x_scale=d["act_scale"], w_scale=d["down_scale"],
                       residual=d["stream"], workspace=ws, stream=stream)


def upload_head(inp: dict, *, fmt: str = "bf16", n_ids: int = 1, top_k: int = 0, logits_dtype=torch.bfloat16,
                eps: float = 1e-6) -> dict:
    """Device tensors of one head_step (workloads.make_head_inputs): stream [M][hidden] fp32, norm_w and the norm's eps, the
    vocabulary's weight w [vocab][hidden] in ``fmt``, logits, and what gdn_logprob answers with; ids int32 [M][n_ids] is the caller's
    to fill."""
    f32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    M, hidden = inp["stream"].shape
    V = inp["w"].shape[0]
    d = {"M": M, "hidden": hidden, "vocab": V, "stream": f32(inp["stream"]), "norm_w": f32(inp["norm_w"]),
         "eps": eps}
    d["w"], d["w_scale"] = quantise_rows(f32(inp["w"]).bfloat16(), fmt)
    d["h"] = torch.empty((M, hidden), dtype=torch.uint8 if fmt != "bf16" else torch.bfloat16, device="cuda").view(CODES[fmt])
    d["h_scale"] = None if fmt == "bf16" else torch.empty(M, dtype=torch.float32, device="cuda")
    d["logits"] = torch.empty((M, V), dtype=logits_dtype, device="cuda")
    d["ids"] = torch.full((M, n_ids), -1, dtype=torch.int32, device="cuda")
    d["answer"] = {"lse": torch.empty(M, device="cuda"), "entropy": torch.empty(M, device="cuda"),
                   "logprob": torch.empty((M, n_ids), device="cuda"),
                   "rank": torch.empty((M, n_ids), dtype=torch.int32, device="cuda")}
    if top_k:
        d["answer"].update(top_ids=torch.empty((M, top_k), dtype=torch.int32, device="cuda"),
                           top_logprob=torch.empty((M, top_k), device="cuda"))
    need = max(_scratch_bytes(M, fmt, (V, hidden, False)), gdn.gdn_logprob_workspace_bytes(M, V, logits_dtype, n_ids, top_k))
    d["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return d


def head_step(d: dict, temperature: float = 1.0, stream=None) -> dict:
    """What the step answers with, behind the last layer: the final norm, the vocabulary's logits, and of them the
    drafted tokens' log probabilities and ranks, the rows' entropy and their top alternatives."""
    M, V, ws = d["M"], d["vocab"], d["workspace"]
    gdn.gdn_norm(d["stream"][:, None], d["norm_w"], d["h"][:, None], M, scale=None if d["h_scale"] is None else d["h_scale"][:, None],
                 eps=d.get("eps", 1e-6), stream=stream)
    gdn.gdn_linear_act(d["h"], d["w"], d["logits"], M, V, d["hidden"], x_scale=d["h_scale"], w_scale=d["w_scale"],
                       workspace=ws, stream=stream)
    gdn.gdn_logprob(d["logits"], M, V, ids=d["ids"], temperature=temperature, workspace=ws, stream=stream, **d["answer"])
    return d["answer"]
