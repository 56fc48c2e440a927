"""The operators of a hybrid model's full-attention layers in a speculative-decode step, as cases
to be timed and compared: rotary positions (gdn_rope), the paged KV cache in 16 or 8 bits
(gdn_kv_write, gdn_kv_read) and the attention of drafted tokens over it, with or without a prefix
shared by the whole batch (gdn_attn_verify).

``run`` computes a case in elementary torch operations where ``own`` is false, and through the
library's entry points where it is true.  ``exact`` is the definition in 64 bits, written apart.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
MAX_SCORES = 2 ** 30  # scores of one drawn case: the plain form holds them all in 32 bits


# ------------------------------------------------------------------------------------------ cases
def listed():
    rope = dict(op="rope", scaling="plain", factor=1.0, orig=4096, sections="", theta=1e4, max_pos=4096,
                inverse=False, dtype="bf16", fused=False)
    write = dict(op="write", rope=False, layout="half", rot=0, theta=1e6, max_start=4096, ragged=False, dtype="bf16")
    attn = dict(op="attn", tree=False, ragged=False, prefix=0, n_q=32, n_kv=8, d=128, page=64, ctx_lo=0)
    return [
        # one decoded token of a layer whose first 64 of 256 channels rotate by three position axes: latency
        dict(rope, name="rope_one_token", n_tok=1, n_q=16, n_kv=2, d=256, rot=64, layout="half",
             sections="11,11,10,0", theta=1e7, max_pos=200000),
        # the 64 x 16 drafted tokens of a verify step, long positions under YaRN, q and k inside fused rows
        dict(rope, name="rope_verify_yarn", n_tok=1024, n_q=32, n_kv=8, d=128, rot=128, layout="interleaved",
             scaling="yarn", factor=8.0, orig=32768, theta=1e6, max_pos=262144, fused=True),
        # a prefill's tokens in 32 bits, rotated back (the rotation's gradient)
        dict(rope, name="rope_prefill_f32_back", n_tok=8191, n_q=32, n_kv=8, d=128, rot=96, layout="half",
             scaling="linear", factor=4.0, max_pos=16384, inverse=True, dtype="f32"),
        # one decoded token's k (rotated) and v into an e4m3 cache: latency
        dict(write, name="kv_write_one_token", fmt="e4m3", n_batch=1, n_tok=1, n_kv=2, d=256, page=64, rope=True, rot=64),
        # the drafted tokens of 64 slots, k rotated as it is written, e4m3
        dict(write, name="kv_write_verify_e4m3", fmt="e4m3", n_batch=64, n_tok=16, n_kv=8, d=128, page=64, rope=True,
             layout="interleaved", rot=128, ragged=True),
        # a prefill of four prompts into an 8-bit integer cache, k already rotated
        dict(write, name="kv_write_prefill_i8", fmt="i8", n_batch=4, n_tok=8191, n_kv=8, d=128, page=128, max_start=100),
        # reading a cached prompt back to 16 bits (to hand it to another cache or a snapshot)
        dict(op="read", name="kv_read_e4m3", fmt="e4m3", n_batch=8, n_tok=4096, n_kv=8, d=128, page=64, max_start=2000,
             ragged=True),
        # one token of one short chat: latency
        dict(attn, name="attn_one_token", fmt="bf16", n_batch=1, n_tok=1, n_q=16, n_kv=2, d=256, ctx_hi=37),
        # the tree verify workload's attention: 8 slots, 64-node trees, some thousand cached tokens each
        dict(attn, name="attn_tree_verify_i8", fmt="i8", n_batch=8, n_tok=64, tree=True, ctx_lo=1000, ctx_hi=6000),
        # plain decode of 64 slots with contexts of very different lengths
        dict(attn, name="attn_decode_ragged_e4m3", fmt="e4m3", n_batch=64, n_tok=1, ctx_lo=50, ctx_hi=20000, page=128),
        # a verify step of 64 slots that share a system prompt of some thousand tokens
        dict(attn, name="attn_prefix_verify_e4m3", fmt="e4m3", n_batch=64, n_tok=16, prefix=8100, ctx_lo=10, ctx_hi=700,
             ragged=True),
        # a few drafted tokens each of 32 slots that share a long document, heads of 256 channels, 16 bits
        dict(attn, name="attn_prefix_long_bf16", fmt="bf16", n_batch=32, n_tok=4, n_q=16, n_kv=2, d=256, prefix=32700,
             ctx_lo=100, ctx_hi=900),
    ]


def _log(rng, lo, hi):
    """A whole number spread over lo .. hi by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    d = rng.choice([64, 128, 128, 256])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 6, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["bf16", "e4m3", "i8"])
    rot = rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        half = rot // 2
        sections = ""
        if half >= 4 and rng.random() < 0.3:
            a, b = sorted(rng.sample(range(1, half), 2))
            sections = "%d,%d,%d,0" % (a, b - a, half - b)
        return dict(op=op, n_tok=_log(rng, 1, 8191), n_q=n_q, n_kv=n_kv, d=d, rot=rot, layout=layout,
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn"]) if rot > 2 else "plain",
                    factor=rng.choice([1.5, 4.0, 8.0, 32.0]), orig=rng.choice([4096, 32768]), sections=sections,
                    theta=rng.choice([1e4, 1e6, 1e7]), max_pos=_log(rng, 100, 1000000), inverse=rng.random() < 0.3,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5)
    if op in ("write", "read"):
        b = _log(rng, 1, 64)
        t = _log(rng, 1, max(1, 32768 // b))
        c = dict(op=op, fmt=fmt, n_batch=b, n_tok=t, n_kv=n_kv, d=d, page=page, max_start=_log(rng, 1, 4096),
                 ragged=rng.random() < 0.5)
        if op == "write":
            c.update(rope=fmt != "i8" and rng.random() < 0.6, layout=layout, rot=rot, theta=rng.choice([1e4, 1e6]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]))
        return c
    b, tree = _log(rng, 1, 64), rng.random() < 0.35
    t = _log(rng, 1, 64 if tree else 256)
    hi = _log(rng, 1, 65536)
    return dict(op=op, fmt=fmt, n_batch=b, n_tok=t, n_q=n_q, n_kv=n_kv, d=d, page=page, tree=tree,
                ragged=rng.random() < 0.4, prefix=_log(rng, 1, 32768) if rng.random() < 0.5 else 0,
                ctx_lo=rng.choice([0, hi // 2]), ctx_hi=hi)


def _scores(c):
    return c["n_batch"] * c["n_tok"] * c["n_q"] * (c["prefix"] + c["ctx_hi"] + c["n_tok"]) if c["op"] == "attn" else 0


def _cost(c):
    w = work(c)
    return w["bytes"] / 4e12 + w["flops"] / 4e14


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("rope", "write", "read", "attn")}
    while True:
        c = _draw(rng)
        if _cost(c) <= most[c["op"]] and _scores(c) <= MAX_SCORES:
            return c


def work(c):
    elem = {"bf16": 2, "f32": 4}.get(c.get("dtype"), 2)
    if c["op"] == "rope":
        values = c["n_tok"] * (c["n_q"] + c["n_kv"]) * c["rot"]  # in place: the channels past rot stay
        return {"bytes": 2 * values * elem + 4 * c["n_tok"] * _axes(c), "flops": 3 * values}
    code = 2 if c["fmt"] == "bf16" else 1
    if c["op"] in ("write", "read"):
        rows = c["n_batch"] * c["n_tok"] * c["n_kv"] * 2 * (0.5 if c["ragged"] else 1)
        return {"bytes": rows * (c["d"] * (elem + code) + (4 if code == 1 else 0)), "flops": 4 * rows * c["d"]}
    ctx = (c["ctx_lo"] + c["ctx_hi"]) / 2
    new = c["n_tok"] * (0.5 if c["ragged"] else 1)
    keys = c["prefix"] + c["n_batch"] * (ctx + new)
    heads = c["n_batch"] * new * c["n_q"]
    return {"bytes": keys * c["n_kv"] * 2 * (c["d"] * code + (4 if code == 1 else 0)) + heads * c["d"] * 4,
            "flops": 4 * heads * (c["prefix"] + ctx + new / 2) * c["d"]}


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _axes(c):
    return 4 if c.get("sections") else 1


def _ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device=DEV)


def _tree(rng, n):
    """Parents of a random draft tree of depth at most 8."""
    parent, depth = np.full(n, -1), np.zeros(n, int)
    for i in range(1, n):
        may = np.nonzero(depth[:i] < 8)[0]
        parent[i] = may[rng.integers(len(may))]
        depth[i] = depth[parent[i]] + 1
    return parent


def _pages(rng, n_batch, most, page, n_more=0):
    """Block tables [B][pages of `most` tokens] over a shuffled pool, and the pages of a shared run of n_more tokens."""
    wide, shared = -(-most // page), -(-n_more // page)
    pool = rng.permutation(n_batch * wide + shared + 3)
    return pool[shared:shared + n_batch * wide].reshape(n_batch, wide), pool[:shared], len(pool)


def _cache(c, n_pages, g, filled):
    """Code and scale tensors of a pool: values of about unit size, or zeros."""
    shape = (n_pages, c["n_kv"], c["page"], c["d"])
    out = {}
    for n in ("k", "v"):
        if not filled:
            dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[c["fmt"]]
            codes = torch.zeros(shape, dtype=dt, device=DEV)
        elif c["fmt"] == "bf16":
            codes = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
        else:
            codes = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
            codes = (codes.mul_(140).clamp_(-448, 448).to(torch.float8_e4m3fn) if c["fmt"] == "e4m3"
                     else codes.mul_(40).round_().clamp_(-127, 127).to(torch.int8))
        out[n] = codes
        if c["fmt"] != "bf16":
            s = torch.rand(shape[:3], device=DEV, generator=g) if filled else torch.zeros(shape[:3], device=DEV)
            out[n + "_scale"] = s.add_(0.5).div_(140 if c["fmt"] == "e4m3" else 40) if filled else s
    return out


def prepare(c, seed):
    rng, g = np.random.default_rng(seed), _gen(seed)
    s = {"case": c}
    if c["op"] == "rope":
        n, hq, hk, d = c["n_tok"], c["n_q"], c["n_kv"], c["d"]
        dt = _dtype(c["dtype"])
        if c["fused"]:  # q and k inside rows that also hold v
            rows = torch.randn((n, hq + 2 * hk, d), device=DEV, generator=g).to(dt)
            s["q"], s["k"] = rows[:, :hq], rows[:, hq:hq + hk]
        else:
            s["q"] = torch.randn((n, hq, d), device=DEV, generator=g).to(dt)
            s["k"] = torch.randn((n, hk, d), device=DEV, generator=g).to(dt)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"].contiguous()), torch.empty_like(s["k"].contiguous())
        s["positions"] = _ints(rng.integers(0, c["max_pos"] + 1, (_axes(c), n)))
    elif c["op"] in ("write", "read"):
        b, t = c["n_batch"], c["n_tok"]
        start = rng.integers(0, c["max_start"] + 1, b)
        s["start"] = _ints(start)
        s["n_new"] = _ints(rng.integers(0, t + 1, b)) if c["ragged"] else None
        table, _, n_pages = _pages(rng, b, c["max_start"] + t, c["page"])
        s["table"] = _ints(table)
        s.update(_cache(c, n_pages, g, c["op"] == "read"))
        if c["op"] == "write":
            rows = torch.randn((b * t, 2 * c["n_kv"], c["d"]), device=DEV, generator=g).to(_dtype(c["dtype"]))
            s["new_k"], s["new_v"] = rows[:, :c["n_kv"]], rows[:, c["n_kv"]:]  # halves of fused rows
            s["positions"] = _ints((start[:, None] + np.arange(t)[None]).reshape(1, -1))
        else:
            s["k_out"], s["v_out"] = (torch.zeros((b * t, c["n_kv"], c["d"]), dtype=torch.bfloat16, device=DEV)
                                      for _ in range(2))
    else:
        b, t = c["n_batch"], c["n_tok"]
        ctx = rng.integers(c["ctx_lo"], c["ctx_hi"] + 1, b)
        s["ctx"] = _ints(ctx)
        s["n_new"] = _ints(rng.integers(1, t + 1, b)) if c["ragged"] else None
        s["parent"] = _ints([_tree(rng, t) for _ in range(b)]) if c["tree"] else None
        table, shared, n_pages = _pages(rng, b, c["ctx_hi"] + t, c["page"], c["prefix"])
        s["table"] = _ints(table)
        s["prefix_pages"] = _ints(shared) if c["prefix"] else None
        s["prefix_len"] = _ints([c["prefix"]]) if c["prefix"] else None
        s.update(_cache(c, n_pages, g, True))
        s["q"] = (2 * torch.randn((b * t, c["n_q"], c["d"]), device=DEV, generator=g)).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program holds beside its tensors: the rotary table, the cache's descriptor, the workspace."""
    from gated_deltanet_linear_verify_amd import gdn
    c = s["case"]
    if c["op"] == "rope" or c.get("rope"):
        s["rope"] = gdn.gdn_rope_init(
            c["rot"], theta=c["theta"], layout={"half": gdn.GDN_ROPE_HALF, "interleaved": gdn.GDN_ROPE_INTERLEAVED}[c["layout"]],
            scaling={"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "ntk": gdn.GDN_ROPE_NTK,
                     "yarn": gdn.GDN_ROPE_YARN}[c.get("scaling", "plain")],
            factor=c.get("factor", 1.0), orig_ctx=c.get("orig", 0),
            sections=[int(x) for x in c["sections"].split(",")] if c.get("sections") else None)
    if c["op"] != "rope":
        s["kv"] = gdn.KvCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
    if c["op"] == "attn":
        need = gdn.gdn_attn_workspace_bytes(s["kv"], c["n_q"], c["n_batch"], c["n_tok"], c["prefix"] > 0)
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------- the plain forms
def _freqs(c):
    """Frequency of every pair, and the factor on cos and sin, in 64 bits."""
    rot, theta, scaling = c["rot"], c["theta"], c.get("scaling", "plain")
    factor = c.get("factor", 1.0)
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        low, high = (rot * math.log(c["orig"] / (turns * 2 * math.pi)) / (2 * math.log(theta)) for turns in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def _angles(c, positions):
    """Angles [n_tok][rot/2] in 64 bits, each pair by its own axis of positions."""
    f, m = _freqs(c)
    axis = torch.zeros(c["rot"] // 2, dtype=torch.long, device=DEV)
    if c.get("sections"):
        counts = torch.tensor([int(x) for x in c["sections"].split(",")], device=DEV)
        axis = torch.repeat_interleave(torch.arange(4, device=DEV), counts)
    return positions.double()[axis].T * f, m


def _rotate(c, x, positions, inverse=False):
    """x [n][heads][d] in 32 bits, rotated."""
    angle, m = _angles(c, positions)
    cos, sin = ((m * t).float()[:, None] for t in (angle.cos(), angle.sin()))
    sin = -sin if inverse else sin
    rot, half = c["rot"], c["rot"] // 2
    out = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        out[..., :half], out[..., half:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return out


def _where(c, s):
    """Token rows in play: their index in [B T], page and place in the page."""
    b, t = c["n_batch"], c["n_tok"]
    pos = s["start"].long()[:, None] + torch.arange(t, device=DEV)
    live = torch.ones_like(pos, dtype=torch.bool)
    if s["n_new"] is not None:
        live = torch.arange(t, device=DEV)[None] < s["n_new"][:, None]
    row = live.reshape(-1).nonzero()[:, 0]
    page = torch.gather(s["table"].long(), 1, pos // c["page"]).reshape(-1)[row]
    return row, page, (pos % c["page"]).reshape(-1)[row]


def _quantise(x, fmt):
    most = torch.full((1,), 448.0 if fmt == "e4m3" else 127.0, device=DEV)
    scale = x.abs().amax(-1) / most  # a tensor's division: a number's would multiply by its reciprocal
    inv = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
    y = x * inv[..., None]
    return (y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().clamp(-127, 127).to(torch.int8)), scale


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _gather(c, s, n, page, at):
    """Rows of cache n at (page, at), any shape of indices: [...][n_kv][d] in 32 bits."""
    x = _bytes(s[n])[page, :, at]
    x = (x.view(torch.float8_e4m3fn) if c["fmt"] == "e4m3" else x).float()
    return x if c["fmt"] == "bf16" else x * s[n + "_scale"][page, :, at][..., None]


def _attend(c, s):
    b, t, hk, d, p = c["n_batch"], c["n_tok"], c["n_kv"], c["d"], c["prefix"]
    grp = c["n_q"] // hk
    q = s["q"].float().view(b, t, hk, grp, d).permute(0, 2, 1, 3, 4)  # [b][hk][t][grp][d]
    length = s["table"].shape[1] * c["page"]
    pos = torch.arange(length, device=DEV)
    page, at = s["table"].long()[:, pos // c["page"]], (pos % c["page"]).expand(b, length)
    k, v = (_gather(c, s, n, page, at).permute(0, 2, 1, 3).contiguous() for n in ("k", "v"))  # [b][hk][length][d]
    # drafted key j is at ctx + j; a query sees the context and its ancestors or itself
    j = torch.arange(t, device=DEV)
    if c["tree"]:
        up = torch.where(s["parent"] < 0, t, s["parent"]).long()  # t: above the root
        up = torch.cat([up, torch.full((b, 1), t, device=DEV)], 1)
        sees = torch.zeros((b, t, t + 1), dtype=torch.bool, device=DEV)
        node = j.expand(b, t).clone()
        for _ in range(9):  # a path holds at most nine nodes
            sees.scatter_(2, node[..., None], True)
            node = torch.gather(up, 1, node)
        sees = sees[..., :t]
    else:
        sees = (j[None] <= j[:, None]).expand(b, t, t)
    rel = pos[None] - s["ctx"][:, None].long()
    draft = torch.gather(sees, 2, rel.clamp(0, t - 1)[:, None].expand(b, t, length)) & ((rel >= 0) & (rel < t))[:, None]
    mask = (draft | (rel < 0)[:, None])[:, None, :, None]  # [b][1][t][1][length]
    score = (q.reshape(b, hk, t * grp, d) @ k.transpose(2, 3).contiguous()).view(b, hk, t, grp, length)
    score = (score * d ** -0.5).masked_fill_(~mask, -math.inf)
    if p:
        pp = torch.arange(p, device=DEV)
        pk, pv = (_gather(c, s, n, s["prefix_pages"].long()[pp // c["page"]], pp % c["page"]).permute(1, 0, 2).contiguous()
                  for n in ("k", "v"))  # [hk][p][d]
        qp = q.permute(1, 0, 2, 3, 4).reshape(hk, b * t * grp, d)
        pre = (qp @ pk.transpose(1, 2).contiguous()).view(hk, b, t, grp, p).transpose(0, 1) * d ** -0.5
        top = torch.maximum(score.amax(-1), pre.amax(-1))[..., None]
        score, pre = (score - top).exp_(), (pre - top).exp_()
        o = (score.reshape(b, hk, t * grp, length) @ v).view(b, hk, t, grp, d)
        o = o + (pre.transpose(0, 1).reshape(hk, b * t * grp, p) @ pv).view(hk, b, t, grp, d).transpose(0, 1)
        total = score.sum(-1) + pre.sum(-1)
    else:
        score = (score - score.amax(-1, keepdim=True)).exp_()
        o = (score.reshape(b, hk, t * grp, length) @ v).view(b, hk, t, grp, d)
        total = score.sum(-1)
    o = (o / total[..., None]).permute(0, 2, 1, 3, 4).reshape(b * t, c["n_q"], d)
    if s["n_new"] is not None:
        live = j[None] < s["n_new"][:, None]
        o = torch.where(live.reshape(-1)[:, None, None], o, torch.zeros_like(o))
    return o.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(c, s)
    if c["op"] == "rope":
        return {"q": _rotate(c, s["q"].float(), s["positions"], c["inverse"]).to(s["q"].dtype),
                "k": _rotate(c, s["k"].float(), s["positions"], c["inverse"]).to(s["k"].dtype)}
    if c["op"] == "write":
        row, page, at = _where(c, s)
        k, v = s["new_k"][row].float(), s["new_v"][row].float()
        if c["rope"]:
            k = _rotate(c, k, s["positions"][:, row])
        for n, x in (("k", k), ("v", v)):
            if c["fmt"] == "bf16":
                s[n][page, :, at] = x.to(torch.bfloat16)
            else:
                codes, scale = _quantise(x, c["fmt"])
                _bytes(s[n])[page, :, at] = _bytes(codes)
                s[n + "_scale"][page, :, at] = scale
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s}
    if c["op"] == "read":
        row, page, at = _where(c, s)
        for n in ("k", "v"):
            s[n + "_out"][row] = _gather(c, s, n, page, at).to(torch.bfloat16)
        return {"k": s["k_out"], "v": s["v_out"]}
    return _attend(c, s)


def _run_own(c, s):
    from gated_deltanet_linear_verify_amd import gdn
    if c["op"] == "rope":
        gdn.gdn_rope(s["rope"], [(s["q"], s["q_out"]), (s["k"], s["k_out"])], s["positions"], c["n_tok"],
                     inverse=c["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "write":
        gdn.gdn_kv_write(s["kv"], s["new_k"], s["new_v"], s["table"], s["start"], s["n_new"], c["n_batch"], c["n_tok"],
                         rope=s.get("rope"), positions=s["positions"] if c["rope"] else None)
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s}
    if c["op"] == "read":
        gdn.gdn_kv_read(s["kv"], s["table"], s["start"], s["n_new"], s["k_out"], s["v_out"], c["n_batch"], c["n_tok"])
        return {"k": s["k_out"], "v": s["v_out"]}
    gdn.gdn_attn_verify(s["kv"], s["q"], s["table"], s["ctx"], s["n_new"], s["parent"], s["prefix_pages"], s["prefix_len"],
                        s["out"], c["n_batch"], c["n_tok"], c["d"] ** -0.5, s["workspace"])
    return s["out"]


# ----------------------------------------------------------------------------- the definition, in 64 bits
def _exact_turn(c, x, positions, back):
    """Rotation as a product of complex numbers, pair by pair."""
    rot, half = c["rot"], c["rot"] // 2
    base, factor, kind = c["theta"], c.get("factor", 1.0), c.get("scaling", "plain")
    m = 1.0
    if kind == "ntk":
        base *= factor ** (rot / (rot - 2.0))
    freq = [1.0 / base ** (2.0 * i / rot) for i in range(half)]
    if kind == "linear":
        freq = [f / factor for f in freq]
    elif kind == "yarn":
        # pairs that turn over 32 times within the trained length keep their frequency, those under once are
        # slowed by the factor, and those between are blended by their index
        at = lambda turns: rot * math.log(c["orig"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        wide = hi - lo if hi > lo else 0.001
        mix = [min(1.0, max(0.0, (i - lo) / wide)) for i in range(half)]
        freq = [f * (w / factor + 1 - w) for f, w in zip(freq, mix)]
        m += 0.1 * math.log(factor)
    owner = []
    for a, n in enumerate(int(v) for v in (c["sections"].split(",") if c.get("sections") else [half])):
        owner += [a] * n
    x, p = x.double(), positions.double()
    out = x.clone()
    first = range(half) if c["layout"] == "half" else range(0, rot, 2)
    step = half if c["layout"] == "half" else 1
    for i, ch in enumerate(first):
        turn = torch.polar(torch.full_like(p[owner[i]], m), p[owner[i]] * (-freq[i] if back else freq[i]))[:, None]
        z = torch.complex(x[..., ch], x[..., ch + step]) * turn
        out[..., ch], out[..., ch + step] = z.real, z.imag
    return out


def _exact_value(c, s, n, page, at, head):
    codes = _bytes(s[n])[page, head, at]
    codes = (codes.view(torch.float8_e4m3fn) if c["fmt"] == "e4m3" else codes).double()
    return codes if c["fmt"] == "bf16" else codes * s[n + "_scale"][page, head, at].double()[:, None]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return {n: _exact_turn(c, s[n], s["positions"], c["inverse"]) for n in ("q", "k")}
    if c["op"] == "write":
        out = {n: None for n in ("k", "v", "k_scale", "v_scale") if n in s}
        new = {"k": _exact_turn(c, s["new_k"], s["positions"], False) if c["rope"] else s["new_k"].double(),
               "v": s["new_v"].double()}
        for n in ("k", "v"):
            made = s[n].double() if c["fmt"] == "bf16" else s[n + "_scale"].double()
            for b in range(c["n_batch"]):
                start, t = int(s["start"][b]), c["n_tok"] if s["n_new"] is None else int(s["n_new"][b])
                pos = torch.arange(start, start + t, device=DEV)
                x = new[n][b * c["n_tok"]:b * c["n_tok"] + t]
                made[s["table"][b].long()[pos // c["page"]], :, pos % c["page"]] = (
                    x if c["fmt"] == "bf16" else x.abs().amax(-1) / (448.0 if c["fmt"] == "e4m3" else 127.0))
            out[n if c["fmt"] == "bf16" else n + "_scale"] = made  # codes of 8 bits have no value between
        return out
    if c["op"] == "read":
        out = {n: torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV) for n in ("k", "v")}
        for n in ("k", "v"):
            for b in range(c["n_batch"]):
                start, t = int(s["start"][b]), c["n_tok"] if s["n_new"] is None else int(s["n_new"][b])
                pos = torch.arange(start, start + t, device=DEV)
                for h in range(c["n_kv"]):
                    out[n][b * c["n_tok"]:b * c["n_tok"] + t, h] = _exact_value(
                        c, s, n, s["table"][b].long()[pos // c["page"]], pos % c["page"], h)
        return out
    t, hk, d = c["n_tok"], c["n_kv"], c["d"]
    grp = c["n_q"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["n_batch"]):
        ctx, new = int(s["ctx"][b]), t if s["n_new"] is None else int(s["n_new"][b])
        pre = torch.arange(c["prefix"], device=DEV)
        pos = torch.arange(ctx + new, device=DEV)
        page, at = s["table"][b].long()[pos // c["page"]], pos % c["page"]
        if c["prefix"]:
            page = torch.cat([s["prefix_pages"].long()[pre // c["page"]], page])
            at = torch.cat([pre % c["page"], at])
        sees = np.zeros((new, new), bool)
        parent = s["parent"][b].tolist() if c["tree"] else list(range(-1, t - 1))
        for i in range(new):
            if parent[i] >= 0:
                sees[i] = sees[parent[i]]
            sees[i, i] = True
        sees = torch.cat([torch.ones((new, c["prefix"] + ctx), dtype=torch.bool, device=DEV),
                          torch.tensor(sees, device=DEV)], 1).repeat_interleave(grp, 0)
        for h in range(hk):
            k, v = (_exact_value(c, s, n, page, at, h) for n in ("k", "v"))
            q = s["q"][b * t:b * t + new, h * grp:(h + 1) * grp].double().reshape(new * grp, d)
            w = torch.where(sees, q @ k.T.contiguous() / math.sqrt(d), torch.full((), -math.inf, dtype=torch.float64, device=DEV))
            o = torch.softmax(w, -1) @ v
            out[b * t:b * t + new, h * grp:(h + 1) * grp] = o.reshape(new, grp, d)
    return out
