"""What stands between and behind a hybrid model's mixers in a speculative-decode step, as cases to be timed and
compared: the norm with the residual's addition and an output in 16 or 8 bits (gdn_norm), products with bias,
activation and residual in their epilogue over operands of 16 or 8 bits (gdn_linear_act), and the log probabilities
of the drafted tokens with ranks, entropy and top alternatives (gdn_logprob).

``run`` computes a case in elementary torch operations where ``own`` is false, and through the library's entry
points where it is true.  ``exact`` is the definition in 64 bits, written apart.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
FULL = {"e4m3": 448.0, "i8": 127.0}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "i8": 1, "": 0}


# ------------------------------------------------------------------------------------------ cases
def listed():
    norm = dict(op="norm", n_heads=1, d=5120, x="bf16", residual="bf16", out="e4m3", fused=False)
    lin = dict(op="linear", dtype="bf16", act="none", gated=False, bias=False, residual="", out="bf16")
    logp = dict(op="logprob", dtype="bf16", n_ids=1, top_k=0, temperature=1.0, masked=False)
    return [
        # the norm before a layer's projections for one decoded token, in 8 bits for their operands: latency
        dict(norm, name="norm_one_token", n_tok=1),
        # the norms of the q heads of a verify step's 64 x 16 tokens, inside the fused q, k and v rows
        dict(norm, name="norm_heads_verify", n_tok=1024, n_heads=16, d=256, residual="", out="bf16", fused=True),
        # a verify step's rows into 8-bit integers
        dict(norm, name="norm_verify_i8", n_tok=1024, out="i8"),
        # a prefill's rows with the residual stream in 32 bits
        dict(norm, name="norm_prefill_e4m3", n_tok=8191, residual="f32"),
        # a mixer's output projection for one decoded token, with the residual: latency and the weight's bytes
        dict(lin, name="linear_one_token", n_tok=1, n=5120, k=4096, residual="bf16"),
        # an FFN's gate and up products for one slot's drafted tokens: the weight's bytes
        dict(lin, name="linear_gate_up_one_slot_e4m3", n_tok=16, n=13824, k=5120, dtype="e4m3", act="silu", gated=True),
        # the same for 64 slots
        dict(lin, name="linear_gate_up_verify_e4m3", n_tok=1024, n=13824, k=5120, dtype="e4m3", act="silu", gated=True),
        # an FFN's down product for 64 slots, 8-bit integers, onto a 32-bit residual stream
        dict(lin, name="linear_down_verify_i8", n_tok=1024, n=5120, k=13824, dtype="i8", residual="f32", out="f32"),
        # a prefill's product with bias and activation in 16 bits; the width of the GDN block's four input projections
        dict(lin, name="linear_prefill_bf16", n_tok=8191, n=12352, k=5120, act="gelu_tanh", bias=True),
        # what one decoded token answers with: latency
        dict(logp, name="logprob_one_token", n_tok=1, vocab=131072, top_k=5),
        # the answers of a verify step of 64 slots over a vocabulary of odd length, part of it masked
        dict(logp, name="logprob_verify", n_tok=1024, vocab=131071, top_k=20, masked=True),
        # 8 trees of 64 nodes, each node scoring its children, logits in 32 bits, sampled at a temperature
        dict(logp, name="logprob_tree_f32", n_tok=512, vocab=32001, dtype="f32", n_ids=4, temperature=0.7),
    ]


def _log(rng, lo, hi):
    """A whole number spread over lo .. hi by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw(rng):
    op = rng.choice(["norm", "linear", "linear", "logprob"])
    if op == "norm":
        heads = rng.choice([1, 1, 1, 2, 8, 24])
        return dict(op=op, n_tok=_log(rng, 1, 8191), n_heads=heads, d=_log(rng, 64, 16384 if heads == 1 else 512),
                    x=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f32", "e4m3", "i8"]), fused=rng.random() < 0.3)
    if op == "linear":
        gated = rng.random() < 0.4
        return dict(op=op, n_tok=_log(rng, 1, 8191), n=_log(rng, 1, 28000), k=16 * _log(rng, 1, 1024),
                    dtype=rng.choice(["bf16", "e4m3", "i8"]), gated=gated, bias=rng.random() < 0.4,
                    act=rng.choice(["silu", "gelu", "gelu_tanh"] + ([] if gated else ["none", "none", "relu", "sigmoid"])),
                    residual=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]))
    vocab = _log(rng, 100, 160000)
    return dict(op=op, n_tok=_log(rng, 1, 2048), vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f32"]),
                n_ids=rng.choice([0, 1, 1, 2, 5]), top_k=rng.choice([0, 1, 5, 20, 50]),
                temperature=rng.choice([1.0, 1.0, 0.6, 1.3]), masked=rng.random() < 0.4)


def _cost(c):
    w = work(c)
    return w["bytes"] / 4e12 + w["flops"] / 4e14


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("norm", "linear", "logprob")}
    while True:
        c = _draw(rng)
        if _cost(c) <= most[c["op"]]:
            return c


def work(c):
    m = c["n_tok"]
    if c["op"] == "norm":
        values = m * c["n_heads"] * c["d"]
        per = SIZE[c["x"]] + 2 * SIZE[c["residual"]] + SIZE[c["out"]]  # the sum is stored where there is a residual
        return {"bytes": values * per + 4 * c["d"] + (4 * m * c["n_heads"] if c["out"] in FULL else 0), "flops": 5 * values}
    if c["op"] == "linear":
        rows = c["n"] * (2 if c["gated"] else 1)
        per_row = (4 if c["dtype"] in FULL else 0)
        return {"bytes": (m + rows) * (c["k"] * SIZE[c["dtype"]] + per_row) + (4 * rows if c["bias"] else 0)
                + m * c["n"] * (SIZE[c["residual"]] + SIZE[c["out"]]), "flops": 2 * m * rows * c["k"]}
    return {"bytes": m * (c["vocab"] * SIZE[c["dtype"]] + 12 * c["n_ids"] + 8 * c["top_k"] + 8), "flops": 5 * m * c["vocab"]}


# ----------------------------------------------------------------------------------------- inputs
def _codes(shape, name, g):
    """Codes of unit variance times Q / 3.2, as rows quantised by their own maximum have them."""
    x = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
    if name == "e4m3":
        return x.mul_(140).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x.mul_(40).round_().clamp_(-127, 127).to(torch.int8)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    m = c["n_tok"]
    randn = lambda *shape: torch.randn(shape, device=DEV, generator=g)  # noqa: E731
    if c["op"] == "norm":
        h, d = c["n_heads"], c["d"]
        wide = randn(m, h + 2 if c["fused"] else h, d).to(TYPES[c["x"]])
        s["x"] = wide[:, :h]
        s["weight"] = 1 + 0.1 * randn(d)
        s["out"] = torch.empty((m, h, d), dtype=TYPES[c["out"]], device=DEV)
        if c["residual"]:
            s["residual"] = (3 * randn(m, h, d)).to(TYPES[c["residual"]])
            s["sum"] = torch.empty_like(s["residual"])
        if c["out"] in FULL:
            s["scale"] = torch.empty((m, h), device=DEV)
    elif c["op"] == "linear":
        rows = c["n"] * (2 if c["gated"] else 1)
        if c["dtype"] == "bf16":
            s["x"] = randn(m, c["k"]).to(torch.bfloat16)
            s["w"] = (randn(rows, c["k"]) * c["k"] ** -0.5).to(torch.bfloat16)
        else:
            unit = 140 if c["dtype"] == "e4m3" else 40
            s["x"], s["w"] = _codes((m, c["k"]), c["dtype"], g), _codes((rows, c["k"]), c["dtype"], g)
            s["x_scale"] = (torch.rand(m, device=DEV, generator=g) + 0.5) / unit
            s["w_scale"] = (torch.rand(rows, device=DEV, generator=g) + 0.5) / (unit * c["k"] ** 0.5)
        if c["bias"]:
            s["bias"] = 0.5 * randn(rows)
        if c["residual"]:
            s["residual"] = (2 * randn(m, c["n"])).to(TYPES[c["residual"]])
        s["out"] = torch.empty((m, c["n"]), dtype=TYPES[c["out"]], device=DEV)
    else:
        v = c["vocab"]
        logits = 2.5 * randn(m, v)
        # most rows are sure of a token, which a drafted one often is
        likely = torch.randint(0, v, (m,), device=DEV, generator=g)
        sure = 12 * torch.rand(m, device=DEV, generator=g) + 4
        logits[torch.arange(m, device=DEV), likely] += sure
        if c["masked"]:  # a block of the vocabulary that may not be emitted, another for every row
            j, first = torch.arange(v, device=DEV), torch.randint(0, v, (m, 1), device=DEV, generator=g)
            gone = (j >= first) & (j < first + v // 4) & (j != likely[:, None])
            logits.masked_fill_(gone, -math.inf)
        s["logits"] = logits.to(TYPES[c["dtype"]])
        if c["n_ids"]:
            ids = torch.randint(0, v, (m, c["n_ids"]), device=DEV, generator=g)
            drafted = torch.rand(m, device=DEV, generator=g) < 0.7
            ids[:, 0] = torch.where(drafted, likely, ids[:, 0])
            if c["n_ids"] > 1:  # a node with fewer children
                ids[:, 1:][torch.rand((m, c["n_ids"] - 1), device=DEV, generator=g) < 0.2] = -1
            s["ids"] = ids.to(torch.int32)
            s["logprob"] = torch.empty((m, c["n_ids"]), device=DEV)
            s["rank"] = torch.empty((m, c["n_ids"]), dtype=torch.int32, device=DEV)
        s["lse"], s["entropy"] = torch.empty(m, device=DEV), torch.empty(m, device=DEV)
        if c["top_k"]:
            s["top_ids"] = torch.empty((m, c["top_k"]), dtype=torch.int32, device=DEV)
            s["top_logprob"] = torch.empty((m, c["top_k"]), device=DEV)
    if own:  # scratch memory, which a program keeps beside its tensors
        s["workspace"] = torch.empty(max(16, _workspace_bytes(c)), dtype=torch.uint8, device=DEV)
    return s


def _workspace_bytes(c):
    from gated_deltanet_linear_verify_amd import gdn
    if c["op"] == "linear":
        return gdn.gdn_linear_act_workspace_bytes(c["n_tok"], c["n"], c["k"], TYPES[c["dtype"]], c["gated"])
    if c["op"] == "logprob":
        return gdn.gdn_logprob_workspace_bytes(c["n_tok"], c["vocab"], TYPES[c["dtype"]], c["n_ids"], c["top_k"])
    return 0


# ------------------------------------------------------------------------------- the plain forms
def _norm(c, s):
    x = s["x"].float()
    out = {}
    if c["residual"]:
        x = x + s["residual"].float()
        out["sum"] = x.to(s["sum"].dtype)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if c["out"] not in FULL:
        out["out"] = y.to(TYPES[c["out"]])
        return out
    scale = y.abs().amax(-1, keepdim=True) / FULL[c["out"]]
    y = y * (1 / scale)
    if c["out"] == "e4m3":
        out["out"] = y.to(torch.float8_e4m3fn)
    else:
        out["out"] = (y.round() * scale).to(torch.bfloat16)
    out["scale"] = scale[..., 0]
    return out


def _activate(name, y):
    if name == "silu":
        return y / (1 + torch.exp(-y))
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-y))
    if name == "relu":
        return y.clamp_min(0)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _linear(c, s):
    y = s["x"].float() @ s["w"].float().t()
    if c["dtype"] in FULL:
        y = y * s["x_scale"][:, None] * s["w_scale"]
    if c["bias"]:
        y = y + s["bias"]
    if c["gated"]:
        y = _activate(c["act"], y[:, :c["n"]]) * y[:, c["n"]:]
    else:
        y = _activate(c["act"], y)
    if c["residual"]:
        y = y + s["residual"].float()
    return {"out": y.to(TYPES[c["out"]])}


def _ordered(x):
    """Whole numbers in the order of the floats x (32 bits, no NaN): of two zeros neither is more."""
    b = (x + 0.0).view(torch.int32).to(torch.int64)
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _logprob(c, s):
    raw = s["logits"].float()
    l = raw / c["temperature"]
    top = l.amax(-1, keepdim=True)
    e = (l - top).exp_()
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    lp = l - lse
    p = e / total
    out = {"lse": lse[:, 0], "entropy": -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)}
    place = torch.arange(c["vocab"], device=DEV)
    if c["n_ids"]:
        ids = s["ids"].long()
        at, given = ids.clamp_min(0), ids >= 0
        mine = torch.gather(raw, 1, at)
        ranks = torch.zeros_like(ids)
        for i in range(c["n_ids"]):
            ranks[:, i] = ((raw > mine[:, i:i + 1]) | ((raw == mine[:, i:i + 1]) & (place < at[:, i:i + 1]))).sum(-1)
        out["logprob"] = torch.where(given, torch.gather(lp, 1, at), torch.full_like(mine, -math.inf))
        out["rank"] = torch.where(given, ranks, -torch.ones_like(ranks)).to(torch.int32)
    if c["top_k"]:
        key = (_ordered(raw) << 20) + (2 ** 20 - 1 - place)  # of equal logits the lower index first
        best = torch.topk(key, c["top_k"], -1).values
        out["top_ids"] = (2 ** 20 - 1 - (best & (2 ** 20 - 1))).to(torch.int32)
        out["top_logprob"] = torch.gather(lp, 1, out["top_ids"].long())
    return out


# ---------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(c, s)
    return {"norm": _norm, "linear": _linear, "logprob": _logprob}[c["op"]](c, s)


def _run_own(c, s):
    from gated_deltanet_linear_verify_amd import gdn
    if c["op"] == "norm":
        gdn.gdn_norm(s["x"], s["weight"], s["out"], c["n_tok"], residual=s.get("residual"), total=s.get("sum"),
                     scale=s.get("scale"), eps=EPS)
        out = {n: s[n] for n in ("sum", "out", "scale") if n in s}
        if c["out"] == "i8":  # codes stand for code * scale
            out["out"] = (s["out"] * s["scale"][..., None]).to(torch.bfloat16)
        return out
    if c["op"] == "linear":
        act = {"none": gdn.GDN_ACT_NONE, "silu": gdn.GDN_ACT_SILU, "gelu": gdn.GDN_ACT_GELU, "relu": gdn.GDN_ACT_RELU,
               "gelu_tanh": gdn.GDN_ACT_GELU_TANH, "sigmoid": gdn.GDN_ACT_SIGMOID}[c["act"]]
        gdn.gdn_linear_act(s["x"], s["w"], s["out"], c["n_tok"], c["n"], c["k"], x_scale=s.get("x_scale"),
                           w_scale=s.get("w_scale"), bias=s.get("bias"), act=act, gated=c["gated"],
                           residual=s.get("residual"), workspace=s["workspace"])
        return {"out": s["out"]}
    gdn.gdn_logprob(s["logits"], c["n_tok"], c["vocab"], ids=s.get("ids"), temperature=c["temperature"],
                    logprob=s.get("logprob"), rank=s.get("rank"), lse=s["lse"], entropy=s["entropy"],
                    top_ids=s.get("top_ids"), top_logprob=s.get("top_logprob"), workspace=s["workspace"])
    return {n: s[n] for n in ("lse", "entropy", "logprob", "rank", "top_ids", "top_logprob") if n in s}


# ----------------------------------------------------------------------------- the definition, in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        x, out = s["x"].double(), {}
        if c["residual"]:
            x = out["sum"] = x + s["residual"].double()
        y = s["weight"].double() * x / ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        if c["out"] in FULL:
            most = y.abs().max(-1).values
            out["scale"] = most / FULL[c["out"]]
            # e4m3: in units of the scale, before the rounding to codes; whole codes have no value between
            y = y / out["scale"][..., None] if c["out"] == "e4m3" else None
        out["out"] = y
        return out
    if c["op"] == "linear":
        x, w = s["x"].double(), s["w"].double()
        if "x_scale" in s:
            x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
        b = s["bias"].double() if c["bias"] else torch.zeros(len(w), dtype=torch.float64, device=DEV)
        a = torch.addmm(b, x, w.t())
        up = a[:, c["n"]:] if c["gated"] else 1.0
        a = a[:, :c["n"]]
        cdf = {"none": lambda t: 1.0, "relu": lambda t: (t > 0).double(), "silu": torch.sigmoid,
               "gelu": lambda t: torch.erfc(-t / math.sqrt(2)) / 2,
               "gelu_tanh": lambda t: torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))}
        a = torch.sigmoid(a) if c["act"] == "sigmoid" else a * cdf[c["act"]](a)
        a = a * up
        return {"out": a + s["residual"].double() if c["residual"] else a}
    l = s["logits"].double() / c["temperature"]
    z = torch.logsumexp(l, -1)
    lp = l - z[:, None]
    out = {"lse": z, "entropy": -torch.special.xlogy(lp.exp(), lp.exp()).sum(-1)}
    if c["n_ids"]:
        ids = s["ids"].cpu().numpy()
        got = np.full(ids.shape, -np.inf)
        row, i = np.nonzero(ids >= 0)
        got[row, i] = lp[torch.from_numpy(row), torch.from_numpy(ids[row, i]).long()].cpu().numpy()
        out["logprob"], out["rank"] = torch.from_numpy(got), None
    if c["top_k"]:
        out["top_ids"], out["top_logprob"] = None, lp.sort(-1, descending=True).values[:, :c["top_k"]].contiguous()
    return out
