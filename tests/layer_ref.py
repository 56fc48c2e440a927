"""Plain 64-bit forms of the norm, the product with its epilogue and the log probabilities, in numpy, from their formulas."""

import math

import numpy as np

FULL = {"e4m3": 448.0, "i8": 127.0}
U32 = 2.0 ** -24          # half a step of fp32, relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def norm(x, weight=None, residual=None, eps=1e-6, rms=True):
    """(s, y) of rows [..., d]."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    y = s
    with np.errstate(invalid="ignore", over="ignore"):
        if rms:
            y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
        return s, y if weight is None else y * np.asarray(weight, np.float64)


def activate(name, v):
    with np.errstate(over="ignore"):
        if name == "silu":
            return v / (1 + np.exp(-v))
        if name == "gelu":
            return 0.5 * v * np.vectorize(lambda t: math.erfc(-t / math.sqrt(2)), otypes=[float])(v)
        if name == "gelu_tanh":
            return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
        if name == "relu":
            return np.maximum(v, 0)
        if name == "sigmoid":
            return 1 / (1 + np.exp(-v))
    return v


def linear(x, w, x_scale=None, w_scale=None, bias=None, act="none", gated=False, residual=None):
    """(out, bound): the result and how far fp32 arithmetic of the epilogue and the sums may take it, before the last
    rounding.  A sum of K products is off by at most K + 2 half steps of the sum of their sizes, whatever the order; where
    the operands are whole numbers whose sums stay below 2^24, by none (the caller subtracts that part)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    k, n = x.shape[1], w.shape[0] // (2 if gated else 1)
    p, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if x_scale is not None:
        f = np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)
        p, size = p * f, size * np.abs(f)
    sums = (k + 2) * U32 * size
    near = 4 * U32 * np.abs(p)
    if bias is not None:
        p = p + np.asarray(bias, np.float64)
        near = near + U32 * np.abs(p)

    def through(name, v):
        # slope at most 1.2; the exponential's argument is rounded (|v| + 1 half steps of the factor next to v), gelu's
        # 1 + erf by a step of 1, each a few times
        y = activate(name, v)
        more = 0 if name == "none" else 8 * U32 * (np.abs(y) * (1 + 2 * np.abs(v)) + (np.abs(v) if name == "gelu" else 0))
        if name == "gelu_tanh":  # its argument is a cube
            more = more + 8 * U32 * np.abs(y) * np.abs(v) ** 3
        return y, more

    if gated:
        y, more = through(act, p[:, :n])
        up = p[:, n:]
        sums = 1.2 * sums[:, :n] * np.abs(up) + sums[:, n:] * np.abs(y)
        near = 1.2 * near[:, :n] * np.abs(up) + near[:, n:] * np.abs(y) + more * np.abs(up)
        y = y * up
        near = near + U32 * np.abs(y)
    else:
        y, more = through(act, p)
        sums, near = 1.2 * sums, 1.2 * near + more
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
        near = near + U32 * np.abs(y)
    return y, sums, near


def order(row):
    """Indices of a row in the order of the alternatives: larger first, of equal ones the lower index, NaN as -infinity."""
    r = np.where(np.isnan(row), -np.inf, np.asarray(row, np.float64)) + 0.0
    return np.lexsort((np.arange(len(r)), -r))


def logprob(logits, ids=None, temperature=1.0, top_k=0):
    """{"lse", "entropy", "logprob", "rank", "top_ids", "top_logprob"} of rows of logits."""
    l = np.asarray(logits, np.float64) / temperature
    n, v = l.shape
    out = {k: np.full(n, np.nan) for k in ("lse", "entropy")}
    m = 0 if ids is None else ids.shape[1]
    out.update(logprob=np.full((n, m), -np.inf), rank=np.full((n, m), -1), top_ids=np.zeros((n, top_k), int),
               top_logprob=np.zeros((n, top_k)))
    for r in range(n):
        o = order(l[r])
        place = np.empty(v, int)
        place[o] = np.arange(v)
        if np.isnan(l[r]).any() or (l[r] == np.inf).any():
            lp = np.full(v, np.nan)
        elif (l[r] == -np.inf).all():
            out["lse"][r], out["entropy"][r] = -np.inf, 0.0
            lp = np.full(v, -np.inf)
        else:
            top = l[r].max()
            logs = np.log(np.exp(l[r] - top).sum())
            lp = (l[r] - top) - logs  # not l - lse: beside a maximum of 10^38 log s would be lost even in 64 bits
            p, z = np.exp(lp), top + logs
            out["lse"][r], out["entropy"][r] = z, -(p[p > 0] * lp[p > 0]).sum()
        for i in range(m):
            if 0 <= ids[r, i] < v:
                out["logprob"][r, i], out["rank"][r, i] = lp[ids[r, i]], place[ids[r, i]]
        out["top_ids"][r], out["top_logprob"][r] = o[:top_k], lp[o[:top_k]]
    return out
