"""Plain references in 64 bits of the full-attention layers' operators, on the CPU in numpy: rotary
positions, the quantised paged cache, attention of a drafted chain or tree.  Written from the
definitions in include/gdn.h; they share nothing with the library."""

import math

import numpy as np


def frequencies(rot, theta, scaling="plain", factor=1.0, orig_ctx=0, fast=32.0, slow=1.0, mscale=0.0):
    """(frequency of every pair, factor on cos and sin)."""
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        def pair_turning(n):
            return rot * math.log(orig_ctx / (n * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair_turning(fast)), 0), min(math.ceil(pair_turning(slow)), rot - 1)
        for i in range(rot // 2):
            r = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f[i] = f[i] / factor * r + f[i] * (1 - r)
        return f, mscale or 0.1 * math.log(factor) + 1
    return f, mscale or 1.0


def rotate(x, positions, rot, f, m=1.0, layout="half", sections=None, inverse=False):
    """x [n][heads][d] fp64; positions [axes][n] ints."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    axis = np.zeros(rot // 2, int)
    if sections:
        axis = np.repeat(np.arange(4), sections)
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        ang = np.array([math.fmod(int(p) * f[i], 2 * math.pi) for p in positions[axis[i]]]) * (-1 if inverse else 1)
        c, s = (m * np.cos(ang))[:, None], (m * np.sin(ang))[:, None]
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return out


def sees(n_tok, parent=None):
    """[n_tok][n_tok] bool: token t sees drafted token j."""
    m = np.zeros((n_tok, n_tok), bool)
    for t in range(n_tok):
        p = t - 1 if parent is None else int(parent[t])
        if 0 <= p < t:
            m[t] = m[p]
        m[t, t] = True
    return m


def attend(q, k, v, mask, scale):
    """q [rows][d], k and v [keys][d] fp64, mask [rows][keys] -> (out [rows][d], weights)."""
    with np.errstate(all="ignore"):
        s = np.where(mask, q @ k.T * scale, -np.inf)
        any_key = mask.any(1)
        top = np.where(any_key, np.max(s, axis=1, initial=-np.inf), 0.0)
        w = np.where(mask, np.exp(s - top[:, None]), 0.0)
        w = w / np.where(any_key, w.sum(1), 1.0)[:, None]
        # a key that a row does not see does not reach it, whatever its v holds
        out = np.stack([wr[mr] @ v[mr] if mr.any() else np.zeros(v.shape[1]) for wr, mr in zip(w, mask)])
    return out, w
