"""Attention over the paged cache where single keys differ from the rest: a key that draws most of the attention
and has nothing in v.  Held to the definition in 64 bits with the bound of the attention tests."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests.gpu_util import say
from tests.test_gpu_attn import FMT, Case

pytestmark = pytest.mark.gpu

# rows that share keys: n_kv, grp, contexts, tokens of an entry, prefix
ROWS = {
    "one row": (2, 1, [4000, 1500], 1, 0),
    "rows of 32": (1, 4, [4000, 30], 8, 0),
    "rows of 64": (1, 4, [3000], 16, 0),
    "rows of 128": (1, 8, [3000], 16, 0),
    "rows of 256": (1, 8, [2500], 32, 0),
    "prefix, few rows": (2, 2, [20, 700], 2, 3000),
    "prefix, many rows": (1, 4, [40, 0, 300], 24, 2500),
}


def sink_case(rows, fmt, d, share=0.9, size=1.0, seed=0):
    """A case whose rows all give about ``share`` of their weight to one early key (of the prefix, or of every entry's
    context); its place is c.sinks, a list of (page, place).  v is ``size`` times a normal value."""
    n_kv, grp, ctx, T, prefix = ROWS[rows]
    c = Case(fmt, d, n_kv, grp, 16, ctx, T, prefix=prefix, seed=seed + d)
    u = torch.from_numpy(np.sign(c.rng.standard_normal(d)))
    c.q = (u + torch.from_numpy(c.rng.standard_normal((c.B * T, n_kv * grp, d)))).to(torch.bfloat16)
    # scores of the others are normal with variance |q|^2 / d = 2: their weights add up to about n e
    n = (prefix or max(ctx))
    score = np.log(n) + 1.0 + np.log(share / (1 - share))
    up = score / d ** 0.5  # k = up u: q . k d^-1/2 = up d^1/2 (1 + u . noise / d)
    runs = [c.shared] if prefix else [t for t, x in zip(c.table, ctx) if x > 3]
    c.sinks = [(int(pages[0]), 3) for pages in runs]
    if fmt == "bf16":
        c.store["v"] = (c.store["v"].float() * size).to(torch.bfloat16)
    else:
        c.store["v_scale"] *= size
    for pg, at in c.sinks:
        if fmt == "bf16":
            c.store["k"][pg, :, at] = (up * u).to(torch.bfloat16)
        else:
            c.store["k"].view(torch.uint8)[pg, :, at] = (u * 3).to(FMT[fmt]).view(torch.uint8)
            c.store["k_scale"][pg, :, at] = up / 3
    return c


def no_value(c):
    """The sinks' v as the cache holds a row of zeros."""
    for pg, at in c.sinks:
        c.store["v"].view(torch.uint8).view(*c.store["v"].shape[:3], -1)[pg, :, at] = 0
        if c.fmt != "bf16":
            c.store["v_scale"][pg, :, at] = 0.0


@pytest.mark.parametrize("size", [1.0, 0.05])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("rows", list(ROWS))
def test_a_strong_key_without_a_value(rows, fmt, d, size):
    """Nine tenths of the weight go to a key whose v is zero: what is left is the others' sum, a tenth as large."""
    c = sink_case(rows, fmt, d, size=size)
    no_value(c)
    c.upload()
    say(f"{rows}, {fmt}, d {d}, v of {size}: {c.check(c.run()):.2f} of the bound")


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_a_strong_key_written_as_zeros(fmt):
    """The same with the row of zeros put into the cache by gdn_kv_write."""
    c = sink_case("rows of 32", fmt, 128, share=0.99, size=0.05)
    c.upload()
    k = c.kv.k[[s[0] for s in c.sinks], :, 3].float() * c.kv.k_scale[[s[0] for s in c.sinks], :, 3][..., None]
    n = len(c.sinks)
    gdn.gdn_kv_write(c.kv, k, torch.zeros_like(k), c.g_table[:n].contiguous(),
                     torch.full((n,), 3, dtype=torch.int32, device="cuda"), None, n, 1)
    for name in c.store:
        c.store[name] = getattr(c.kv, name).cpu()
    assert all((c.store["v_scale"][pg, :, at] == 0).all() for pg, at in c.sinks)
    say(f"{fmt}: {c.check(c.run()):.2f} of the bound")
