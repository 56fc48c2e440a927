"""Attention over the paged cache where single keys differ from the rest: a key that draws most of the attention
and has nothing in v, or nothing but one channel; values that are not finite.  Held to the definition in 64 bits,
with the bound of the attention tests or with the one below that takes each cache format for what its weights are
rounded to."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import attn_ref as ref
from tests.gpu_util import say
from tests.test_gpu_attn import FMT, Case

pytestmark = pytest.mark.gpu

class Fine(Case):
    """A case whose bound counts the rounding of the weights w by the cache's format: in a bf16 cache 2^-8 of each, in the
    8-bit formats 2^-11 of w_j vs_j (fp16, half a step) or, where fp16 has no full precision, half of its smallest
    step 2^-24 where the row's largest w vs is taken as 2^7 or more, 2^-32 of that largest one, times |code|."""

    def weight_error(self, b):
        return 2.0 ** -8 if self.fmt == "bf16" else 2.0 ** -11

    def want(self, b):
        out, tol = super().want(b)
        T, ctx = len(out), int(self.ctx[b])
        draft = ref.sees(self.T, None if self.parent is None else self.parent[b])[:T, :T]
        sees = np.concatenate([np.ones((T, self.prefix + ctx), bool), draft], 1).repeat(self.grp, 0)
        pre, pos = np.arange(self.prefix), np.arange(ctx + T)
        for h in range(self.n_kv):
            at = slice(h * self.grp, (h + 1) * self.grp)
            k, v = (np.concatenate([self.values(n, self.shared, pre, h), self.values(n, self.table[b], pos, h)]) for n in ("k", "v"))
            q = self.q.double().numpy().reshape(self.B, self.T, -1, self.d)[b, :T, at].reshape(-1, self.d)
            _, w = ref.attend(q, k, v, sees, self.scale)
            e = (self.d + 8) * 2.0 ** -24 * self.scale * (np.abs(q) @ np.abs(k).T).max()
            t = (w @ np.abs(v)) * (self.weight_error(b) + 2 * e + len(k) * 2.0 ** -24 + 2.0 ** -20)
            if self.fmt != "bf16":
                vs = np.concatenate([self.scales(self.shared, pre, h), self.scales(self.table[b], pos, h)])
                codes = np.abs(v) / np.where(vs > 0, vs, 1.0)[:, None]
                t = t + 2.0 ** -32 * (w * vs).max(1, keepdims=True) * (sees @ codes)
            o = out[:, at].reshape(-1, self.d)
            tol[:, at] = (t + 2.0 ** -8 * (np.abs(o) + t)).reshape(T, self.grp, self.d)
        return out, tol

    def scales(self, pages, pos, head):
        pg, place = self.at(pages, pos)
        return self.store["v_scale"][pg, head, place].double().numpy()


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


def sink_case(rows, fmt, d, share=0.9, size=1.0, seed=0, kind=Case):
    """A case whose rows all give about ``share`` of their weight to one early key (of the prefix, or of every entry's
    context); its place is c.sinks, a list of (page, place).  v is ``size`` times a normal value."""
    n_kv, grp, ctx, T, prefix = ROWS[rows]
    c = kind(fmt, d, n_kv, grp, 16, ctx, T, prefix=prefix, seed=seed + d)
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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("rows", list(ROWS))
def test_a_strong_key_with_one_channel(rows, fmt, d):
    """All but a thousandth of the weight goes to a key whose v holds its first channel alone.  The other channels are
    the rest's, whose weights are about 2^-22 of the largest (fp16 gives those steps of 2^-24)."""
    c = sink_case(rows, fmt, d, share=0.999, kind=Fine)
    for pg, at in c.sinks:
        codes = c.store["v"].view(torch.uint8).view(*c.store["v"].shape, -1)
        codes[pg, :, at, 1:] = 0
    c.upload()
    say(f"{rows}, {fmt}, d {d}: {c.check(c.run()):.2f} of the bound")


@pytest.mark.parametrize("grp,T", [(2, 8), (4, 16), (4, 20), (8, 32)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_values_that_are_not_finite_in_every_first_tile(fmt, grp, T):
    """Entries whose only tile holds drafted keys, one of them with a v that is not finite: every entry's rows that see
    it have it in their result, in every one of several runs (16, 64, 80 and 256 rows share keys)."""
    n = 48
    c = Case(fmt, 128, 2, grp, 64, [(7 * i) % 20 for i in range(n)], T, seed=T)
    for b in range(n):
        pos = int(c.ctx[b]) + b % T
        pg, at = int(c.table[b][pos // 64]), pos % 64
        if fmt == "bf16":
            c.store["v"][pg, b % 2, at, 7 * b % 128] = float("inf") if b % 3 else float("nan")
        elif fmt == "e4m3" and b % 3:
            c.store["v"].view(torch.uint8)[pg, b % 2, at, 7 * b % 128] = 0x7f
        else:
            c.store["v_scale"][pg, b % 2, at] = float("nan")
    c.upload()
    with np.errstate(all="ignore"):
        c.check(c.run())
    first = torch.nan_to_num(c.out.float(), nan=-5.0)
    for _ in range(5):
        again = c.run(out=torch.full_like(c.out, 7.0))
        assert torch.equal(torch.nan_to_num(again.float(), nan=-5.0), first)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("grp,T,prefix", [(1, 1, 0), (4, 8, 0), (4, 16, 0), (8, 16, 0), (8, 32, 0), (2, 2, 300), (8, 24, 300)])
def test_values_that_are_not_finite_in_the_context(grp, T, prefix, fmt, d):
    """Infinities and a NaN in v of cached keys that every row sees, in a prefix too: each in its channel, with its
    sign, however the weights are split for the product."""
    c = Case(fmt, d, 1, grp, 16, [200, 90], T, prefix=prefix, seed=3)
    for pages in ([c.shared] if prefix else []) + [c.table[0]]:
        for pos, ch, x in ((5, 3, float("inf")), (70, 9, float("-inf")), (71, 11, float("nan"))):
            pg, at = int(pages[pos // 16]), pos % 16
            if fmt == "bf16":
                c.store["v"][pg, 0, at, ch] = x
            else:  # NaN is all that e4m3 has
                c.store["v"].view(torch.uint8)[pg, 0, at, ch] = 0x7f
    c.upload()
    with np.errstate(all="ignore"):
        say(f"{c.check(c.run()):.2f} of the bound")


def test_index_check_refuses_paths_of_nodes_that_do_not_count():
    """gdn_kv_commit moves no row of a token at or past n_new; under GDN_F_CHECK_INDICES a path that names one is refused."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randint(-127, 128, (4, 1, 16, 64), dtype=torch.int8, device="cuda") for _ in range(2))
    kv = gdn.KvCache(k, v, *(torch.ones(4, 1, 16, device="cuda") for _ in range(2)))
    kv.c.flags = gdn.GDN_F_CHECK_INDICES
    table, start, path, before = i32([[0, 1], [2, 3]]), i32([10, 3]), i32([[1, 4], [0, 2]]), k.clone()
    def commit(n_new):
        gdn.gdn_kv_commit(kv, table, start, path, i32([2, 2]), 2, 6, n_new=None if n_new is None else i32(n_new))
    for n_new in ([4, 6], [6, 2], [5, 0]):
        with pytest.raises(gdn.GdnError) as e:
            commit(n_new)
        assert e.value.code == gdn.GDN_ERR_RANGE and torch.equal(k, before)
    commit([5, 3])
    assert torch.equal(k[0, 0, 10], before[0, 0, 11]) and torch.equal(k[0, 0, 11], before[0, 0, 14])
    assert torch.equal(k[2, 0, 4], before[2, 0, 5])
    k.copy_(before)
    commit(None)
    assert not torch.equal(k, before)


def test_workspace_must_be_memory_of_its_size():
    """A tensor expanded to the bytes that are needed, and a strided one, are refused before anything is launched."""
    c = Case("bf16", 64, 1, 1, 16, [20], 1, seed=1).upload()
    need = c.ws.numel()
    for ws in (torch.zeros(16, dtype=torch.uint8, device="cuda")[:1].expand(need),
               torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(gdn.GdnError) as e:
            c.run(workspace=ws)
        assert e.value.code == gdn.GDN_ERR_ARG
    assert (c.out == 7.0).all()
