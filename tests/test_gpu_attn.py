"""Attention of drafted tokens over the paged cache, against the definition in 64 bits on the cache's own
stored values.

Bound on an output, with A = sum_j w_j |v_j| of its row and channel: the weights are rounded to bf16
(2^-8 of each), their exponents carry the scores' fp32 rounding (|s| error e = (d + 8) 2^-24 scale sum |q k|,
which moves w by at most 2 e relative with the sum), exp2 and the scale products a few ulp (2^-20), the sums
over n keys n 2^-24; the stored bf16 adds 2^-8 of the value."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import attn_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

FMT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


class Case:
    """Inputs of one call: a pool of garbage in which only the places the call may read hold values."""

    def __init__(self, fmt, d, n_kv, grp, page, ctx, T, *, tree=False, n_new=None, prefix=0, seed=0, spare=2, wide=None):
        rng = self.rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = self.B = len(ctx)
        self.fmt, self.d, self.n_kv, self.grp, self.T, self.page, self.prefix = fmt, d, n_kv, grp, T, page, prefix
        self.ctx = np.array(ctx, np.int32)
        self.n_new = None if n_new is None else np.array(n_new, np.int32)
        wide = wide or -(-(max(max(ctx), 0) + T) // page)
        shared = -(-prefix // page)
        n_pages = B * wide + shared + spare
        pool = rng.permutation(n_pages).astype(np.int32)
        self.shared, self.table = pool[:shared].copy(), pool[shared:shared + B * wide].reshape(B, wide).copy()
        es = 2 if fmt == "bf16" else 1
        shape = (n_pages, n_kv, page, d)
        self.store = {}
        for n in ("k", "v"):
            raw = torch.randint(0, 256, (*shape, es), dtype=torch.uint8, generator=g)  # NaNs and infinities among it
            raw[..., es - 1] |= torch.randint(0, 2, shape, dtype=torch.uint8, generator=g) * 0x7f
            self.store[n] = raw.view(FMT[fmt])[..., 0].contiguous()
            if fmt != "bf16":
                self.store[n + "_scale"] = torch.full(shape[:3], float("nan"))
        for b in range(B):
            if ctx[b] >= 0:
                self.fill(self.table[b], 0, ctx[b] + (T if n_new is None else max(0, min(T, n_new[b]))))
        self.fill(self.shared, 0, prefix)
        self.parent = None
        if tree:
            self.parent = np.full((B, T), -1, np.int32)
            for b in range(B):
                for t in range(1, T):
                    self.parent[b, t] = rng.integers(max(-1, t - 9), t)
        self.q = torch.from_numpy(rng.standard_normal((B * T, n_kv * grp, d)) * 2).to(torch.bfloat16)
        self.scale = d ** -0.5

    def at(self, pages, pos):
        return pages[pos // self.page].astype(int), pos % self.page

    def fill(self, pages, lo, hi):
        pos = np.arange(lo, min(hi, len(pages) * self.page))
        if not len(pos):
            return
        pg, place = self.at(pages, pos)
        for n in ("k", "v"):
            x = torch.from_numpy(self.rng.standard_normal((len(pos), self.n_kv, self.d)))
            if self.fmt == "bf16":
                self.store[n][pg, :, place] = x.to(torch.bfloat16)
                continue
            codes = (x * 100).clamp(-448, 448).to(FMT["e4m3"]) if self.fmt == "e4m3" else (x * 30).round().clamp(-127, 127).to(torch.int8)
            self.store[n].view(torch.uint8)[pg, :, place] = codes.view(torch.uint8)
            s = torch.from_numpy(self.rng.uniform(0.5, 1.5, (len(pos), self.n_kv))).float()
            self.store[n + "_scale"][pg, :, place] = s / (100 if self.fmt == "e4m3" else 30)

    def values(self, n, pages, pos, head):
        pg, place = self.at(pages, pos)
        x = self.store[n][pg, head, place].float().double().numpy()
        if self.fmt != "bf16":
            x = x * self.store[n + "_scale"][pg, head, place].double().numpy()[:, None]
        return x

    def upload(self):
        dev = {k: v.cuda() for k, v in self.store.items()}
        self.kv = gdn.KvCache(dev["k"], dev["v"], dev.get("k_scale"), dev.get("v_scale"))
        i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.g_table, self.g_ctx, self.g_new, self.g_parent = i32(self.table), i32(self.ctx), i32(self.n_new), i32(self.parent)
        self.g_pages = i32(self.shared) if self.prefix else None
        self.g_plen = i32(np.array([self.prefix], np.int32)) if self.prefix else None
        self.g_q = self.q.cuda()
        self.out = torch.full_like(self.g_q, 7.0)
        need = gdn.gdn_attn_workspace_bytes(self.kv, self.n_kv * self.grp, self.B, self.T, self.prefix > 0)
        assert need > 0
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")  # NaNs: nothing may be read unwritten
        return self

    def run(self, **kw):
        a = dict(q=self.g_q, out=self.out, workspace=self.ws)
        a.update(kw)
        gdn.gdn_attn_verify(self.kv, a["q"], self.g_table, self.g_ctx, self.g_new, self.g_parent, self.g_pages, self.g_plen,
                            a["out"], self.B, self.T, self.scale, a["workspace"], stream=a.get("stream"))
        return a["out"]

    def want(self, b):
        """(rows [T_live][heads][d], bound) of entry b."""
        T = self.T if self.n_new is None else min(self.T, int(self.n_new[b]))
        ctx = int(self.ctx[b])
        cap = self.table.shape[1] * self.page
        pos = np.arange(min(ctx + T, cap))
        ok = (self.table[b][pos // self.page] >= 0) & (self.table[b][pos // self.page] < len(self.store["k"]))
        draft = ref.sees(self.T, None if self.parent is None else self.parent[b])[:T, :T]
        sees = np.concatenate([np.ones((T, ctx), bool), draft], 1)[:, :len(pos)] & ok
        pre = np.arange(self.prefix)
        sees = np.concatenate([np.ones((T, self.prefix), bool), sees], 1).repeat(self.grp, 0)
        table = np.where((self.table[b] >= 0) & (self.table[b] < len(self.store["k"])), self.table[b], 0)
        out, tol = (np.zeros((T, self.n_kv * self.grp, self.d)) for _ in range(2))
        for h in range(self.n_kv):
            k, v = (np.concatenate([self.values(n, self.shared, pre, h), self.values(n, table, pos, h)]) for n in ("k", "v"))
            q = self.q.double().numpy().reshape(self.B, self.T, -1, self.d)[b, :T, h * self.grp:(h + 1) * self.grp].reshape(-1, self.d)
            o, w = ref.attend(q, k, v, sees, self.scale)
            kk, vv = np.where(np.isfinite(k), k, 0), np.where(np.isfinite(v), v, 0)
            e = (self.d + 8) * 2.0 ** -24 * self.scale * (np.abs(q) @ np.abs(kk).T).max()
            mass = w @ np.abs(vv)
            t = mass * (2.0 ** -8 + 2 * e + len(k) * 2.0 ** -24 + 2.0 ** -20)
            t = t + 2.0 ** -8 * (np.abs(o) + t)
            out[:, h * self.grp:(h + 1) * self.grp] = o.reshape(T, self.grp, self.d)
            tol[:, h * self.grp:(h + 1) * self.grp] = t.reshape(T, self.grp, self.d)
        return out, tol

    def check(self, out):
        got = out.double().cpu().numpy().reshape(self.B, self.T, -1, self.d)
        worst = 0.0
        for b in range(self.B):
            T = self.T if self.n_new is None else max(0, min(self.T, int(self.n_new[b])))
            if self.ctx[b] < 0:
                T = 0
            assert (got[b, T:] == 7.0).all(), f"entry {b}: rows that do not count were written"
            if not T:
                continue
            want, tol = self.want(b)
            same = np.isfinite(want)
            assert (np.isnan(got[b, :T]) == np.isnan(want)).all() and (got[b, :T][np.isinf(want)] == want[np.isinf(want)]).all(), b
            err = np.abs(got[b, :T][same] - want[same])
            assert np.isfinite(err).all() and (err <= tol[same]).all(), (b, float((err / tol[same]).max()))
            worst = max(worst, float((err / np.maximum(tol[same], 1e-300)).max()))
        return worst


SHAPES = {
    # n_kv, grp, page, ctx, T, keywords
    "one token, no context": (2, 8, 16, [0], 1, {}),
    "one token, one tile": (1, 1, 64, [37], 1, {}),
    "decode, ragged, tile edges": (2, 4, 64, [0, 62, 63, 64, 127, 128, 300], 1, {}),
    "decode, skipped entries": (1, 3, 32, [5, -1, 200, -7], 1, {}),
    "decode, many parts": (1, 2, 64, [9000], 1, {}),
    "chain of 16": (2, 4, 128, [0, 700, 64], 16, {}),
    "chain of 5, odd group": (3, 3, 16, [100, 31], 5, {}),
    "chain of 3, group of 7, ragged": (1, 7, 32, [40, 41, 0, 1], 3, dict(n_new=[3, 0, 1, 2])),
    "long chain": (1, 2, 64, [10, 130], 301, dict(n_new=[301, 77])),
    "tree of 64": (2, 4, 64, [90, 0, 63], 64, dict(tree=True)),
    "tree of 37, ragged": (1, 6, 16, [200, 3], 37, dict(tree=True, n_new=[37, 20])),
    "tree of 200": (1, 1, 64, [33], 200, dict(tree=True)),
    "prefix, decode": (2, 2, 64, [0, 100, 5], 1, dict(prefix=65)),
    "prefix of one, chain": (1, 4, 16, [20, 0], 6, dict(prefix=1)),
    "prefix, ragged chain, skipped entry": (2, 5, 32, [50, -1, 3, 0, 90], 9, dict(prefix=700, n_new=[9, 9, 0, 4, 1])),
    "prefix, tree": (1, 8, 128, [0, 77], 20, dict(prefix=513, tree=True)),
    "prefix, many rows": (1, 8, 64, [3] * 20, 2, dict(prefix=2000)),
}


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_matches_the_definition(shape, fmt, d):
    n_kv, grp, page, ctx, T, kw = SHAPES[shape]
    c = Case(fmt, d, n_kv, grp, page, ctx, T, seed=len(shape) + d, **kw).upload()
    say(f"{shape}, {fmt}, d {d}: {c.check(c.run()):.2f} of the bound")
    again = c.run(out=torch.full_like(c.out, 7.0))
    assert torch.equal(again, c.out)  # no sum depends on the order of anything


@pytest.mark.parametrize("fmt", list(FMT))
def test_hidden_values_do_not_leak(fmt):
    """Infinities and NaNs in drafted keys reach the rows that see them and no others."""
    c = Case(fmt, 128, 1, 3, 16, [30, 0], 24, tree=True, seed=4)
    for b, t, n, x in [(0, 3, "v", float("inf")), (0, 3, "k", float("nan")), (1, 7, "v", float("nan")),
                       (1, 7, "v", float("-inf")), (0, 20, "k", float("inf")), (1, 23, "v", float("inf"))]:
        pos = int(c.ctx[b]) + t
        pg, at = int(c.table[b][pos // 16]), pos % 16
        if fmt == "bf16":
            c.store[n][pg, 0, at, 5 if x > 0 else 9] = x
        elif fmt == "e4m3" and np.isnan(x):
            c.store[n].view(torch.uint8)[pg, 0, at, 17] = 0x7f
        else:
            c.store[n + "_scale"][pg, 0, at] = float("nan")
    c.upload()
    c.run()
    got = c.out.double().cpu().numpy().reshape(2, 24, 3, 128)
    for b in range(2):
        with np.errstate(all="ignore"):
            want, tol = c.want(b)
        clean = np.isfinite(want)
        assert clean.any() and not clean.all()
        assert (np.isfinite(got[b]) == clean).all(), b
        assert (np.abs(got[b] - want)[clean] <= tol[clean]).all()


@pytest.mark.parametrize("fmt", ["bf16", "i8"])
def test_places_that_do_not_exist(fmt):
    """Pages outside the pool and positions past the table are seen by no row; a row with no key is zero."""
    c = Case(fmt, 64, 2, 2, 16, [100, 40, 3], 4, seed=9, wide=4)  # entry 0 runs past its 64 places
    c.table[1][1] = -1
    c.table[1][2] = 10 ** 6
    c.table[2][0] = 99999
    c.upload()
    c.check(c.run())
    assert (c.out.view(3, 4, -1)[2] == 0).all()


def test_prefix_length_is_clamped_and_may_be_zero():
    c = Case("e4m3", 128, 2, 4, 64, [10, 5], 3, prefix=128, seed=3).upload()
    a = c.run().clone()
    c.g_plen.fill_(5000)  # two pages hold 128
    assert torch.equal(c.run(), a)
    c.g_plen.fill_(0)
    b = c.run().clone()
    c.prefix = 0
    c.check(b)
    c.g_plen.fill_(-3)
    assert torch.equal(c.run(), b)


def test_prefix_is_the_same_as_its_copy_in_every_table():
    """The shared form against the plain one over tables that all start with the prefix's pages: the same
    bound holds for both, so they differ by at most twice it."""
    c = Case("bf16", 128, 2, 4, 64, [70, 9, 200], 5, prefix=256, seed=8).upload()
    c.check(c.run())
    d = Case("bf16", 128, 2, 4, 64, [70, 9, 200], 5, prefix=256, seed=8)
    d.table = np.concatenate([np.broadcast_to(d.shared, (3, 4)), d.table], 1)
    d.ctx, d.prefix = d.ctx + 256, 0
    d.upload()
    d.check(d.run())


def test_strided_rows_and_long_offsets():
    """q and out inside fused rows; a pool whose rows pass 2^31 bytes."""
    c = Case("bf16", 256, 2, 2, 64, [130, 20], 3, seed=6)
    n = c.B * c.T
    c.upload()
    big = torch.zeros((40000, 2, 64, 256), dtype=torch.bfloat16, device="cuda")  # 2.6 GB
    v = torch.zeros_like(big)
    n_pages = c.kv.k.shape[0]
    big[-n_pages:], v[-n_pages:] = c.kv.k, c.kv.v
    c.g_table += 40000 - n_pages
    c.kv = gdn.KvCache(big, v)
    fused = torch.zeros((n, 12, 256), dtype=torch.bfloat16, device="cuda")
    fused[:, 4:8] = c.g_q
    out = torch.full((4, n, 256), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    c.check(c.run(q=fused[:, 4:8], out=out).contiguous())


def test_replays_in_a_graph_with_other_lengths():
    c = Case("e4m3", 128, 2, 4, 64, [300, 20, 0], 4, prefix=200, seed=12).upload()
    c.run()
    out = torch.full_like(c.out, 7.0)
    ws = torch.full_like(c.ws, 0xff)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, workspace=ws)
    for ctx in ([300, 20, 0], [5, 290, 100], [0, 0, 0], [120, -1, 200]):
        c.g_ctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        for t in (out, c.out):
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.run()
        assert torch.equal(torch.nan_to_num(out.float(), nan=-5), torch.nan_to_num(c.out.float(), nan=-5)), ctx


def test_two_streams_with_a_workspace_each():
    cs = [Case("i8", 128, 4, 2, 64, [2000 + i, 5], 8, seed=20 + i).upload() for i in range(2)]
    want = [c.run().clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c, s in zip(cs, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c.out, w)


def test_index_check_refuses():
    c = Case("i8", 64, 1, 2, 16, [20, 3], 4, prefix=20, tree=True, seed=2).upload()
    c.kv.c.flags = gdn.GDN_F_CHECK_INDICES
    c.run()
    done = c.out.clone()
    def refused():
        with pytest.raises(gdn.GdnError) as e:
            c.run()
        assert e.value.code == gdn.GDN_ERR_RANGE
    for t, at, x in ((c.g_table, (0, 0), 10 ** 6), (c.g_ctx, (1,), -1), (c.g_ctx, (0,), 10 ** 6), (c.g_parent, (0, 2), 2),
                     (c.g_parent, (1, 0), 0), (c.g_plen, (0,), 33), (c.g_pages, (1,), -1)):
        was = t[at].clone()
        t[at] = x
        refused()
        t[at] = was
    assert torch.equal(c.run(), done)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("fmt", list(FMT))
def test_runs_longer_than_the_table_entries_at_hand(fmt, d):
    """Contexts of 1250 pages, so many entries that a workgroup's run of key tiles crosses several hundred table
    entries.  All entries name the same pages and ask the same."""
    c = Case(fmt, d, 2, 1, 16, [20000], 1, seed=d).upload()
    want, tol = c.want(0)
    n = c.B = 96
    c.g_table, c.g_ctx = c.g_table.repeat(n, 1), c.g_ctx.repeat(n)
    c.g_q, c.out = c.g_q.repeat(n, 1, 1), torch.full((n, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    c.ws = torch.full((gdn.gdn_attn_workspace_bytes(c.kv, 2, n, 1, False),), 0xff, dtype=torch.uint8, device="cuda")
    got = c.run().double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("shape", ["wide group", "more entries than threads", "more entries than threads, prefix",
                                   "prefix of more rows than a tile", "largest page, odd context"])
def test_sizes_at_the_edges(shape, fmt):
    n_kv, grp, page, ctx, T, kw = {
        "wide group": (1, 130, 16, [5, 100], 1, {}),
        "more entries than threads": (1, 2, 16, [(7 * i) % 90 - 3 for i in range(700)], 1, {}),
        "more entries than threads, prefix": (2, 1, 16, [(11 * i) % 40 for i in range(300)], 2,
                                              dict(prefix=50, n_new=[i % 4 for i in range(300)])),
        "prefix of more rows than a tile": (1, 4, 64, [(5 * i) % 70 for i in range(40)], 7, dict(prefix=130, tree=True)),
        "largest page, odd context": (2, 2, 4096, [4095, 4096, 1], 3, {}),
    }[shape]
    c = Case(fmt, 128, n_kv, grp, page, ctx, T, seed=len(shape), **kw).upload()
    say(f"{shape}, {fmt}: {c.check(c.run()):.2f} of the bound")


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("small", [0.0, 1e-42, 3e-39, 1e-20])
def test_very_small_scales(fmt, small):
    """v scales far below the others', down to subnormal ones, for some keys and for all: below 2^-64 they count as
    2^-64, which moves a row of at most 448 by 448 2^-64 at most; nothing becomes infinite or NaN."""
    for every in (3, 1):
        c = Case(fmt, 128, 2, 4, 16, [100, 40], 3, seed=17)
        c.store["v_scale"][:, :, ::every] = small
        c.store["k_scale"][:, :, 1::5] = small
        c.store["v"].view(torch.uint8)[:, :, ::every] &= 0xff if small else 0
        c.upload()
        got = c.run().double().cpu().numpy().reshape(2, 3, 8, 128)
        for b in range(2):
            want, tol = c.want(b)
            assert (np.abs(got[b] - want) <= tol + 448 * 2.0 ** -64).all(), (every, b)


def test_output_in_place_of_q():
    c = Case("bf16", 128, 2, 4, 16, [100, 40, 3000], 3, seed=5).upload()
    want = c.run().clone()
    q = c.g_q.clone()
    assert torch.equal(c.run(q=q, out=q), want)


@pytest.mark.parametrize("slope", [2.0, 7.0, 25.0, -7.0])
@pytest.mark.parametrize("fmt", list(FMT))
def test_scores_that_keep_growing(fmt, slope):
    """Scores that rise (or fall) by a steady amount per 64 keys, in powers of two, below and above what the running
    maximum is let grow by before the sums are rescaled."""
    c = Case(fmt, 128, 1, 4, 64, [1500, 700], 4, seed=31, prefix=650)
    u = torch.from_numpy(np.sign(c.rng.standard_normal(128)))
    for pages, n in ((c.shared, 650), (c.table[0], 1504), (c.table[1], 704)):
        pos = np.arange(n)
        pg, at = c.at(pages, pos)
        up = torch.from_numpy(pos if slope > 0 else n - pos) * (abs(slope) / 64 * np.log(2) / 128 ** 0.5)  # times u . u = 128
        if fmt == "bf16":
            c.store["k"][pg, 0, at] = (up[:, None] * u).to(torch.bfloat16)
        else:
            c.store["k"].view(torch.uint8)[pg, 0, at] = (u * 3).to(FMT[fmt]).view(torch.uint8)
            c.store["k_scale"][pg, 0, at] = (up / 3).float()
    c.q = (u + torch.from_numpy(c.rng.standard_normal((8, 4, 128)) * 0.01)).to(torch.bfloat16)
    c.upload()
    say(f"slope {slope}, {fmt}: {c.check(c.run()):.2f} of the bound")
