"""The paged KV cache through the C ABI.

Without a rotation codes, scales and values are exact: the same IEEE operations in fp32 give the same
bits on the CPU.  With one, a value may differ from the 64-bit one by the rotation's own error before it
is rounded, so it is held to that plus half a step of its format (bf16 2^-8 of the value, e4m3 2^-4 of it
or 2^-10 scales below the normal range, i8 half a scale), the scale to 2^-23 beside the rotation's error."""

import numpy as np
import pytest
import torch

from gated_deltanet_linear_verify_amd import gdn
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu

FMT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
FULL = {"e4m3": 448.0, "i8": 127.0}
ROPE = 6.1e-7  # of |x_a| + |x_b|, see the rotary tests


def make(fmt, n_pages, n_kv, page, d, fill=None):
    g = torch.Generator().manual_seed(1)
    shape = (n_pages, n_kv, page, d)
    def codes():
        return torch.randint(0, 256, (*shape, 2 if fmt == "bf16" else 1), dtype=torch.uint8, generator=g).view(FMT[fmt])[..., 0].contiguous().cuda()
    sc = [] if fmt == "bf16" else [torch.rand(shape[:3], generator=g).cuda() for _ in range(2)]
    return gdn.KvCache(codes(), codes(), *sc)


def raw(t):
    return t.contiguous().view(torch.uint8)


def places(table, start, n_new, page, n_tok):
    """(entry, token, page, place) of every token that counts."""
    out = []
    for b in range(len(start)):
        for t in range(min(n_new[b], n_tok)):
            p = int(start[b]) + t
            if start[b] >= 0 and p // page < table.shape[1]:
                out.append((b, t, int(table[b, p // page]), p % page))
    return out


def quantise(x, fmt):
    """CPU, fp32: (codes, scales) of rows x [..., d]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1)
    scale = top / torch.tensor([FULL[fmt]])
    inv = torch.ones(1) / scale
    dead = ~torch.isfinite(inv)
    bad = ~torch.isfinite(x).all(-1)
    scale = torch.where(dead, torch.zeros(()), scale)
    inv = torch.where(dead | bad, torch.zeros(()), inv)
    y = torch.where((dead | bad)[..., None], torch.zeros(()), x * inv[..., None])
    scale = torch.where(bad, torch.full((), float("nan")), scale)
    codes = y.to(FMT[fmt]) if fmt == "e4m3" else y.round().clamp(-127, 127).to(torch.int8)
    return codes, scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("B,T,n_kv,d,page,ragged", [
    (1, 1, 1, 64, 16, False), (3, 5, 2, 128, 16, True), (2, 70, 3, 256, 64, True), (5, 1, 8, 128, 4096, False),
    (4, 3001, 2, 64, 32, False),
])
def test_write_and_read_are_exact(B, T, n_kv, d, page, ragged, fmt, dtype):
    rng = np.random.default_rng(B * T + d)
    wide = -(-(200 + T) // page)
    table = rng.permutation(B * wide + 2)[:B * wide].reshape(B, wide).astype(np.int32)
    start = rng.integers(0, 200, B).astype(np.int32)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if ragged else np.full(B, T, np.int32)
    kv = make(fmt, B * wide + 2, n_kv, page, d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows = torch.from_numpy(rng.standard_normal((B * T, 2 * n_kv, d)) * np.exp(rng.normal(0, 2, (B * T, 1, 1)))).to(dt)
    rows[0, 0] = 0.0  # a row of zeros
    rows[-1, 1 % (2 * n_kv), 3] = float("inf")
    rows[-1, -1, d - 1] = float("nan")
    if dtype == "f32" and B > 1:
        rows[T, 0] = 1e-42  # 1 / scale overflows
    dev = rows.cuda()
    dt_, ds, dn = (torch.from_numpy(a).cuda() for a in (table, start, n_new))
    before = [None if t is None else t.clone() for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]
    gdn.gdn_kv_write(kv, dev[:, :n_kv], dev[:, n_kv:], dt_, ds, dn if ragged else None, B, T)
    where = places(table, start, n_new, page, T)
    pg, at = [w[2] for w in where], [w[3] for w in where]
    src = [w[0] * T + w[1] for w in where]
    for i, (half, n) in enumerate(((rows[:, :n_kv], "k"), (rows[:, n_kv:], "v"))):
        codes, scale = quantise(half[src].float(), fmt)
        want = before[i].cpu()
        raw(want).view(want.shape[0], n_kv, page, -1)[pg, :, at] = raw(codes).view(len(where), n_kv, -1)
        got = getattr(kv, n).cpu()
        if fmt == "bf16":
            assert torch.equal(torch.nan_to_num(got.float(), nan=7e30), torch.nan_to_num(want.float(), nan=7e30))
        else:
            assert torch.equal(raw(got), raw(want))
            ws = before[2 + i].cpu()
            ws[pg, :, at] = scale
            assert torch.equal(torch.nan_to_num(getattr(kv, n + "_scale").cpu(), nan=-1), torch.nan_to_num(ws, nan=-1))
    for dt in (torch.bfloat16, torch.float32):
        out = [torch.full((B * T, n_kv, d), -3.0, dtype=dt, device="cuda") for _ in range(2)]
        gdn.gdn_kv_read(kv, dt_, ds, dn if ragged else None, *out, B, T)
        for o, n in zip(out, ("k", "v")):
            want = torch.full((B * T, n_kv, d), -3.0)
            val = getattr(kv, n).cpu()[pg, :, at].float()
            if fmt != "bf16":
                val = val * getattr(kv, n + "_scale").cpu()[pg, :, at][..., None]
            want[src] = val
            assert torch.equal(torch.nan_to_num(o.cpu().float(), nan=7e30), torch.nan_to_num(want.to(dt).float(), nan=7e30))


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("layout,rot,d,sections", [
    ("half", 64, 256, (11, 11, 10, 0)), ("half", 62, 64, None), ("interleaved", 128, 128, None),
    ("interleaved", 36, 64, None), ("half", 128, 128, None), ("half", 12, 128, None),
])
def test_write_rotates(layout, rot, d, sections, fmt):
    rng = np.random.default_rng(rot)
    B, T, n_kv, page = 3, 9, 2, 16
    table = rng.permutation(B * 4).reshape(B, 4).astype(np.int32)
    start = np.array([0, 15, 40], np.int32)
    kv = make(fmt, B * 4, n_kv, page, d)
    x = torch.from_numpy(rng.standard_normal((B * T, 2 * n_kv, d))).to(torch.bfloat16).cuda()
    pos = rng.integers(0, 300000, (4 if sections else 1, B * T)).astype(np.int32)
    lay = gdn.GDN_ROPE_HALF if layout == "half" else gdn.GDN_ROPE_INTERLEAVED
    gdn.gdn_kv_write(kv, x[:, :n_kv], x[:, n_kv:], torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(), None, B, T,
                     rope=gdn.gdn_rope_init(rot, theta=1e6, layout=lay, sections=sections), positions=torch.from_numpy(pos).cuda())
    f, _ = ref.frequencies(rot, 1e6)
    xd = x.double().cpu().numpy()
    want = {"k": ref.rotate(xd[:, :n_kv], pos, rot, f, layout=layout, sections=sections), "v": xd[:, n_kv:]}
    slack = {"k": ROPE * 2 * np.abs(xd[:, :n_kv]).max(), "v": 0.0}
    for b, t, pg, at in places(table, start, np.full(B, T), page, T):
        for n in ("k", "v"):
            got = getattr(kv, n)[pg, :, at].float().cpu().double().numpy()
            w = want[n][b * T + t]
            if fmt == "bf16":
                assert (np.abs(got - w) <= slack[n] + 2.0 ** -8 * (np.abs(w) + slack[n])).all()
                continue
            sc = getattr(kv, n + "_scale")[pg, :, at].cpu().double().numpy()[:, None]
            exact = np.abs(w).max(-1, keepdims=True) / FULL[fmt]
            assert (np.abs(sc - exact) <= slack[n] / FULL[fmt] + 2.0 ** -23 * exact).all()
            # x (1 / s) rounds twice more before the code, each 2^-24 of x
            half = 0.5 * sc if fmt == "i8" else np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10 * sc)
            assert (np.abs(got * sc - w) <= (half + slack[n]) * (1 + 2.0 ** -4) + 2.0 ** -22 * np.abs(w)).all()


@pytest.mark.parametrize("fmt", list(FMT))
def test_places_outside_are_left_alone(fmt):
    """Skipped entries, positions past the table and pages outside the pool: nothing is written or read."""
    B, T, n_kv, d, page = 4, 40, 2, 64, 16
    kv = make(fmt, 6, n_kv, page, d)
    table = torch.tensor([[0, 1], [2, -1], [6, 3], [4, 5]], dtype=torch.int32).cuda()
    start = torch.tensor([-1, 0, 0, 20], dtype=torch.int32).cuda()
    n_new = torch.tensor([40, 100, 40, -3], dtype=torch.int32).cuda()
    rows = torch.randn(B * T, n_kv, d, device="cuda")
    before = [None if t is None else t.clone() for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]
    gdn.gdn_kv_write(kv, rows, rows, table, start, n_new, B, T)
    for t, was in zip((kv.k, kv.v, kv.k_scale, kv.v_scale), before):
        if t is not None:
            for pg in (0, 1, 4, 5):
                assert torch.equal(raw(t[pg]), raw(was[pg]))
            assert not torch.equal(raw(t[2]), raw(was[2])) and not torch.equal(raw(t[3]), raw(was[3]))
    out = torch.full((B * T, n_kv, d), -3.0, device="cuda")
    gdn.gdn_kv_read(kv, table, start, n_new, out, out.clone(), B, T)
    read = (out.view(B, T, -1) != -3.0).any(-1).cpu()
    want = torch.zeros(B, T, dtype=torch.bool)
    want[1, :16] = True  # its second page is -1
    want[2, 16:32] = True  # its first page is past the pool
    assert torch.equal(read, want)


@pytest.mark.parametrize("fmt", list(FMT))
def test_commit_moves_the_path(fmt):
    rng = np.random.default_rng(2)
    B, T, n_kv, d, page = 4, 40, 3, 256, 16
    kv = make(fmt, B * 5, n_kv, page, d)
    table = rng.permutation(B * 5).reshape(B, 5).astype(np.int32)
    start = np.array([0, 13, 37, -1], np.int32)
    path = np.full((B, 20), 99, np.int32)
    n_path = np.array([20, 5, 0, 3], np.int32)
    path[0] = np.sort(rng.permutation(T)[:20])
    path[1, :5] = [0, 1, 7, 8, 39]
    path[3, :3] = [0, 2, 4]
    tensors = [t for t in (kv.k, kv.v, kv.k_scale, kv.v_scale) if t is not None]
    want = [t.clone().cpu() for t in tensors]
    for b in range(B):
        for j in range(n_path[b] if start[b] >= 0 else 0):
            s, e = start[b] + path[b, j], start[b] + j
            for w in want:
                u = w if w.dtype == torch.float32 else raw(w).view(*w.shape[:3], -1)
                u[table[b, e // page], :, e % page] = u[table[b, s // page], :, s % page].clone()
    gdn.gdn_kv_commit(kv, *(torch.from_numpy(a).cuda() for a in (table, start, path, n_path)), B, T)
    for t, w in zip(tensors, want):
        assert torch.equal(raw(t).cpu(), raw(w))


def test_index_check_refuses_before_writing():
    kv = make("i8", 4, 1, 16, 64)
    kv.c.flags = gdn.GDN_F_CHECK_INDICES
    rows = torch.randn(8, 1, 64, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    before = kv.k.clone()
    good = i32([[0, 1]]), i32([10])
    for table, start, n_new in ((i32([[0, 4]]), good[1], None), (good[0], i32([-1]), None), (good[0], i32([25]), None),
                                (good[0], good[1], i32([9]))):
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_kv_write(kv, rows, rows, table, start, n_new, 1, 8)
        assert e.value.code == gdn.GDN_ERR_RANGE
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_kv_commit(kv, *good, i32([[3, 3]]), i32([2]), 1, 8)
    assert e.value.code == gdn.GDN_ERR_RANGE
    assert torch.equal(kv.k, before)
    gdn.gdn_kv_write(kv, rows, rows, *good, None, 1, 8)
    assert not torch.equal(kv.k, before)


def test_write_and_read_replay_in_a_graph():
    B, T, n_kv, d, page = 2, 6, 2, 128, 16
    kv = make("e4m3", 8, n_kv, page, d)
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    start = torch.tensor([3, 14], dtype=torch.int32).cuda()
    x = torch.randn(B * T, 2 * n_kv, d, device="cuda", dtype=torch.bfloat16)
    out = [torch.zeros(B * T, n_kv, d, device="cuda") for _ in range(4)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv_write(kv, x[:, :n_kv], x[:, n_kv:], table, start, None, B, T)
        gdn.gdn_kv_read(kv, table, start, None, out[0], out[1], B, T)
    for step in range(3):
        x.copy_(torch.randn_like(x))
        start.add_(step)
        g.replay()
        torch.cuda.synchronize()
        gdn.gdn_kv_write(kv, x[:, :n_kv], x[:, n_kv:], table, start, None, B, T)
        gdn.gdn_kv_read(kv, table, start, None, out[2], out[3], B, T)
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3]), step
