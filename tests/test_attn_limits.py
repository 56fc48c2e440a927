"""The ends of what the full-attention layers' entry points take, on the host: no launch is made."""

import ctypes
import os

import numpy as np
import pytest

from gated_deltanet_linear_verify_amd import gdn

FAKE = 0x1000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return gdn.lib()


def _rows(n_heads=4, d=128, **kw):
    return gdn.gdn_rows(**{**dict(ptr=FAKE, ld=n_heads * d, hd=d, n_heads=n_heads, dtype=gdn.GDN_BF16), **kw})


def _kv(**kw):
    return gdn.gdn_kv(**{**dict(n_kv=4, d=128, page_size=64, n_pages=10, format=gdn.GDN_KV_I8, flags=0, k=FAKE, v=FAKE,
                                k_scale=FAKE, v_scale=FAKE), **kw})


def _batch(**kw):
    return gdn.gdn_kv_batch(**{**dict(block_table=FAKE, start=FAKE, n_new=None, max_pages=4, n_batch=2, n_tok=3), **kw})


def _attn(L, kv=None, batch=None, q=None, out=None, pages=None, n_pages=0, plen=None, ws_bytes=1 << 62):
    """gdn_attn_verify with a workspace that is too small unless ws_bytes says otherwise: the check that comes last."""
    return L.gdn_attn_verify(ctypes.byref(kv or _kv()), ctypes.byref(batch or _batch()), None, pages, n_pages, plen,
                             ctypes.byref(q or _rows()), ctypes.byref(out or _rows(ptr=2 * FAKE)), 0.1, FAKE, ws_bytes, None)


def test_attention_rows_stay_below_what_a_launch_holds(L):
    """2^26 rows of 64 lanes (d 256) would be 2^32 threads, one too many."""
    kv = _kv(n_kv=1, d=256)
    ws = lambda n_q, b, t, p: L.gdn_attn_workspace_bytes(ctypes.byref(kv), n_q, b, t, p)  # noqa: E731
    for n_q, b, t in ((1, 1 << 13, 1 << 13), (4, 1 << 12, 1 << 12), (65536, 1 << 10, 1)):
        for prefix in (0, 1):
            assert ws(n_q, b, t, prefix) == 0 and "2^26" in gdn.last_error()
            assert ws(n_q, b - 1, t, prefix) > 0
        r, o = (_rows(n_heads=n_q, d=256, ptr=p) for p in (FAKE, 2 * FAKE))
        assert _attn(L, kv, _batch(n_batch=b, n_tok=t), r, o) == gdn.GDN_ERR_SHAPE
        assert _attn(L, kv, _batch(n_batch=b - 1, n_tok=t), r, o, ws_bytes=16) == gdn.GDN_ERR_ARG  # only the workspace


def test_attention_positions_stay_in_32_bits(L):
    """A table's end plus the call's tokens, and the tile that holds it, have to be int32 positions."""
    for page, n_tok in ((16, 3), (64, 1), (4096, 5000), (64, 1000)):
        most = ((1 << 31) - max(n_tok, 64) - 1) // page  # pages
        kv, r = _kv(page_size=page, n_kv=1), _rows(n_heads=1)
        for pages, code in ((most, gdn.GDN_ERR_ARG), (most + 1, gdn.GDN_ERR_SHAPE)):  # ARG: the workspace, looked at last
            assert _attn(L, kv, _batch(n_batch=1, n_tok=n_tok, max_pages=pages), r, r, ws_bytes=16) == code, (page, n_tok, pages)
            assert _attn(L, kv, _batch(n_batch=1, n_tok=n_tok), r, r, pages=FAKE, n_pages=pages, plen=FAKE, ws_bytes=16) == code


def test_attention_in_place_takes_the_same_strides(L):
    """out on q's memory: the same rows at the same places, or a row that one workgroup writes is another's q."""
    def code(rows, q, out):
        return _attn(L, batch=_batch(n_batch=1, n_tok=rows), q=_rows(**q), out=_rows(**out), ws_bytes=16)
    same, wide, turned = dict(ptr=FAKE), dict(ptr=FAKE, ld=1024), dict(ptr=FAKE, ld=128, hd=384)
    small = "workspace smaller"  # what is looked at last
    assert code(3, same, same) == gdn.GDN_ERR_ARG and small in gdn.last_error()
    assert code(3, same, dict(ptr=2 * FAKE, ld=1024)) == gdn.GDN_ERR_ARG and small in gdn.last_error()
    for rows, q, out in ((3, same, wide), (3, wide, same), (3, same, turned), (1, same, turned)):
        assert code(rows, q, out) == gdn.GDN_ERR_ARG and "strides" in gdn.last_error()
    assert code(1, same, wide) == gdn.GDN_ERR_ARG and small in gdn.last_error()  # one row: nothing is stepped over


def test_written_rows_on_top_of_each_other_are_refused(L):
    """Every combination of strides, against a count of the elements that two rows share."""
    table = gdn.gdn_rope_init(2)
    d, rng = 8, np.random.default_rng(0)
    cases = [(3, 4, 8, 8), (3, 4, 32, 8), (3, 4, 8, 24), (3, 4, 8, 16), (2, 2, 16, 24), (5, 3, 24, 16), (5, 3, 24, -16), (1, 4, 0, 8),
             (4, 1, 8, 0), (2, 3, -40, 12), (2, 3, 9, 1 << 62), (70000, 5, 1 << 40, 1 << 20)]
    cases += [tuple(int(x) for x in (*rng.integers(1, 7, 2), *rng.integers(-60, 61, 2))) for _ in range(3000)]
    seen = {True: 0, False: 0}
    for n, heads, ld, hd in cases:
        if n * heads < 1000:
            starts = sorted(a * ld + b * hd for a in range(n) for b in range(heads))
            apart = all(b - a >= d for a, b in zip(starts, starts[1:]))
        else:
            apart = True
        x = gdn.gdn_rows(FAKE, 0, 0, heads, gdn.GDN_F32)
        out = gdn.gdn_rows(2 * FAKE, ld, hd, heads, gdn.GDN_F32)
        # the segment behind it has a NULL pointer: the check that comes after the first one's
        xs, outs = (gdn.gdn_rows * 2)(x, gdn.gdn_rows()), (gdn.gdn_rows * 2)(out, gdn.gdn_rows())
        assert L.gdn_rope(ctypes.byref(table), xs, outs, 2, d, FAKE, n, 0, None) == gdn.GDN_ERR_ARG
        assert ("NULL" if apart else "on top of") in gdn.last_error(), (n, heads, ld, hd)
        seen[apart] += 1
    assert min(seen.values()) > 500


def test_rope_sections_are_all_counted(L):
    """A fifth section is refused, whatever the first four add up to; fewer than four are followed by zeros."""
    for sections in ((8, 8, 8, 8, 1), (32, 0, 0, 0, 0), (8, 8, 8, 4, 4)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_rope_init(64, sections=sections)
        assert e.value.code == gdn.GDN_ERR_SHAPE
    assert list(gdn.gdn_rope_init(64, sections=(20, 12)).axis_end) == [20, 32, 32, 32]
