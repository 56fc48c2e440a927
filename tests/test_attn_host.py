"""Rotary tables and the refusals of the full-attention layers' entry points, on the host: no launch is made."""

import ctypes
import math

import numpy as np
import pytest

from gated_deltanet_linear_verify_amd import gdn
from tests import attn_ref as ref

FAKE = 0x1000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(gdn.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return gdn.lib()


@pytest.mark.parametrize("scaling", ["plain", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,theta,factor,orig", [(64, 1e7, 4.0, 4096), (128, 1e4, 1.0, 32768), (36, 1e6, 40.0, 1), (4, 10.0, 2.5, 100)])
def test_rope_table(L, rot, theta, factor, orig, scaling):
    code = ["plain", "linear", "ntk", "yarn"].index(scaling)
    t = gdn.gdn_rope_init(rot, theta=theta, scaling=code, factor=factor, orig_ctx=orig, sections=(rot // 2 - 1, 0, 1, 0))
    f, m = ref.frequencies(rot, theta, scaling, factor if scaling != "plain" else 1.0, orig)
    got = np.array(t.turns[:rot // 2]) * 2 * math.pi
    assert np.abs(got / f - 1).max() < 1e-14  # a few roundings of pow and the products
    assert t.mscale == np.float32(m)
    assert (t.n_axes, list(t.axis_end)) == (4, [rot // 2 - 1, rot // 2 - 1, rot // 2, rot // 2])


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=7), gdn.GDN_ERR_SHAPE), (dict(rot_dim=0), gdn.GDN_ERR_SHAPE), (dict(rot_dim=258), gdn.GDN_ERR_SHAPE),
    (dict(layout=2), gdn.GDN_ERR_ARG), (dict(scaling=4), gdn.GDN_ERR_ARG), (dict(theta=1.0), gdn.GDN_ERR_ARG),
    (dict(theta=float("nan")), gdn.GDN_ERR_ARG), (dict(theta=float("inf")), gdn.GDN_ERR_ARG),
    (dict(scaling=1, factor=0.5), gdn.GDN_ERR_ARG), (dict(scaling=1, factor=float("nan")), gdn.GDN_ERR_ARG),
    (dict(rot_dim=2, scaling=2, factor=2.0), gdn.GDN_ERR_ARG), (dict(scaling=3, factor=2.0), gdn.GDN_ERR_ARG),
    (dict(scaling=3, factor=2.0, orig_ctx=4096, beta_fast=1.0, beta_slow=2.0), gdn.GDN_ERR_ARG),
    (dict(sections=(1, 2, 3, 4)), gdn.GDN_ERR_SHAPE), (dict(sections=(-1, 33, 0, 0)), gdn.GDN_ERR_SHAPE),
    (dict(mscale=-1.0), gdn.GDN_ERR_ARG),
])
def test_rope_init_refuses(L, kw, code):
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_rope_init(**{"rot_dim": 64, **kw})
    assert e.value.code == code
    assert L.gdn_rope_init(None, None) == gdn.GDN_ERR_ARG


def _rows(**kw):
    return gdn.gdn_rows(**{**dict(ptr=FAKE, ld=512, hd=128, n_heads=4, dtype=gdn.GDN_BF16), **kw})


def _kv(**kw):
    return gdn.gdn_kv(**{**dict(n_kv=4, d=128, page_size=64, n_pages=10, format=gdn.GDN_KV_I8, flags=0, k=FAKE, v=FAKE,
                                k_scale=FAKE, v_scale=FAKE), **kw})


def _batch(**kw):
    return gdn.gdn_kv_batch(**{**dict(block_table=FAKE, start=FAKE, n_new=None, max_pages=4, n_batch=2, n_tok=3), **kw})


def test_rope_refuses(L):
    t = gdn.gdn_rope_init(64)
    r = lambda x, o, n_segs=1, d=128, n=3, tab=t, pos=FAKE: L.gdn_rope(  # noqa: E731
        ctypes.byref(tab) if tab is not None else None, ctypes.byref(x), ctypes.byref(o), n_segs, d, pos, n, 0, None)
    ok = _rows()
    assert r(ok, ok, tab=None) == gdn.GDN_ERR_ARG
    assert r(ok, ok, pos=None) == gdn.GDN_ERR_ARG
    assert r(ok, ok, n_segs=0) == gdn.GDN_ERR_SHAPE
    assert r(ok, ok, n_segs=5) == gdn.GDN_ERR_SHAPE
    assert r(ok, ok, d=257) == gdn.GDN_ERR_SHAPE
    assert r(ok, ok, d=62) == gdn.GDN_ERR_SHAPE
    assert r(ok, ok, n=-1) == gdn.GDN_ERR_RANGE
    assert r(_rows(ptr=None), ok) == gdn.GDN_ERR_ARG
    assert r(_rows(ptr=FAKE + 1), ok) == gdn.GDN_ERR_ARG
    assert r(_rows(dtype=5), ok) == gdn.GDN_ERR_DTYPE
    assert r(_rows(n_heads=3), ok) == gdn.GDN_ERR_SHAPE
    assert r(_rows(hd=64), ok) == gdn.GDN_ERR_ARG
    assert r(_rows(dtype=gdn.GDN_F32), ok) == gdn.GDN_ERR_ARG
    assert r(ok, ok, tab=gdn.gdn_rope_table()) == gdn.GDN_ERR_ARG
    assert r(ok, ok, n=0) == gdn.GDN_OK  # nothing to do: no launch


KV_BAD = [
    (dict(format=3), gdn.GDN_ERR_DTYPE), (dict(d=96), gdn.GDN_ERR_SHAPE), (dict(n_kv=0), gdn.GDN_ERR_SHAPE),
    (dict(n_pages=0), gdn.GDN_ERR_SHAPE), (dict(page_size=48), gdn.GDN_ERR_SHAPE), (dict(page_size=8), gdn.GDN_ERR_SHAPE),
    (dict(page_size=8192), gdn.GDN_ERR_SHAPE), (dict(flags=1), gdn.GDN_ERR_ARG), (dict(k=None), gdn.GDN_ERR_ARG),
    (dict(v=FAKE + 8), gdn.GDN_ERR_ARG), (dict(k_scale=None), gdn.GDN_ERR_ARG), (dict(v_scale=FAKE + 2), gdn.GDN_ERR_ARG),
    (dict(format=gdn.GDN_KV_BF16), gdn.GDN_ERR_ARG),
]
BATCH_BAD = [
    (dict(block_table=None), gdn.GDN_ERR_ARG), (dict(start=None), gdn.GDN_ERR_ARG), (dict(n_batch=0), gdn.GDN_ERR_RANGE),
    (dict(n_batch=65536), gdn.GDN_ERR_RANGE), (dict(n_tok=0), gdn.GDN_ERR_RANGE), (dict(max_pages=0), gdn.GDN_ERR_SHAPE),
    (dict(n_batch=60000, n_tok=60000), gdn.GDN_ERR_SHAPE),
]
ROWS_BAD = [
    (dict(ptr=None), gdn.GDN_ERR_ARG), (dict(dtype=9), gdn.GDN_ERR_DTYPE), (dict(n_heads=2), gdn.GDN_ERR_SHAPE),
    (dict(ptr=FAKE + 8), gdn.GDN_ERR_ARG), (dict(ld=516), gdn.GDN_ERR_ARG), (dict(hd=130), gdn.GDN_ERR_ARG),
]


@pytest.mark.parametrize("kv,batch,k,v,code", [(_kv(**a), _batch(), _rows(), _rows(), c) for a, c in KV_BAD] +
                         [(_kv(), _batch(**a), _rows(), _rows(), c) for a, c in BATCH_BAD] +
                         [(_kv(), _batch(), _rows(**a), _rows(), c) for a, c in ROWS_BAD] +
                         [(_kv(), _batch(), _rows(), _rows(**a), c) for a, c in ROWS_BAD])
def test_kv_refuses(L, kv, batch, k, v, code):
    kb, kr, vr = ctypes.byref(batch), ctypes.byref(k), ctypes.byref(v)
    assert L.gdn_kv_write(ctypes.byref(kv), kb, kr, vr, None, None, None) == code
    assert L.gdn_kv_read(ctypes.byref(kv), kb, kr, vr, None) == code
    assert gdn.last_error()


def test_kv_refuses_the_rest(L):
    kv, b, r = ctypes.byref(_kv()), ctypes.byref(_batch()), ctypes.byref(_rows())
    f32 = ctypes.byref(_rows(dtype=gdn.GDN_F32))
    assert L.gdn_kv_write(None, b, r, r, None, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_write(kv, None, r, r, None, None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_write(kv, b, r, f32, None, None, None) == gdn.GDN_ERR_DTYPE
    big, t = gdn.gdn_rope_init(256), gdn.gdn_rope_init(64)
    assert L.gdn_kv_write(kv, b, r, r, ctypes.byref(t), None, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_write(kv, b, r, r, ctypes.byref(big), FAKE, None) == gdn.GDN_ERR_SHAPE
    assert L.gdn_kv_commit(kv, b, None, FAKE, 2, None) == gdn.GDN_ERR_ARG
    assert L.gdn_kv_commit(kv, b, FAKE, FAKE, 0, None) == gdn.GDN_ERR_RANGE
    assert L.gdn_kv_commit(kv, b, FAKE, FAKE, 4, None) == gdn.GDN_ERR_RANGE
    for a, code in KV_BAD:
        assert L.gdn_kv_commit(ctypes.byref(_kv(**a)), b, FAKE, FAKE, 2, None) == code


def test_kv_bytes(L):
    assert gdn.gdn_kv_bytes(8, 128, 64, 1000, gdn.GDN_KV_E4M3) == (8 * 128 * 64 * 1000, 4 * 8 * 64 * 1000)
    assert gdn.gdn_kv_bytes(2, 256, 16, 1 << 20, gdn.GDN_KV_BF16) == (2 * 256 * 16 * 2 << 20, 0)
    assert gdn.gdn_kv_bytes(2, 100, 16, 3, gdn.GDN_KV_BF16) == (0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(kv=None), gdn.GDN_ERR_ARG), (dict(batch=None), gdn.GDN_ERR_ARG), (dict(q=None), gdn.GDN_ERR_ARG),
    (dict(out=None), gdn.GDN_ERR_ARG), (dict(q=_rows(n_heads=6)), gdn.GDN_ERR_SHAPE), (dict(q=_rows(n_heads=2)), gdn.GDN_ERR_SHAPE),
    (dict(out=_rows(n_heads=8)), gdn.GDN_ERR_SHAPE), (dict(q=_rows(dtype=gdn.GDN_F32)), gdn.GDN_ERR_DTYPE),
    (dict(out=_rows(dtype=gdn.GDN_F32)), gdn.GDN_ERR_DTYPE), (dict(q=_rows(ptr=FAKE + 2)), gdn.GDN_ERR_ARG),
    (dict(scale=0.0), gdn.GDN_ERR_ARG), (dict(scale=float("nan")), gdn.GDN_ERR_ARG), (dict(scale=float("inf")), gdn.GDN_ERR_ARG),
    (dict(parent=FAKE, batch=_batch(n_tok=1025)), gdn.GDN_ERR_SHAPE), (dict(pages=FAKE), gdn.GDN_ERR_ARG),
    (dict(plen=FAKE), gdn.GDN_ERR_ARG), (dict(pages=FAKE, plen=FAKE, n_pages=0), gdn.GDN_ERR_SHAPE),
    (dict(ws=None), gdn.GDN_ERR_ARG), (dict(ws=FAKE + 4), gdn.GDN_ERR_ARG), (dict(ws_bytes=100), gdn.GDN_ERR_ARG),
    (dict(batch=_batch(max_pages=1 << 25)), gdn.GDN_ERR_SHAPE),
])
def test_attn_refuses(L, kw, code):
    a = dict(kv=_kv(), batch=_batch(), parent=None, pages=None, n_pages=3, plen=None, q=_rows(), out=_rows(), scale=0.1,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    ref_ = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    assert L.gdn_attn_verify(ref_(a["kv"]), ref_(a["batch"]), a["parent"], a["pages"], a["n_pages"], a["plen"], ref_(a["q"]),
                             ref_(a["out"]), a["scale"], a["ws"], a["ws_bytes"], None) == code, gdn.last_error()


def test_attn_refuses_bad_caches_and_batches(L):
    r = ctypes.byref(_rows())
    for kv, b, code in [(_kv(**x), _batch(), c) for x, c in KV_BAD] + [(_kv(), _batch(**x), c) for x, c in BATCH_BAD]:
        assert L.gdn_attn_verify(ctypes.byref(kv), ctypes.byref(b), None, None, 0, None, r, r, 0.1, FAKE, 1 << 40, None) == code


def test_attn_workspace(L):
    n = lambda n_q, b, t, p, **kw: L.gdn_attn_workspace_bytes(ctypes.byref(_kv(**kw)), n_q, b, t, p)  # noqa: E731
    assert 0 < n(32, 64, 16, 0) < n(32, 64, 16, 1)
    assert n(6, 1, 1, 0) == n(32, 0, 1, 0) == n(32, 1, 0, 0) == n(32, 70000, 1, 0) == n(32, 1, 1, 0, d=96) == 0


def test_refuses_outputs_on_top_of_each_other(L):
    """A broadcast row may be read, never written."""
    t = gdn.gdn_rope_init(64)
    ok, flat, heads, back = _rows(), _rows(ptr=2 * FAKE, ld=0), _rows(ptr=2 * FAKE, hd=64), _rows(ptr=2 * FAKE, ld=-64)
    ref_, kv, b = ctypes.byref, _kv(), _batch()
    for bad in (flat, heads, back):
        assert L.gdn_rope(ref_(t), ref_(ok), ref_(bad), 1, 128, FAKE, 3, 0, None) == gdn.GDN_ERR_ARG
        assert L.gdn_kv_read(ref_(kv), ref_(b), ref_(bad), ref_(ok), None) == gdn.GDN_ERR_ARG
        assert L.gdn_kv_read(ref_(kv), ref_(b), ref_(ok), ref_(bad), None) == gdn.GDN_ERR_ARG
        assert L.gdn_attn_verify(ref_(kv), ref_(b), None, None, 0, None, ref_(ok), ref_(bad), 0.1, FAKE, 1 << 40, None) == gdn.GDN_ERR_ARG


def test_refuses_more_rows_than_a_launch_holds(L):
    b, r, kv = _batch(n_batch=60000, n_tok=1119), ctypes.byref(_rows()), ctypes.byref(_kv())  # just over 2^26
    assert L.gdn_kv_write(kv, ctypes.byref(b), r, r, None, None, None) == gdn.GDN_ERR_SHAPE
    assert L.gdn_kv_read(kv, ctypes.byref(b), r, r, None) == gdn.GDN_ERR_SHAPE
    n = lambda n_q, b, t: L.gdn_attn_workspace_bytes(kv, n_q, b, t, 0)  # noqa: E731
    assert n(4, 60000, 1118) and not n(4, 60000, 1119) and not n(8, 60000, 1118)
    wide = _batch(n_batch=60000, n_tok=1118)
    assert L.gdn_attn_verify(kv, ctypes.byref(wide), None, None, 0, None, ctypes.byref(_rows(n_heads=8, ld=1024)),
                             ctypes.byref(_rows(n_heads=8, ld=1024)), 0.1, FAKE, 1 << 62, None) == gdn.GDN_ERR_SHAPE


def test_refuses_a_scale_that_overflows(L):
    r = ctypes.byref(_rows())
    for scale in (3e38, -1.0):
        assert L.gdn_attn_verify(ctypes.byref(_kv()), ctypes.byref(_batch()), None, None, 0, None, r, r, scale, FAKE, 1 << 40,
                                 None) == gdn.GDN_ERR_ARG
