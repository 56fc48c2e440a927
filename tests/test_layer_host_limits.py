"""gdn_norm's row lengths on the host: longer ones without the division than with it."""

import pytest

from gated_deltanet_linear_verify_amd import gdn
from tests.test_layer_host import A, B, BF, D, E, I8, SHAPE, built, norm, rows  # noqa: F401


@pytest.mark.parametrize("d,mode", [(16385, gdn.GDN_NORM_RMS), (65536, gdn.GDN_NORM_RMS), (65537, gdn.GDN_NORM_NONE), (0, gdn.GDN_NORM_NONE),
                                    (2 ** 31 - 1, gdn.GDN_NORM_NONE)])
def test_rows_that_are_too_long(d, mode):
    x, out = rows(A, ld=1 << 20, hd=0, heads=1), rows(B, ld=1 << 20, hd=0, heads=1, dtype=I8)
    assert norm(x=x, out=out, scale=D, weight=None, d=d, mode=mode) == SHAPE
    assert ("65536" if mode else "16384") in gdn.last_error()
    # the longest rows of no tokens
    assert norm(x=x, out=out, scale=D, weight=None, d=65536 if mode else 16384, mode=mode, n_tok=0) == gdn.GDN_OK


def test_long_rows_are_checked_like_others():
    x, out = rows(A, ld=20000, hd=0, heads=1), rows(B, ld=17407, hd=0, heads=1, dtype=BF)
    assert norm(x=x, out=out, weight=None, d=17408, mode=gdn.GDN_NORM_NONE) == gdn.GDN_ERR_ARG  # rows on top of each other
    assert norm(x=x, out=rows(B, ld=20000, hd=0, heads=1), weight=E + 2, d=17408, mode=gdn.GDN_NORM_NONE) == gdn.GDN_ERR_ARG
