"""Attention over the paged cache held to what its weights are rounded to, path by path."""

import pytest

from tests.attn_bounds import SHARP, sharp_case
from tests.gpu_util import say
from tests.test_gpu_attn import FMT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("shape", list(SHARP))
def test_weights_keep_their_bits(shape, fmt, d):
    c = sharp_case(shape, fmt, d).upload()
    most, rms = c.check(c.run())
    say(f"{shape}, {fmt}, d {d}: {most:.2f} of the bound, rms {rms:.2f}")
