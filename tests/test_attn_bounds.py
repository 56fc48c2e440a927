"""The attention tests' narrow bounds, tried on the CPU: results computed in 64 bits but for the weights, which are
rounded as the kernels round them or, for the mistakes that the bounds are there to show, more coarsely."""

import numpy as np
import pytest
import torch

from tests.attn_bounds import SHARP, sharp_case


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def _below(x):
    bits = np.maximum(np.float32(x).view(np.uint32), 1) - 1 & 0xffff0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


ROUND = {
    "two bf16": lambda w: _below(w) + _bf16(w - _below(w)),
    "bf16": _bf16,
    "fp16": lambda w: np.float16(w * 2.0 ** 7).astype(np.float64) / 2.0 ** 7,
    "e5m2": lambda w: torch.from_numpy(w).to(torch.float8_e5m2).double().numpy(),
}


def attend(c, own, prefix=None):
    """c's results in bf16 with the weights of the entries' keys (and of the prefix's) rounded by ROUND's entries."""
    out = torch.full((c.B * c.T, c.n_kv * c.grp, c.d), 7.0, dtype=torch.bfloat16)
    view = out.view(c.B, c.T, c.n_kv, c.grp, c.d)
    for b in range(c.B):
        for h in range(c.n_kv):
            q, k, v, vs, sees = c.keys(b, h)
            s = np.where(sees, q @ k.T * c.scale * np.log2(np.e) + np.log2(vs), -np.inf)
            w = np.exp2(s - s.max(1, keepdims=True))
            got = np.concatenate([ROUND[prefix or own](w[:, :c.prefix]), ROUND[own](w[:, c.prefix:])], 1)
            o = got @ (v / vs[:, None]) / (w / vs).sum(1, keepdims=True)
            view[b, :len(o) // c.grp, h] = torch.from_numpy(o).to(torch.bfloat16).view(-1, c.grp, c.d)
    return out


def _right(c, shape):
    if c.fmt != "bf16":
        return "fp16", "fp16"
    return tuple("two bf16" if r < 2.0 ** -9 else "bf16" for r in c.weight_errors()[::-1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("shape", list(SHARP))
def test_bounds_hold_for_the_right_rounding(shape, fmt):
    c = sharp_case(shape, fmt, 128)
    c.check(attend(c, *_right(c, shape)))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("shape", list(SHARP))
def test_bounds_tell_one_step_less(shape, fmt):
    """One bf16 part in the place of two or of fp16, e5m2 in the place of one bf16 part."""
    c = sharp_case(shape, fmt, 128)
    right = _right(c, shape)
    wrong = tuple("e5m2" if r == "bf16" else "bf16" for r in right)
    for own, prefix in [(wrong[0], right[1])] + ([(right[0], wrong[1])] if c.prefix else []):
        with pytest.raises(AssertionError):
            c.check(attend(c, own, prefix))
