"""Bounds on the attention's results that take every path for what it rounds its weights to: narrow enough to tell
weights of one bf16 part from two, or fp16 weights from bf16 ones."""

import numpy as np
import torch

from tests import attn_ref as ref
from tests.test_gpu_attn import Case

# Half a step of fp16, relative; what two bf16 parts leave (the first is up to a whole step, 2^-7, below the weight,
# the second is rounded to half a step of what is left, 2^-8); half a step of bf16.
FP16, TWO_BF16, BF16 = 2.0 ** -11, 2.0 ** -15, 2.0 ** -8


class Sharp(Case):
    """Per output |error| <= t + 2^-8 (|o| + t), its own rounding on top of t, the sum over the keys j of w_j |v_j| times
    the weight's rounding, the exponent's error (2 e, e that of the scores) and the sums' (n 2^-24, and 2^-20 for exp2 and the
    scale products); fp16 weights add 2^-32 of the row's largest w vs for each |code| (half of fp16's smallest step, the
    largest taken as 2^7 or more).

    Over a whole call the root mean square of the error is held to that of rounding the exact results to bf16 and of
    weights rounded independently, evenly within half a step (variance a third of its square), plus a tenth."""

    def weight_errors(self):
        """Of the prefix's keys and of the entries' own: bf16 weights go in two parts where at most 64 rows share keys."""
        if self.fmt != "bf16":
            return FP16, FP16
        rows = self.T * self.grp
        return tuple(TWO_BF16 if n <= 64 else BF16 for n in (rows * self.B, rows))

    def keys(self, b, h):
        """(q, k, v, v scales, mask) of the rows of entry b and KV head h, fp64, in full."""
        T, ctx = self.T if self.n_new is None else min(self.T, int(self.n_new[b])), int(self.ctx[b])
        draft = ref.sees(self.T, None if self.parent is None else self.parent[b])[:T, :T]
        sees = np.concatenate([np.ones((T, self.prefix + ctx), bool), draft], 1).repeat(self.grp, 0)
        runs = (self.shared, np.arange(self.prefix)), (self.table[b], np.arange(ctx + T))
        k, v = (np.concatenate([self.values(n, pages, pos, h) for pages, pos in runs]) for n in ("k", "v"))
        vs = np.ones(len(k))
        if self.fmt != "bf16":
            at = [self.at(pages, pos) for pages, pos in runs]
            vs = np.concatenate([self.store["v_scale"][pg, h, place].double().numpy() for pg, place in at])
        q = self.q.double().numpy().reshape(self.B, self.T, -1, self.d)[b, :T, h * self.grp:(h + 1) * self.grp]
        return q.reshape(-1, self.d), k, v, vs, sees

    def check(self, out):
        """The largest error as a part of its bound, and the root mean square as a part of its own."""
        got = out.double().cpu().numpy().reshape(self.B, self.T, self.n_kv, self.grp, self.d)
        most, err2, own2, n = 0.0, 0.0, 0.0, 0
        for b in range(self.B):
            for h in range(self.n_kv):
                q, k, v, vs, sees = self.keys(b, h)
                o, w = ref.attend(q, k, v, sees, self.scale)
                r = np.repeat(self.weight_errors(), [self.prefix, len(k) - self.prefix])
                e = (self.d + 8) * 2.0 ** -24 * self.scale * (np.abs(q) @ np.abs(k).T).max()
                t = (w * r) @ np.abs(v) + (w @ np.abs(v)) * (2 * e + len(k) * 2.0 ** -24 + 2.0 ** -20)
                if self.fmt != "bf16":
                    t = t + 2.0 ** -32 * (w * vs).max(1, keepdims=True) * (sees @ (np.abs(v) / np.where(vs > 0, vs, 1.0)[:, None]))
                t = t + 2.0 ** -8 * (np.abs(o) + t)
                err = np.abs(got[b, :len(o) // self.grp, h].reshape(-1, self.d) - o)
                assert np.isfinite(err).all()
                most = max(most, float((err / np.maximum(t, 1e-300)).max()))
                rounding = torch.from_numpy(o).to(torch.bfloat16).double().numpy() - o
                err2, n = err2 + (err ** 2).sum(), n + err.size
                own2 += (rounding ** 2).sum() + ((w * r) ** 2 @ v ** 2).sum() / 3
        rms = float(np.sqrt(err2 / own2))
        assert most <= 1 and rms <= 1.1, (most, rms)
        return most, rms


# n_kv, grp, page, ctx, T, keywords: few enough keys that one weight's rounding shows in a result
SHARP = {
    "one row": (2, 1, 16, [40, 17, 9], 1, {}),
    "32 rows": (1, 4, 16, [20, 33], 8, {}),
    "64 rows": (1, 4, 64, [30, 0], 16, {}),
    "64 rows, tree, ragged": (2, 2, 16, [30, 5], 32, dict(tree=True, n_new=[32, 11])),
    "72 rows": (1, 4, 16, [30], 18, {}),
    "256 rows": (1, 8, 16, [10], 32, {}),
    "prefix, 12 rows": (2, 2, 16, [12, 10, 14], 2, dict(prefix=16)),
    "prefix, 160 rows of 32": (1, 8, 16, [25, 20, 30, 23, 21], 4, dict(prefix=5)),
}


def sharp_case(shape, fmt, d):
    n_kv, grp, page, ctx, T, kw = SHARP[shape]
    c = Sharp(fmt, d, n_kv, grp, page, ctx, T, seed=len(shape) + d, **kw)
    c.q = c.q / 4  # scores of unit size: their fp32 rounding stays below 2^-15 of a weight
    return c
