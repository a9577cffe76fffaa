"""GPU: repetition penalties at the ends of their range.  A penalty below the
smallest normal number is flagged and taken as 1 (its reciprocal is infinite);
from there to the largest finite one the quotient is the quotient."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import dev

pytestmark = pytest.mark.gpu

TINY, HUGE = float(np.finfo(np.float32).tiny), float(np.finfo(np.float32).max)


def call(ctx, x, rep, n):
    rows = torch.from_numpy(x.astype(np.float32)).cuda()
    B = len(rep)
    return ctx.constrain(rows, 1, t_offsets=dev(np.arange(B)), hist=dev([list(range(n))] * B), n_hist=dev([n] * B),
                         rep=torch.tensor(rep, dtype=torch.float32, device="cuda"))


def test_penalties_over_the_whole_range():
    ctx = dk.Context(0)
    try:
        V, n = 64, 40
        rng = np.random.RandomState(1)
        rep = [TINY, TINY * 1.7, 1e-37, 3e-30, 0.3, 1.0, 7.7, 1e30, 2.0 ** 126, 1.3 * 2.0 ** 126, 1.9 * 2.0 ** 127, HUGE]
        rep = [float(np.float32(r)) for r in rep]
        for size in (1e-30, 1e-5, 30.0, 1e25):
            x = (rng.randn(len(rep), V) * size).astype(np.float32)
            got = call(ctx, x, rep, n).double().cpu().numpy()
            ctx.check()
            r = np.array(rep)[:, None]
            with np.errstate(over="ignore", under="ignore"):
                want = np.where(x > 0, x / r, x * r)
                want = np.where(np.abs(want) > HUGE, np.copysign(np.inf, want), want)
            want = np.maximum(np.where(np.arange(V)[None, :] < n, want, x), dk.MASKED)
            inf = np.isinf(want)
            assert np.array_equal(got[inf], want[inf])
            # one unit of the last place: half a step of each of two roundings; steps of 2^-149 where it is subnormal
            assert (np.abs(got[~inf] - want[~inf]) <= 2.0 ** -23 * np.abs(want[~inf]) + 2.0 ** -149).all(), size
        for bad in (1e-39, 1e-45, float(np.nextafter(np.float32(TINY), np.float32(0)))):
            x = rng.randn(2, V).astype(np.float32) * 1e-5
            got = call(ctx, x, [bad, 2.0], n).cpu().numpy()
            with pytest.raises(dk.DSparkError, match="repetition penalty"):
                ctx.check()
            assert np.array_equal(got[0], x[0]) and np.isfinite(got).all()
            assert np.array_equal(got[1], np.where((np.arange(V) < n), np.where(x[1] > 0, x[1] / 2, x[1] * 2), x[1]))
    finally:
        ctx.close()
