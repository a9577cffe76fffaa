"""GPU: scores up to 1.8e8, where a float's step is 8 to 16 units of the
exponent.  The weights themselves are then what rounding leaves of them, but
they are the same in a row's sum and in its products: over values that are
all alike the result is that value, whatever steps the maximum rose by.

Tolerance: the result's rounding 2^-8, a weight's 2^-11 and, where the largest
is as small as 2^-8, 2^-17 more; sums of n terms n 2^-24."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exponent", [4, 12, 15, 16, 17, 18])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 8), (256, 2)])
@pytest.mark.parametrize("eight", [False, True])
def test_values_alike(eight, d, group, exponent, sign):
    ctx = dk.Context(0)
    try:
        s = make(exponent + d, [2500, 70, 33], [7, 3, 0], 4, group, d, 16, "token", eight)
        rng = np.random.RandomState(exponent)
        q, k = torch.zeros_like(s["q"]), s["kc"].float().zero_()
        q[..., 0], q[..., 1], q[..., 2] = sign * 2.0 ** exponent, 8.0, 8.0
        k[..., 0] = 448.0                                        # the common part, and up to 30 steps of 8 above it
        for b, (L, K) in enumerate(zip(s["length"], s["K"])):
            t = np.arange(L + K + 1)
            level = (np.minimum(t * 40 // len(t), 28) + rng.randint(0, 3, len(t))).clip(0, 30)
            for p in range(-(-len(t) // 16)):
                x = torch.zeros(16, device="cuda")
                part = level[16 * p:16 * p + 16]
                x[:len(part)] = torch.from_numpy(part.astype(np.float32)).cuda()
                page = int(s["table"][b][p])
                k[page, :, :, 1], k[page, :, :, 2] = x.clamp(max=16)[:, None], (x - 16).clamp(min=0)[:, None]
        s["kc"].copy_(k.to(s["kc"].dtype))
        v = torch.linspace(-2, 2, 4 * d, device="cuda").view(4, d).to(s["vc"].dtype).float()
        s["vc"].copy_(v.expand(s["vc"].shape).to(s["vc"].dtype))
        s["q"], s["scale"] = q, 1.0
        if eight:
            s["ks"].fill_(1.0)
            s["vs"].fill_(1.0)
        out, lse = call(ctx, s)
        ctx.check()
        want = v.repeat_interleave(group, 0)[None].double()
        err = (out.double() - want).abs()
        assert torch.isfinite(out.float()).all()
        assert (err <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17 + 2540 * 2.0 ** -24) * want.abs()).all(), err.max()
        base = sign * 448.0 * 2.0 ** exponent
        assert (lse.double() - base >= -2.0 ** -21 * abs(base)).all()
        assert (lse.double() - base <= 240 + np.log(2540) + 2.0 ** -21 * abs(base)).all()
    finally:
        ctx.close()
