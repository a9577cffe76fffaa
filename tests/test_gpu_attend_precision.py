"""GPU: how finely dspark_attend weighs the values it adds.  The result is one
bf16 rounding away from the exact one, and the weights must not add another of
its kind.

Rounding of a weight p: bf16 caches, p as its leading 8 bits (what is cut off
is below 2^-7 p) and that remainder to nearest bf16 (2^-8 of it): 2^-15 p.
e4m3 caches, p to nearest f16: 2^-11 p, and 2^-25 where f16 is subnormal, with
the row's largest weight at least 2^7: 2^-32 of the largest."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from attend_reference import worst_error
from test_gpu_attend import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def bounds(eight):
    return dict(weight=2.0 ** -11, floor=2.0 ** -32) if eight else dict(weight=2.0 ** -15)


@pytest.mark.parametrize("d,group", [(64, 1), (64, 4), (128, 2), (128, 8), (256, 1), (256, 3)])
@pytest.mark.parametrize("eight", [False, True])
def test_values_that_cancel(ctx, d, group, eight):
    """Values of +1 and -1 under nearly equal weights: the sum is small, so that its own rounding hides nothing."""
    print(f"precision d={d} group={group} 8bit={eight}", flush=True)
    s = make(21 + d, [1, 2, 3, 4, 7, 40, 300], [7, 7, 7, 7, 7, 7, 7], 8, group, d, 16, "token", eight, spread=0.15)
    s["vc"].copy_(s["vc"].float().sign().to(s["vc"].dtype))
    if eight:
        s["vs"].fill_(1.0)
    for causal in (True, False):
        out, lse = call(ctx, s, causal)
        ctx.check()
        worst = worst_error(s, out, lse, causal, **bounds(eight))
        print("worst error over its bound: %.3f" % worst, flush=True)
        assert worst <= 1.0


@pytest.mark.parametrize("low", [14.0, 18.0, 20.0])
@pytest.mark.parametrize("eight", [False, True])
def test_many_small_weights(ctx, low, eight):
    """One token far above 20000 others, which alone carry a value: weights of 2^-20 to 2^-29 of the largest, in steps
    before the large one, behind it and around it."""
    for place in (0, 9000, 20000):
        s = make(5, [20000], [0], 1, 2, 64, 16, "token", eight)
        for c in (s["kc"], s["vc"]):
            c.copy_(torch.zeros_like(c.float()).to(c.dtype))
        page, at = int(s["table"][0][place // 16]), place % 16
        s["q"].zero_()
        s["q"][..., 0] = 1
        k, v = s["kc"].float(), s["vc"].float()
        k[page, at, 0, 0] = low
        v[:] = 1
        v[page, at] = 0
        s["kc"].copy_(k.to(s["kc"].dtype))
        s["vc"].copy_(v.to(s["vc"].dtype))
        s["scale"] = 1.0
        if eight:
            s["ks"].fill_(1.0)
            s["vs"].fill_(1.0)
        out, lse = call(ctx, s)
        ctx.check()
        worst = worst_error(s, out, lse, True, **bounds(eight))
        print(f"small weights low={low} place={place}: worst error over its bound {worst:.3f}", flush=True)
        assert worst <= 1.0
