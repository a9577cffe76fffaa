"""GPU: calls over the paged cache and constraints at the ends of what their
documentation allows: results written where inputs stand are refused, the
largest batch, a batch that takes no part at all, the smallest pages, many
heads, one row and one head with arbitrary strides, a scale of zero."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, check, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def test_results_over_inputs_are_refused(ctx):
    s = make(1, [20, 9], [1, 0], 1, 2, 64, 8)
    before = s["q"].clone()
    with pytest.raises(dk.DSparkError, match="out may not be q"):
        call(ctx, s, out=s["q"])
    x = torch.randn((4, 64), device="cuda")
    for bad in (lambda: ctx.constrain(x[:2, :32], 1, t_offsets=dev([0, 1]), out=x.view(2, 128)[:, :32]),
                lambda: ctx.constrain(x[:2].view(torch.bfloat16)[:, :64], 1, t_offsets=dev([0, 1]), out=x[:2])):
        with pytest.raises(dk.DSparkError, match="in place"):
            bad()
    ctx.check()
    assert torch.equal(s["q"], before)


def test_the_largest_batch(ctx):
    """4096 requests: pages reserved, one row each (some none), attention, pages back."""
    B, page = 4096, 8
    rng = np.random.RandomState(2)
    s = make(2, rng.randint(0, 40, B), rng.randint(-1, 1, B), 1, 1, 64, page)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)
    with pytest.raises(dk.DSparkError, match="B must be"):
        ctx.attend(s["q"], s["kc"], s["vc"], dev(np.zeros((B + 1, 2))), dev(np.zeros(B + 1)), 0, K=dev(np.zeros(B + 1) - 1),
                   t_offsets=dev(np.zeros(B + 1)))


def test_nobody_takes_part(ctx):
    s = make(3, [20, 0, 300], [0, 0, 0], 2, 2, 128, 16)
    out = torch.full_like(s["q"], 7)
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    ctx.attend(s["q"], s["kc"], s["vc"], dev(s["table"]), dev(s["length"]), 3, K=dev([-1] * 3), t_offsets=dev([0] * 4), out=out,
               lse=lse)
    ctx.check()
    assert (out == 7).all() and (lse == 7).all()
    held = dev([2, 0, 19])
    offs, req, pos, slot = ctx.pages_reserve(dev([-1] * 3), dev(s["length"]), dev(s["table"]), held, dev([0] * 30), dev([0]), 16,
                                             30, n_rows=0)
    ctx.check()
    assert offs.tolist() == [0] * 4 and len(req) == len(pos) == len(slot) == 0 and held.tolist() == [2, 0, 19]
    x = torch.randn((3, 2, 40), device="cuda")
    y = torch.full_like(x, 7)
    ctx.constrain(x, 2, K=dev([-1] * 3), out=y)
    ctx.check()
    assert (y == 7).all()


@pytest.mark.parametrize("heads,group,d,eight", [(96, 1, 64, False), (40, 3, 128, True), (1, 64, 256, False)])
def test_many_heads(ctx, heads, group, d, eight):
    s = make(4, [100, 0, 37], [2, 0, 1], heads, group, d, 8, "head", eight)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_a_scale_of_zero(ctx):
    """A head whose scale is 0 weighs every token that a row sees alike, and none behind it."""
    s = make(5, [13, 50], [3, 6], 2, 2, 64, 8, "token", True)
    s["ks"][1] = 0.0
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_one_row_and_one_head_with_arbitrary_strides(ctx):
    """Dimensions of a single entry: torch leaves their strides as they come."""
    s = make(6, [40], [0], 1, 1, 64, 8)
    a, la = call(ctx, s)
    t = dict(s)
    t["q"] = torch.as_strided(s["q"].contiguous(), (1, 1, 64), (1, 3, 1))
    out = torch.as_strided(torch.zeros(64, dtype=torch.bfloat16, device="cuda"), (1, 1, 64), (5, 7, 1))
    b, lb = call(ctx, t, out=out)
    ctx.check()
    assert torch.equal(a, b) and torch.equal(la, lb)
