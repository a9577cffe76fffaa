"""GPU: a cache dimension of a single entry has no stride to compare: key and
value caches that lie alike in memory are taken, whatever torch calls the step
of such a dimension."""
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, check, dev, make

pytestmark = pytest.mark.gpu


def with_step(x, dim, step):
    strides = list(x.stride())
    strides[dim] = step
    return torch.as_strided(x, x.shape, strides)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("order", ["token", "head"])
def test_single_entries(order, eight):
    ctx = dk.Context(0)
    try:
        s = make(3, [20, 3], [1, 2], 1, 4, 64, 8, order, eight)   # one head
        want, _ = call(ctx, s)
        got, lse = call(ctx, dict(s, vc=with_step(s["vc"], 2, 3)))
        again, _ = call(ctx, dict(s, kc=with_step(s["kc"], 2, 1)))
        ctx.check()
        check(s, got, lse)
        assert torch.equal(got, want) and torch.equal(again, want)
        kc, vc = [torch.zeros_like(s["kc"]) for _ in range(2)]
        k = torch.randn((2, 1, 64), device="cuda").to(torch.bfloat16)
        ctx.cache_write(k, -k, dev([9, 3]), kc, with_step(vc, 2, 5), s["ks"], s["vs"])
        ctx.check()
        at = (torch.tensor([1, 0]), torch.tensor([1, 3]))
        if not eight:
            assert torch.equal(kc[at], k) and torch.equal(vc[at], -k)
        assert kc[at].float().abs().sum() > 0 and vc[at].float().abs().sum() > 0
        one = make(4, [3], [2], 2, 1, 64, 8, order, eight)        # one page used of one
        kc, vc = one["kc"][:1], one["vc"][:1]
        one["table"][one["table"] >= 0] = 0
        one.update(kc=kc, vc=vc)
        a, _ = call(ctx, one)
        b, _ = call(ctx, dict(one, vc=with_step(vc, 0, 16)))
        ctx.check()
        assert torch.equal(a, b)
        with pytest.raises(ValueError, match="one set of strides"):
            call(ctx, dict(s, vc=torch.empty((s["vc"].shape[0], 9, 1, 64), dtype=s["vc"].dtype, device="cuda")[:, :8]))
    finally:
        ctx.close()
