"""GPU: calls that make their own outputs and are given a stream.  What they
make, and the zeros behind rows of no request, belong to that stream: work that
is still queued on the current one comes neither before nor after."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, dev, make

pytestmark = pytest.mark.gpu


def busy():
    """A few tens of milliseconds of work on the current stream."""
    x = torch.ones((8192, 8192), device="cuda")
    for _ in range(20):
        x = x @ x * 1e-4
    return x


def test_results_of_another_stream():
    ctx = dk.Context(0)
    try:
        s = make(1, [20, 900], [1, 3], 2, 2, 64, 8)
        want, _ = call(ctx, s)
        x = torch.randn((6, 512), device="cuda").to(torch.bfloat16)
        books = lambda: (dev([2, 0]), dev([5, 9]), dev([[0, -1], [1, 2]]), dev([1, 2]), dev([3, 4, 5, 6, 7, 0, 0, 0]), dev([5]), 8, 8)
        rows = ctx.pages_reserve(*books(), n_rows=5)
        args = [dev(s["table"]), dev(s["length"]), 3]
        kw = dict(K=dev(s["K"]), t_offsets=dev(s["offs"]), scale=s["scale"])
        offs, B = dev([0]), books()
        busy()                                                    # the products' first call
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        keep = busy()                                            # the current stream is busy, the other one free
        got = ctx.attend(s["q"], s["kc"], s["vc"], *args, **kw, stream=side)
        con = ctx.constrain(x, 6, t_offsets=offs, stream=side)
        res = ctx.pages_reserve(*B, n_rows=5, stream=side)
        torch.cuda.synchronize()
        ctx.check()
        assert torch.equal(got, want) and torch.equal(con, x.float())
        for a, b in zip(rows, res):
            assert torch.equal(a, b)
        assert torch.isfinite(keep).all()
    finally:
        ctx.close()
