"""GPU: bias rows longer than dspark_constrain indexes in 32 bits are refused on
the host; the longest below work."""
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import dev

pytestmark = pytest.mark.gpu


def test_the_longest_bias_row():
    ctx = dk.Context(0)
    try:
        x = torch.zeros((1, 64), device="cuda")
        ids = torch.full((1, 2 ** 29), 63, dtype=torch.int32, device="cuda")
        values = torch.ones((1, 2 ** 29), device="cuda")
        ids[0, :3] = torch.tensor([2, 5, 5])
        count = dev([3])
        with pytest.raises(dk.DSparkError, match="bias_max"):
            ctx.constrain(x, 1, t_offsets=dev([0]), bias=(ids, values, count))
        got = ctx.constrain(x, 1, t_offsets=dev([0]), bias=(ids[:, :-1], values[:, :-1], count))
        ctx.check()
        want = torch.zeros((1, 64), device="cuda")
        want[0, 2], want[0, 5] = 1, 2
        assert torch.equal(got, want)
    finally:
        ctx.close()
