"""GPU: row arrays of the largest size that dspark_pages_reserve takes (2^31 - 1
entries, 8.6 GB each): rows at the beginning, -1 to the very end, nothing
before the arrays or behind them."""
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_pages import dev

pytestmark = pytest.mark.gpu


def test_the_most_rows():
    n, guard = 2 ** 31 - 1, 4096
    ctx = dk.Context(0)
    try:
        # the row arrays in one allocation, guards before, between and behind them
        whole = torch.full((3 * n + 4 * guard,), 7, dtype=torch.int32, device="cuda")
        at = [guard + i * (n + guard) for i in range(3)]
        req, pos, slot = [whole[a:a + n] for a in at]
        offs = torch.empty((3,), dtype=torch.int32, device="cuda")
        ctx.pages_reserve(dev([2, 0]), dev([7, 0]), dev([[3, -1, -1], [-1, -1, -1]]), dev([1, 0]), dev([0, 1, 2, 4]), dev([3]), 8, 4,
                          out=(offs, req, pos, slot))
        ctx.check()
        assert offs.tolist() == [0, 3, 4]
        assert req[:6].tolist() == [0, 0, 0, 1, -1, -1] and pos[:6].tolist() == [7, 8, 9, 0, -1, -1]
        assert slot[:6].tolist() == [31, 16, 17, 8, -1, -1]
        step = 2 ** 28
        for x in (req, pos, slot):
            for lo in range(4, n, step):
                assert bool((x[lo:lo + step] == -1).all()), lo
        for a in [0] + [b + n for b in at]:
            assert bool((whole[a:a + guard] == 7).all())
    finally:
        ctx.close()
