"""GPU: a request whose pages do not hold the tokens it has cached is refused:
new pages would stand for tokens that were never written to them."""
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from test_gpu_pages import dev

pytestmark = pytest.mark.gpu

BOOKS = dict(table=[[5, 3, -1, -1], [4, -1, -1, -1], [1, 2, -1, -1]], free=[7, 6, 0, 0, 0, 0, 0, 0], n_free=2)


@pytest.mark.parametrize("K,length,held,fits", [
    ([0, 0, -1], [15, 8, 16], [2, 1, 2], True),                  # full pages hold what they have
    ([0, 0, -1], [15, 9, 16], [2, 1, 2], False),
    ([0, -1, -1], [15, 9, 16], [2, 1, 2], False),                # also where the request takes no rows
    ([0, 0, 0], [15, 8, 16], [2, 1, 1], False),
    ([-1, -1, -1], [1, 0, 0], [0, 0, 0], False),
    ([-1, -1, -1], [0, 0, 0], [0, 0, 0], True),
    ([0, 0, -1], [2 ** 31 - 9, 8, 16], [2, 1, 2], False),
])
def test_too_few_pages_for_the_cached_tokens(K, length, held, fits):
    ctx = dk.Context(0)
    try:
        table, h, n_free = dev(BOOKS["table"]), dev(held), dev([BOOKS["n_free"]])
        offs, req, pos, slot = ctx.pages_reserve(dev(K), dev(length), table, h, dev(BOOKS["free"]), n_free, 8, 8, n_rows=6)
        want = oracle.pages_reserve(K, length, BOOKS["table"], held, BOOKS["free"], BOOKS["n_free"], 8, 6)
        assert (want is not None) == fits
        if fits:
            ctx.check()
            for w, g in zip(want, (offs, req, pos, slot, table, h, n_free)):
                assert dev(w).reshape(-1).tolist() == g.reshape(-1).tolist()
        else:
            with pytest.raises(dk.DSparkError, match="page or row count out of range"):
                ctx.check()
            assert table.tolist() == BOOKS["table"] and h.tolist() == held and n_free.item() == 2
            assert not offs.any() and (slot == -1).all() and (req == -1).all()
    finally:
        ctx.close()
