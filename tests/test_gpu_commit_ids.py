"""GPU: a page id that is no page's does not enter the pool: the commit that
would give it back is refused as a whole, whichever workgroup meets it, and a
later call finds the counter of finished workgroups as it should be."""
import numpy as np
import pytest

import oracle
import semi_ar_draft_amd as dk
from test_gpu_pages import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def commit(ctx, s, finished=None):
    """The device state after the call: lengths, pages held, pool top, pool."""
    ln, hd, nf, free = dev(s["length"]), dev(s["held"]), dev([s["n_free"]]), dev(s["free"])
    ctx.pages_commit(ln, dev(s["acc"]), dev(s["table"]), hd, free, nf, 8, s["n_pages"],
                     finished=None if finished is None else dev(finished))
    return [x.cpu().numpy() for x in (ln, hd, nf, free)]


def state(B, cols, seed):
    rng = np.random.RandomState(seed)
    held = rng.randint(1, cols + 1, B)
    n_pages = int(held.sum()) + 5
    ids = rng.permutation(n_pages)
    table = np.full((B, cols), -1)
    at = 5
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.concatenate([ids[:5], np.full(n_pages - 5, -1)])
    length = rng.randint(0, 8 * held - 3)
    return dict(length=length, held=held, table=table, free=free, n_free=5, n_pages=n_pages, acc=rng.randint(-1, 3, B))


@pytest.mark.parametrize("B,cols", [(2, 4), (40, 6), (600, 30), (4096, 5)])   # one workgroup to 32
@pytest.mark.parametrize("bad", [-1, 0, 2 ** 31 - 1])                          # 0: one past the last id
@pytest.mark.parametrize("ending", [False, True])
def test_a_bad_id_is_not_given_back(ctx, B, cols, bad, ending):
    print(f"commit ids B={B} cols={cols} bad={bad} ending={ending}", flush=True)
    s = state(B, cols, B)
    fin = (np.arange(B) % 3 == 0).astype(np.int32) if ending else None
    good = oracle.pages_commit(s["length"], s["acc"], s["table"], s["held"], s["free"], 5, 8, fin, s["n_pages"])
    keep = good[1]
    given = [(b, p) for b in range(B) for p in range(keep[b], s["held"][b])]
    bad = bad or s["n_pages"]
    for at in (given[0], given[len(given) // 2], given[-1]):
        t = dict(s, table=s["table"].copy())
        t["table"][at] = bad
        assert oracle.pages_commit(t["length"], t["acc"], t["table"], t["held"], t["free"], 5, 8, fin, s["n_pages"]) is None
        ln, hd, nf, free = commit(ctx, t, fin)
        with pytest.raises(dk.DSparkError, match="page id out of range"):
            ctx.check()
        assert np.array_equal(ln, s["length"]) and np.array_equal(hd, s["held"]) and nf[0] == 5
        assert np.array_equal(free[:5], s["free"][:5])
        got = commit(ctx, s, fin)                                 # the next call is as ever
        ctx.check()
        for w, g in zip((good[0], good[1], [good[3]], good[2]), got):
            assert np.array_equal(w, g)
    kept = [(b, 0) for b in range(B) if keep[b] > 0]
    if kept:                                                      # an id that stays is not looked at
        t = dict(s, table=s["table"].copy())
        t["table"][kept[-1]] = bad
        got = commit(ctx, t, fin)
        ctx.check()
        for w, g in zip((good[0], good[1], [good[3]], good[2]), got):
            assert np.array_equal(w, g)
