"""GPU: page bookkeeping (dspark_pages_reserve, dspark_pages_commit) and cache
writes (dspark_cache_write) against the oracle, exactly: integers, copied bf16
bits and e4m3 values are the same or wrong.  Batches that do not fit change
nothing and raise the error flag; calls that the host checks refuse enqueue
nothing."""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def books(rng, B, gamma, page, hi, spare, stride_pad=0):
    """Random page books: lengths from 0 to hi, pages held for them in random order."""
    length = rng.randint(0, hi + 1, B)
    length[0] = 0
    if B > 2:
        length[1], length[2] = min(hi, page), hi                 # a full page, the longest
    K = rng.randint(-1, gamma + 1, B)
    held = -(-length // page)
    need = -(-(length + K + 1) // page)
    n_pages = int(np.maximum(need, held).sum()) + spare
    cols = int(need.max()) + 2
    ids = rng.permutation(n_pages)
    table = np.full((B, cols + stride_pad), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.concatenate([ids[at:], np.full(at, -1)])
    return dict(length=length, K=K, held=held, table=table, cols=cols, free=free, n_free=n_pages - at,
                n_pages=n_pages, page=page)


CASES = [  # B, gamma, page size, longest length, spare pages, entries behind the last row, table padding
    (1, 0, 8, 0, 0, 0, 0),
    (1, 7, 16, 1000, 3, 0, 0),
    (3, 32, 8, 40, 0, 5, 3),
    (64, 7, 16, 700, 10, 1, 0),
    (65, 16, 1024, 5000, 0, 0, 1),
    (300, 7, 32, 3000, 1, 300, 0),
    (4096, 3, 8, 100, 9, 7, 0),
    (5, 4000, 64, 9000, 2, 2, 0),                                # prompts
]


@pytest.mark.parametrize("B,gamma,page,hi,spare,behind,pad", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve_and_commit_match_the_oracle(ctx, B, gamma, page, hi, spare, behind, pad, in_place):
    print(f"pages B={B} gamma={gamma} page={page} hi={hi} in_place={in_place}", flush=True)
    rng = np.random.RandomState(B + gamma)
    s = books(rng, B, gamma, page, hi, spare, pad)
    total = int((s["K"] + 1).sum())
    n_rows = total + behind
    want = oracle.pages_reserve(s["K"], s["length"], s["table"], s["held"], s["free"], s["n_free"], page, n_rows)
    table, held, n_free = dev(s["table"]), dev(s["held"]), dev([s["n_free"]])
    held_in, free = dev(s["held"]), dev(s["free"])
    extra = {} if in_place else dict(held_out=torch.empty_like(held), n_free_out=torch.empty_like(n_free))
    for _ in range(1 if in_place else 2):                        # not in place: the same call twice, the same answer
        offs, req, pos, slot = ctx.pages_reserve(dev(s["K"]), dev(s["length"]), table[:, :s["cols"]], held, free, n_free,
                                                 page, s["n_pages"], n_rows=n_rows, **extra)
    ctx.check()
    got = [offs, req, pos, slot, table, extra.get("held_out", held), extra.get("n_free_out", n_free)]
    for name, w, g in zip(("offs", "req", "pos", "slot", "table", "held", "n_free"), want, got):
        assert np.array_equal(np.asarray(w).reshape(-1), g.cpu().numpy().reshape(-1)), name
    if not in_place:
        assert torch.equal(held, held_in) and n_free.item() == s["n_free"]
    assert torch.equal(free, dev(s["free"]))

    _, _, _, _, t2, h2, top = want
    acc = np.array([rng.randint(-1, k + 1) for k in s["K"]])
    fin = (rng.rand(B) < 0.2).astype(np.int32)
    for finished in (None, fin):
        wl, wh, wf, wt = oracle.pages_commit(s["length"], acc, t2, h2, s["free"], top, page, finished)
        length, held, n_free, free = dev(s["length"]), dev(h2), dev([top]), dev(s["free"])
        outs = {} if in_place else dict(len_out=torch.empty_like(length), held_out=torch.empty_like(held),
                                        n_free_out=torch.empty_like(n_free))
        ctx.pages_commit(length, dev(acc), dev(t2)[:, :s["cols"]], held, free, n_free, page, s["n_pages"],
                         finished=None if finished is None else dev(finished), **outs)
        ctx.check()
        assert np.array_equal(wl, outs.get("len_out", length).cpu().numpy())
        assert np.array_equal(wh, outs.get("held_out", held).cpu().numpy())
        assert outs.get("n_free_out", n_free).item() == wt
        assert np.array_equal(wf, free.cpu().numpy())


def _refused(ctx, s, n_rows, word):
    table, held, n_free, free = dev(s["table"]), dev(s["held"]), dev([s["n_free"]]), dev(s["free"])
    offs, req, pos, slot = ctx.pages_reserve(dev(s["K"]), dev(s["length"]), table, held, free, n_free, s["page"],
                                             s["n_pages"], n_rows=n_rows)
    with pytest.raises(dk.DSparkError, match=word) as e:
        ctx.check()
    assert e.value.code == dk.DSPARK_EDEVICE
    assert torch.equal(table, dev(s["table"])) and torch.equal(held, dev(s["held"])) and n_free.item() == s["n_free"]
    assert not offs.any() and (req == -1).all() and (pos == -1).all() and (slot == -1).all()


def test_a_batch_that_does_not_fit_changes_nothing(ctx):
    rng = np.random.RandomState(7)
    s = books(rng, 40, 7, 8, 60, 0)
    s["K"][:] = 7
    rows = 40 * 8
    need = int((-(-(s["length"] + 8) // 8) - s["held"]).sum())
    assert s["n_free"] < need
    _refused(ctx, s, rows, "page pool")
    s = books(rng, 40, 7, 8, 60, 400)
    fits = int((s["K"] + 1).sum())
    _refused(ctx, s, fits - 1, "out of range")
    for field, b, value in (("K", 3, -2), ("length", 5, -1), ("held", 0, -1), ("held", 9, 1000), ("K", 11, 10 ** 6),
                            ("K", 0, 2 ** 31 - 1), ("length", 0, 2 ** 31 - 1)):
        t = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
        t[field][b] = value
        _refused(ctx, t, fits, "out of range")
    t = dict(s, n_free=-1)
    _refused(ctx, t, fits, "page pool")
    t = dict(s, n_free=s["n_pages"] + 1)
    _refused(ctx, t, fits, "page pool")


def test_a_bad_page_id_is_flagged_and_its_rows_have_no_slot(ctx):
    table = dev([[2, 99, -1]])
    offs, req, pos, slot = ctx.pages_reserve(dev([3]), dev([13]), table, dev([2]), dev([0] * 8), dev([3]), 8, 8,
                                             n_rows=4)
    with pytest.raises(dk.DSparkError, match="page id"):
        ctx.check()
    assert slot.tolist() == [-1, -1, -1, 0] and pos.tolist() == [13, 14, 15, 16] and table.tolist() == [[2, 99, 0]]


def test_commit_refuses_what_cannot_be(ctx):
    length, held, table = [6, 20], [2, 3], [[1, 2, -1], [3, 4, 5]]
    for acc, lens, hold, n_free, word in (([-2, 0], length, held, 0, "out of range"), ([0, 4], length, held, 0, "out of range"),
                                          ([0, 0], [-1, 20], held, 0, "out of range"), ([0, 0], length, [2, 4], 0, "out of range"),
                                          ([0, 0], length, held, 6, "page pool"), ([0, 0], length, held, -1, "page pool")):
        ln, hd, nf, free = dev(lens), dev(hold), dev([n_free]), dev([7, 7, 7, 7, 7, 7])
        ctx.pages_commit(ln, dev(acc), dev(table), hd, free, nf, 8, 6)
        with pytest.raises(dk.DSparkError, match=word):
            ctx.check()
        assert ln.tolist() == lens and hd.tolist() == hold and nf.item() == n_free and free.tolist() == [7] * 6


# ---------------------------------------------------------------------------
# cache writes
# ---------------------------------------------------------------------------
WRITES = [  # rows, heads, d, page, order, 8-bit
    (1, 1, 64, 8, "token", False),
    (1, 1, 64, 8, "head", True),
    (9, 3, 128, 16, "token", True),
    (100, 8, 128, 16, "head", False),
    (257, 5, 256, 32, "token", False),
    (33, 16, 64, 64, "head", True),
    (1025, 2, 256, 128, "token", True),
]


def make_cache(rng, n_pages, page, heads, d, order, eight):
    shape = (n_pages, page, heads, d) if order == "token" else (n_pages, heads, page, d)
    x = torch.from_numpy(rng.randn(*shape).astype(np.float32))
    x = x.to(torch.float8_e4m3fn) if eight else x.to(torch.bfloat16)
    x = x.cuda()
    return x if order == "token" else x.permute(0, 2, 1, 3)


@pytest.mark.parametrize("n,heads,d,page,order,eight", WRITES)
def test_cache_write_matches_the_oracle(ctx, n, heads, d, page, order, eight):
    print(f"write n={n} heads={heads} d={d} page={page} {order} 8bit={eight}", flush=True)
    rng = np.random.RandomState(n)
    n_pages = n // page + 4
    kc, vc = make_cache(rng, n_pages, page, heads, d, order, eight), make_cache(rng, n_pages, page, heads, d, order, eight)
    before = [c.float().cpu().double().numpy() for c in (kc, vc)]
    slot = rng.permutation(n_pages * page)[:n]
    slot[::7] = -1
    qkv = torch.from_numpy((rng.randn(n, 3, heads, d) * rng.choice([1e-3, 1, 300], (n, 3, 1, 1))).astype(np.float32))
    qkv = qkv.to(torch.bfloat16).cuda()
    k, v = qkv[:, 1], qkv[:, 2]
    scales = [torch.from_numpy((rng.rand(heads) + 0.1).astype(np.float32)).cuda() for _ in range(2)] if eight else [None] * 2
    ctx.cache_write(k, v, dev(slot), kc, vc, k_scale=scales[0], v_scale=scales[1])
    ctx.check()
    for cache, was, x, scale in zip((kc, vc), before, (k, v), scales):
        want = was.copy()
        x = x.float().cpu().double().numpy()
        if eight:
            # in exact arithmetic the quotient is irrational-like: float64 stands 2^-29 closer than any border
            x = oracle.to_e4m3(x / scale.cpu().double().numpy()[None, :, None])
        for r in np.flatnonzero(slot >= 0):
            want[slot[r] // page, slot[r] % page] = x[r]
        assert np.array_equal(cache.float().cpu().double().numpy(), want)


def test_every_bf16_value_rounds_to_its_e4m3_value(ctx):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(1024, 1, 64)
    for scale in (None, 1.0, 0.0625, 3.0, 0.7, 1.1e-3):
        kc = torch.zeros((128, 8, 1, 64), dtype=torch.float8_e4m3fn, device="cuda")
        vc = torch.zeros_like(kc)
        sc = None if scale is None else torch.tensor([scale], device="cuda")
        ctx.cache_write(bits.cuda(), bits.cuda(), dev(np.arange(1024)), kc, vc, k_scale=sc, v_scale=sc)
        ctx.check()
        with np.errstate(invalid="ignore", over="ignore"):
            x = bits.float().double().numpy().reshape(-1) / (1.0 if sc is None else sc.cpu().double().item())
        want = oracle.to_e4m3(x)
        for c in (kc, vc):
            got = c.float().cpu().double().numpy().reshape(-1)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)]), scale


def test_a_quotient_next_to_a_border_is_rounded_once(ctx):
    """x / s just beside the middle of two e4m3 values, nearer than a float's half step: s = x / m (1 +- 2^-24 ..) for
    the middles m, x of 8 bits.  Checked in exact integer arithmetic."""
    from fractions import Fraction
    lv = oracle.e4m3_levels()
    rows, scales = [], []
    for i in range(8, 120, 3):
        m = (lv[i] + lv[i + 1]) / 2
        for x in (1.0, 1.2421875, 1.7890625):
            s = np.float32(x / m)
            for t in (s, np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(1e9))):
                rows.append(x)
                scales.append(t)
    H = len(rows)
    x = torch.tensor(rows, dtype=torch.bfloat16)
    assert np.array_equal(x.double().numpy(), np.array(rows))
    k = x.view(1, H, 1).expand(1, H, 64).contiguous().cuda()
    sc = torch.from_numpy(np.array(scales, dtype=np.float32)).cuda()
    kc = torch.zeros((1, 8, H, 64), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    ctx.cache_write(k, -k, dev([3]), kc, vc, k_scale=sc, v_scale=sc)
    ctx.check()
    got_k, got_v = kc[0, 3, :, 0].float().cpu().numpy(), vc[0, 3, :, 63].float().cpu().numpy()
    near = 0
    for h in range(H):
        q = Fraction(float(rows[h])) / Fraction(float(scales[h]))
        best = min(range(127), key=lambda c: (abs(Fraction(float(lv[c])) - q), c % 2))
        assert got_k[h] == lv[best] and got_v[h] == -lv[best], (rows[h], scales[h])
        near += abs(float(q / Fraction(float((lv[best] + lv[min(126, best + 1)]) / 2)) - 1)) < 2.0 ** -24
    assert near > 0


def test_bad_slots_are_flagged_and_skipped(ctx):
    kc = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    ctx.cache_write(x, x, dev([32, 5, -2, 2 ** 31 - 1]), kc, vc)
    with pytest.raises(dk.DSparkError, match="cache slot"):
        ctx.check()
    assert (kc.sum(), vc.sum()) == (128, 128) and (kc[0, 5] == 1).all()


def test_empty_write(ctx):
    kc = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    ctx.cache_write(x, x, dev(np.zeros(0)), kc, kc.clone())
    ctx.check()


def test_refusals(ctx):
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    good = dict(K=i(2), length=i(2), table=i(2, 3), held=i(2), free_list=i(6), n_free=i(1), page_size=8, n_pages=6, n_rows=4)
    for change, error in ((dict(page_size=12), dk.DSparkError), (dict(page_size=4), dk.DSparkError),
                          (dict(page_size=2048), dk.DSparkError), (dict(n_pages=0, free_list=i(0)), dk.DSparkError),
                          (dict(n_rows=-1, out=(i(3), i(4), i(4), i(4))), ValueError), (dict(length=i(3)), ValueError),
                          (dict(K=i(2).long()), TypeError), (dict(free_list=i(5)), ValueError),
                          (dict(table=i(3, 3)), ValueError), (dict(table=i(2, 0)), dk.DSparkError),
                          (dict(n_rows=None), ValueError), (dict(held=i(2).cpu()), ValueError)):
        with pytest.raises(error):
            ctx.pages_reserve(**{**good, **change})
    with pytest.raises(dk.DSparkError):
        ctx.pages_reserve(i(4097), i(4097), i(4097, 1), i(4097), i(6), i(1), 8, 6, n_rows=1)
    com = dict(length=i(2), accept_len=i(2), table=i(2, 3), held=i(2), free_list=i(6), n_free=i(1), page_size=8, n_pages=6)
    for change, error in ((dict(page_size=9), dk.DSparkError), (dict(accept_len=i(1)), ValueError),
                          (dict(finished=torch.zeros(2, dtype=torch.bool, device="cuda")), TypeError),
                          (dict(n_free=i(2)), ValueError)):
        with pytest.raises(error):
            ctx.pages_commit(**{**com, **change})
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    k, c = bf(2, 2, 64), bf(4, 8, 2, 64)
    for args, error in (((k.float(), k, i(2), c, c), TypeError), ((k, k, i(3), c, c), ValueError),
                        ((k, k, i(2), c.float(), c.float()), TypeError), ((k, k, i(2), bf(4, 8, 3, 64), c), ValueError),
                        ((bf(2, 2, 32), bf(2, 2, 32), i(2), bf(4, 8, 2, 32), bf(4, 8, 2, 32)), dk.DSparkError),
                        ((k, k, i(2), bf(4, 12, 2, 64), bf(4, 12, 2, 64)), dk.DSparkError),
                        ((k, k, i(2), bf(4, 8, 2, 68)[..., :64], bf(4, 8, 2, 68)[..., :64]), dk.DSparkError),
                        ((k, bf(2, 2, 68)[..., 2:66], i(2), c, c), dk.DSparkError),
                        ((k, k, i(2), bf(1, 8, 2, 64).expand(4, 8, 2, 64), bf(1, 8, 2, 64).expand(4, 8, 2, 64)), dk.DSparkError)):
        with pytest.raises(error):
            ctx.cache_write(*args)
    with pytest.raises(dk.DSparkError, match="scales"):
        ctx.cache_write(k, k, i(2), c, c.clone(), k_scale=torch.ones(2, device="cuda"))
    ctx.check()
