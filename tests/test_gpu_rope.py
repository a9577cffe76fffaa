"""GPU: rotary positions (dspark_rope, dspark_rope_write) against the oracle.

Tolerance of a turned value y = F (x0 cos - x1 sin) with N = |F| (|x0| + |x1|):
  2^-8 |y|           the result rounded to bf16
  4 * 2^-24 N        sine and cosine rounded to float32, a product and a sum
  t f 2^-51 N        the angle: two float64 products of a position and a frequency
Keys for a cache of few bits are turned in float64: a stored value is the nearest
one up to 2^-40 N (and the angle's error) of distance.
"""
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


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def f64(t):
    return t.float().cpu().double().numpy()


def frequencies(rot, kind=None):
    if kind == "yarn":
        return dk.rope_frequencies(rot, 500000.0, "yarn", 16.0, trained=4096, device="cuda")
    f, _ = dk.rope_frequencies(rot, 10000.0, device="cuda")
    return f, 0.75 if kind == "factor" else 1.0


def positions(rng, n):
    pos = rng.randint(0, 200000, n)
    for i, p in enumerate([0, 1, -1, 131071, 1 << 30, 2 ** 31 - 1]):
        if i < n - 1:
            pos[i] = p
    return pos


def bound(x, pos, freq, inter, factor):
    """N of every value, times 4 * 2^-24 and its angle's error."""
    n = len(freq)
    a = np.abs(x)
    N, extra = a.copy(), np.zeros_like(a)
    u, v = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if inter else (np.arange(n), np.arange(n, 2 * n))
    both = abs(factor) * (a[..., u] + a[..., v])
    N[..., u] = N[..., v] = both
    turn = np.maximum(pos, 0)[:, None, None] * freq[None, None] * 2.0 ** -51 * both
    extra[..., u] = extra[..., v] = turn
    return N, extra


def rows(g, n, heads, d, wide=True):
    """Rows that lie between others, as columns of a projection's output."""
    x = torch.randn((n, heads + (2 if wide else 0), d), generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    return x[:, 1:-1] if wide else x


CASES = [  # rows, query heads, heads, d, rot, interleaved, kind
    (1, 32, 8, 128, 128, False, None),
    (1, 1, 1, 16, 16, True, None),
    (7, 3, 1, 64, 64, True, "yarn"),
    (9, 5, 0, 80, 32, False, None),
    (13, 0, 3, 96, 96, False, "factor"),
    (33, 4, 2, 256, 64, True, "factor"),
    (50, 2, 2, 24, 16, False, None),
    (130, 7, 5, 192, 48, False, "yarn"),
    (5, 2, 1, 1024, 1024, False, None),
    (3, 1, 2, 1000, 16, True, None),
    (2500, 2, 1, 64, 32, False, None),
    (4200, 1, 1, 128, 128, True, "yarn"),
]


@pytest.mark.parametrize("n,hq,h,d,rot,inter,kind", CASES)
def test_rows_are_turned(ctx, n, hq, h, d, rot, inter, kind):
    print(f"rope n={n} heads={hq},{h} d={d} rot={rot} interleaved={inter} {kind}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    pos = positions(np.random.RandomState(n), n)
    freq, factor = frequencies(rot, kind)
    q, k = rows(g, n, hq, d) if hq else None, rows(g, n, h, d, False) if h else None
    out = ctx.rope(q, k, i32(pos), freq, interleaved=inter, factor=factor)
    ctx.check()
    few = np.unique(np.r_[np.arange(min(n, 40)), np.arange(max(0, n - 20), n)])      # the oracle's rows
    for x, y in zip((q, k), out):
        if x is None:
            assert y is None
            continue
        x0, y0 = f64(x)[few], f64(y)[few]
        want = oracle.rope(x0, pos[few], freq.cpu().numpy(), inter, factor)
        N, extra = bound(x0, pos[few], freq.cpu().numpy(), inter, factor)
        live = pos[few] >= 0
        tol = 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -24 * N + extra
        assert (np.abs(y0 - want)[live] <= tol[live]).all()
        assert np.array_equal(y0[live][..., rot:], x0[live][..., rot:])
        assert (y0[~live] == 0).all()
    # all rows, in place: the same bits; rows of position -1 stay
    inp = [None if x is None else x.clone() for x in (q, k)]
    ctx.rope(*inp, i32(pos), freq, interleaved=inter, factor=factor, q_out=inp[0], k_out=inp[1])
    ctx.check()
    live = torch.from_numpy(pos >= 0).cuda()
    for x, y, z in zip((q, k), out, inp):
        if x is not None:
            assert torch.equal(z[live], y[live]) and torch.equal(z[~live], x[~live])


def test_one_side_in_place_and_the_other_apart(ctx):
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = rows(g, 20, 4, 64), rows(g, 20, 2, 64)
    pos, (freq, _) = i32(np.arange(20) * 77), frequencies(32)
    a, b = ctx.rope(q, k, pos, freq)
    q2 = q.clone()
    _, k_out = ctx.rope(q2, k, pos, freq, q_out=q2)
    ctx.check()
    assert torch.equal(q2, a) and torch.equal(k_out, b)


def test_infinities_and_nan_stay_in_their_pair(ctx):
    g = torch.Generator(device="cuda").manual_seed(4)
    for inter in (False, True):
        q = rows(g, 3, 2, 64, False)
        want, _ = ctx.rope(q, None, i32([5, 6, 7]), frequencies(32)[0], interleaved=inter)
        bad = q.clone()
        bad[1, 1, 3], bad[2, 0, 40] = float("inf"), float("nan")
        got, _ = ctx.rope(bad, None, i32([5, 6, 7]), frequencies(32)[0], interleaved=inter)
        ctx.check()
        hit = torch.zeros_like(q, dtype=torch.bool)
        hit[1, 1, [2, 3] if inter else [3, 19]] = True
        hit[2, 0, 40] = True
        assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], want[~hit])


def four_bit_cache(n_pages, page, h, d, order):
    shape = (n_pages, page, h, d // 2) if order == "token" else (n_pages, h, page, d // 2)
    c = [torch.full(shape, 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2)]
    c = [x if order == "token" else x.permute(0, 2, 1, 3) for x in c]
    return c, [torch.full((n_pages, h, page, d // 32), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]


def caches(kv, n_pages, page, h, d, order):
    """kcache, vcache, k_scale, v_scale with something in every place."""
    if kv == "mxfp4":
        c, p = four_bit_cache(n_pages, page, h, d, order)
        return (*c, *p)
    shape = (n_pages, page, h, d) if order == "token" else (n_pages, h, page, d)
    c = [torch.full(shape, 3.0, device="cuda").to(torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn) for _ in range(2)]
    c = [x if order == "token" else x.permute(0, 2, 1, 3) for x in c]
    if kv == "bf16":
        return (*c, None, None)
    g = torch.Generator(device="cuda").manual_seed(h)
    return (*c, *[(torch.rand(h, generator=g, device="cuda") + 0.5) / 40 for _ in range(2)])


def codes_of(cache):
    """MXFP4 codes [n_pages][page][heads][d] of a cache."""
    b = cache.cpu().numpy()
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def values(cache, scale):
    """What a cache stands for, [n_pages][page][heads][d] in float64."""
    if cache.dtype == torch.uint8:
        return oracle.from_mxfp4(codes_of(cache), scale.cpu().numpy().transpose(0, 2, 1, 3))
    x = f64(cache)
    return x if scale is None else x * f64(scale)[:, None]


WRITES = [  # rows, query heads, heads, d, rot, interleaved, page, order, kind
    (1, 4, 1, 128, 128, False, 16, "token", None),
    (9, 0, 3, 64, 64, True, 8, "head", "yarn"),
    (37, 6, 2, 64, 32, False, 32, "token", "factor"),
    (20, 2, 2, 256, 256, False, 64, "head", None),
    (26, 3, 1, 256, 48, True, 16, "token", "yarn"),
    (60, 1, 5, 128, 48, False, 128, "head", None),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("n,hq,h,d,rot,inter,page,order,kind", WRITES)
def test_turned_keys_and_values_go_to_their_slots(ctx, kv, n, hq, h, d, rot, inter, page, order, kind):
    print(f"rope_write {kv} n={n} heads={hq},{h} d={d} rot={rot} {inter} page={page} {order} {kind}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.RandomState(n)
    pos = positions(rng, n)
    n_pages = n // page + 3
    slot = rng.permutation(n_pages * page)[:n]
    if n > 8:
        slot[7] = -1
    freq, factor = frequencies(rot, kind)
    q = rows(g, n, hq, d) if hq else None
    k, v = rows(g, n, h, d), rows(g, n, h, d)
    k[-1] *= 2.0 ** -30                                  # small keys among large ones
    kc, vc, ks, vs = caches(kv, n_pages, page, h, d, order)
    before = [values(kc, ks), values(vc, vs)]
    got_q = ctx.rope_write(q, k, v, i32(pos), i32(slot), freq, kc, vc, ks, vs, interleaved=inter, factor=factor)
    ctx.check()
    want_q, turned = ctx.rope(q, k, i32(pos), freq, interleaved=inter, factor=factor)
    assert (got_q is None) if q is None else torch.equal(got_q, want_q)
    live = (pos >= 0) & (slot >= 0)
    at = (slot[live] // page, slot[live] % page)
    after = [values(kc, ks), values(vc, vs)]
    rest = np.ones((n_pages, page), dtype=bool)
    rest[at] = False
    for a, b in zip(before, after):
        assert np.array_equal(a[rest], b[rest])          # nothing else is touched
    exact_k, exact_v = oracle.rope(f64(k), pos, freq.cpu().numpy(), inter, factor)[live], f64(v)[live]
    if kv == "bf16":
        assert np.array_equal(after[0][at], f64(turned)[live]) and np.array_equal(after[1][at], exact_v)
        return
    slack, extra = bound(f64(k), pos, freq.cpu().numpy(), inter, factor)
    slack = (2.0 ** -40 * slack + extra)[live]
    if kv == "e4m3":
        for x, scale, a, s in ((exact_k, ks, after[0], slack), (exact_v, vs, after[1], 0)):
            scale = f64(scale)[None, :, None]
            nearest = oracle.to_e4m3(x / scale) * scale
            assert (np.abs(a[at] - x) <= np.abs(nearest - x) * (1 + 1e-12) + s).all()
        return
    byte = [p.cpu().numpy().transpose(0, 2, 1, 3)[at] for p in (ks, vs)]
    code, power = oracle.to_mxfp4(exact_v)
    assert np.array_equal(byte[1], power) and np.array_equal(codes_of(vc)[at], code)
    code, power = oracle.to_mxfp4(exact_k)
    near = np.abs(oracle.from_mxfp4(code, power) - exact_k)
    assert np.array_equal(byte[0], power)                # (no largest value lies within its slack of a border here)
    assert (np.abs(after[0][at] - exact_k) <= near * (1 + 1e-12) + slack).all()


def test_positions_and_slots_that_are_none(ctx):
    """Bad positions and slots are flagged, their rows left; the others are as without them."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = rows(g, 6, 2, 64), rows(g, 6, 1, 64), rows(g, 6, 1, 64)
    freq, _ = frequencies(64)
    good, slot = i32([4, 9, -1, 7, 8, 3]), i32([0, 5, 2, -1, 3, 1])
    kc, vc, ks, vs = caches("mxfp4", 2, 8, 1, 64, "token")
    want = ctx.rope_write(q, k, v, good, slot, freq, kc, vc, ks, vs)
    ctx.check()
    for pos, s in (([4, 9, -7, 7, 8, 3], [0, 5, 2, -1, 3, 1]), ([4, 9, -1, 7, 8, 3], [0, 5, 16, -1, 3, 1]),
                   ([4, 9, -1, 7, 8, 3], [0, 5, 2, 16, 3, 1]), ([4, 9, -1, 7, 8, 3], [0, 5, 2, -2, 3, 1])):
        k2, v2, a, b = caches("mxfp4", 2, 8, 1, 64, "token")
        out = ctx.rope_write(q, k, v, i32(pos), i32(s), freq, k2, v2, a, b)
        if pos[2] == -7 or s[3] != -1:
            with pytest.raises(dk.DSparkError, match="position" if pos[2] == -7 else "slot"):
                ctx.check()
        else:
            ctx.check()                                  # the row has no position: its slot is not read
        assert torch.equal(out, want)
        for x, y in zip((k2, v2, a, b), (kc, vc, ks, vs)):
            assert torch.equal(x, y)
    with pytest.raises(dk.DSparkError, match="position"):
        ctx.rope(q, None, i32([4, 9, -2, 7, 8, 3]), freq)
        ctx.check()


def refused(f, match):
    with pytest.raises((dk.DSparkError, ValueError, TypeError), match=match):
        f()


def test_refusals(ctx):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = rows(g, 4, 2, 64), rows(g, 4, 1, 64), rows(g, 4, 1, 64)
    pos, freq = i32([0, 1, 2, 3]), frequencies(64)[0]
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    refused(lambda: ctx.rope(q, k, pos[:3], freq), "n_rows")
    refused(lambda: ctx.rope(q, k, pos, freq.float()), "freq")
    refused(lambda: ctx.rope(q, k, pos, freq[:5]), "rot")
    refused(lambda: ctx.rope(q, k, pos, torch.cat([freq, freq])), "rot")
    refused(lambda: ctx.rope(q, k, pos, freq, factor=float("nan")), "factor")
    refused(lambda: ctx.rope(z(4, 2, 12), None, pos, freq[:8]), "head size")
    refused(lambda: ctx.rope(z(4, 2, 1032), None, pos, freq), "head size")
    refused(lambda: ctx.rope(q, k, pos, freq, q_out=z(4, 3, 64)), "q_out")
    refused(lambda: ctx.rope(q, k, pos, freq, q_out=q[:, :, :].transpose(0, 1)[:, :].transpose(0, 1)[:, :1]), "q_out")
    refused(lambda: ctx.rope(k, k, pos, freq, q_out=k), "q_out")
    same = z(4, 1, 64)
    refused(lambda: ctx.rope(k, v, pos, freq, q_out=same, k_out=same), "q_out")
    refused(lambda: ctx.rope(z(4, 2, 64), None, pos, freq, q_out=z(4, 1, 64).expand(4, 2, 64)), "overlap")
    refused(lambda: ctx.rope(z(4, 2, 72)[:, :, 4:68], None, pos, freq), "16-byte")
    refused(lambda: ctx.rope(None, None, pos, freq), "q must")
    kc, vc, ks, vs = caches("mxfp4", 2, 8, 1, 64, "token")
    slot = i32([0, 1, 2, 3])
    refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, kc, vc), "k_scale")
    refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, kc, vc, ks, ks), "powers")
    refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, kc, vc, ks[:1], vs), "k_scale")
    refused(lambda: ctx.rope_write(q, k, v, pos, slot[:3], freq, kc, vc, ks, vs), "row_slot")
    refused(lambda: ctx.rope_write(q, k, v[:3], pos, slot, freq, kc, vc, ks, vs), "k and v")
    refused(lambda: ctx.rope_write(k, k, v, pos, slot, freq, kc, vc, ks, vs, q_out=v), "q_out")
    b = caches("bf16", 2, 8, 1, 64, "token")
    refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, *b[:2], torch.ones(1, device="cuda")), "scales")
    none = ctx.rope(q[:0], k[:0], pos[:0], freq)
    assert none[0].shape == (0, 2, 64)
    ctx.rope_write(q[:0], k[:0], v[:0], pos[:0], slot[:0], freq, kc, vc, ks, vs)
    ctx.check()


def test_another_stream_and_a_captured_graph(ctx):
    """On a stream of its own, captured once and replayed over changing inputs, with eager work between."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n = 300
    q, k, v = rows(g, n, 4, 128), rows(g, n, 2, 128), rows(g, n, 2, 128)
    pos, slot, (freq, _) = i32(np.arange(n) * 11), i32(np.arange(n)[::-1].copy()), frequencies(128)
    kc, vc, ks, vs = caches("mxfp4", 40, 8, 2, 128, "token")
    back = [torch.zeros((n, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q_out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        ctx.rope_write(q, k, v, pos, slot, freq, kc, vc, ks, vs, q_out=q_out)
        ctx.cache_read(kc, vc, slot, ks, vs, out=back)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        x = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
        q.copy_(x)
        k.copy_(x[:, :2] * 3)
        v.copy_(x[:, 2:] * 0.1)
        pos.add_(1000)
        for t in (kc, vc, ks, vs):                       # (20 slots that no row has)
            t.zero_()
        step()
        eager = [t.clone() for t in (q_out, *back, kc, vc, ks, vs)]
        for t in (q_out, *back, kc, vc, ks, vs):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all([torch.equal(a, b) for a, b in zip(eager, (q_out, *back, kc, vc, ks, vs))])
    ctx.check()


def test_timing_class_and_many_rows(ctx):
    """Counted as launches of the rope class; more rows than a workgroup each would have threads for."""
    n = (1 << 23) + 5
    q = torch.ones((n, 1, 16), dtype=torch.bfloat16, device="cuda")
    q[n - 1] = 2
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[n - 1] = 3
    freq = torch.full((8,), np.pi / 2, dtype=torch.float64, device="cuda")
    ctx.timing(True)
    ctx.read_timing()
    ctx.rope(q, None, pos, freq, q_out=q)
    assert ctx.read_timing()["rope"][1] == 1
    ctx.timing(False)
    ctx.check()
    assert (q[:-1] == 1).all()
    assert torch.equal(q[n - 1, 0], torch.tensor([2.0] * 8 + [-2.0] * 8, dtype=torch.bfloat16, device="cuda"))
    wide = torch.ones((1, 1, 1024), dtype=torch.bfloat16, device="cuda").expand(n, 1, 1024)
    refused(lambda: ctx.rope(wide, None, pos, torch.zeros(512, dtype=torch.float64, device="cuda"),
                             q_out=torch.empty((n, 1, 1024), dtype=torch.bfloat16, device="cuda")), "too many rows")


@pytest.mark.parametrize("kv", ["e4m3", "mxfp4"])
@pytest.mark.parametrize("inter", [False, True])
def test_at_position_0_keys_are_rounded_as_the_cache_write_rounds_them(ctx, kv, inter):
    """Every finite bf16 value, borders of the quotients with a scale that is no power of two among them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[torch.isfinite(bits.float())]
    n = len(bits) // 32                                  # 65024 values
    k = torch.zeros((n, 1, 64), dtype=torch.bfloat16)
    if inter:
        k[:, 0, 0::2] = bits.view(n, 32)
    else:
        k[:, 0, :32] = bits.view(n, 32)
    k = k.cuda()
    pages = n // 64 + 1
    a, b = caches(kv, pages, 64, 1, 64, "token"), caches(kv, pages, 64, 1, 64, "token")
    if kv == "e4m3":
        scale = torch.tensor([0.75 * 1.25], device="cuda")
        a, b = (*a[:2], scale, scale), (*b[:2], scale, scale)
    slot, pos = i32(np.arange(n)), torch.zeros(n, dtype=torch.int32, device="cuda")
    ctx.cache_write(k, k, slot, *a)
    ctx.rope_write(None, k, k, pos, slot, frequencies(64)[0], *b, interleaved=inter)
    ctx.check()
    for x, y, s in ((a[0], b[0], 2), (a[1], b[1], 3)):
        assert np.array_equal(values(x, a[s]), values(y, b[s]))
    if kv == "mxfp4":
        assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
