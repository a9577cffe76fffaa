"""GPU: attention of packed rows over the paged cache (dspark_attend) against
the float64 oracle.

Tolerance of an output value o = sum p v / sum p with A = sum p |v| / sum p:
  2^-8 |o|                the result rounded to bf16
  2^-8 A                  every weight rounded to bf16 before its product
  (2 ds + n 2^-24 + 2^-20) A   weights: ds bounds a score's error (float32 sum
                          of D exact products, (D + 4) 2^-24 scale sum |q k|,
                          a relative error of p), n terms summed in float32, a
                          few units of the hardware exponential
and of a log-sum-exp: ds + n 2^-24 + 2^-20 (1 + |lse|).
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


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def f64(t):
    return None if t is None else t.float().cpu().double().numpy()


def make(seed, length, K, heads, group, d, page, order="token", eight=False, spread=1.5):
    """Random books, cache and queries; queries are the middle columns of a wider tensor."""
    rng = np.random.RandomState(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    length, K = np.array(length), np.array(K)
    B = len(length)
    held = -(-(length + K + 1) // page)
    n_pages = int(held.sum()) + 2
    table = np.full((B, int(held.max()) + 1), -1)
    ids = rng.permutation(n_pages)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    shape = (n_pages, page, heads, d) if order == "token" else (n_pages, heads, page, d)

    def cache():
        x = torch.randn(shape, generator=g, device="cuda")
        x = (x * 50).clamp(-448, 448).to(torch.float8_e4m3fn) if eight else x.to(torch.bfloat16)
        return x if order == "token" else x.permute(0, 2, 1, 3)

    rows = int((K + 1).sum())
    wide = torch.randn((rows, heads * group + 2, d), generator=g, device="cuda").mul_(spread).to(torch.bfloat16)
    s = dict(q=wide[:, 1:-1], kc=cache(), vc=cache(), table=table, length=length, K=K,
             offs=np.concatenate([[0], np.cumsum(K + 1)]), ks=None, vs=None, scale=d ** -0.5)
    if eight:
        s["ks"], s["vs"] = [(torch.rand(heads, generator=g, device="cuda") + 0.5) / 50 for _ in range(2)]
    return s


def call(ctx, s, causal=True, **kw):
    out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    kw = {**dict(K=dev(s["K"]), t_offsets=dev(s["offs"]), out=out, lse=lse), **kw}
    gamma = kw.pop("gamma", max(0, int(s["K"].max())))
    ctx.attend(s["q"], s["kc"], s["vc"], dev(s["table"]), dev(s["length"]), gamma, causal=causal, scale=s["scale"],
               k_scale=s["ks"], v_scale=s["vs"], **kw)
    return kw["out"], kw["lse"]


def check(s, out, lse, causal=True):
    q, kc, vc = f64(s["q"]), f64(s["kc"]), f64(s["vc"])
    ks, vs = f64(s["ks"]), f64(s["vs"])
    args = (s["table"], s["length"], s["K"], s["offs"])
    how = dict(causal=causal, scale=s["scale"], k_scale=ks, v_scale=vs)
    want, wl = oracle.attend(q, kc, vc, *args, **how)
    mean, _ = oracle.attend(q, kc, np.abs(vc), *args, **how)
    n, D = int((s["length"] + s["K"]).max()) + 1, q.shape[2]
    top = np.abs(np.where(np.isfinite(kc), kc, 0)).max(axis=(0, 1)) * (1.0 if ks is None else ks[:, None])   # [H][D]
    group = q.shape[1] // kc.shape[2]
    ds = (D + 4) * 2.0 ** -24 * s["scale"] * np.abs(q * np.repeat(top, group, 0)).sum(2)
    out, lse = f64(out), f64(lse)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * ds[..., None] + n * 2.0 ** -24 + 2.0 ** -20) * mean
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(out), fine), "infinities or NaN in other places than the oracle's"
    assert np.array_equal(np.isnan(out), np.isnan(want))
    worst = (np.abs(out - want)[fine] / tol[fine]).max() if fine.any() else 0.0
    assert worst <= 1.0, worst
    tl = ds + n * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(wl))
    ok = np.isfinite(wl)
    assert np.array_equal(np.isnan(lse), np.isnan(wl))
    assert (np.abs(lse - wl)[ok] <= tl[ok]).all()
    return worst


LENGTHS = [0, 1, 7, 15, 16, 31, 32, 100, 126, 127, 128, 129, 300]

CASES = [  # heads, group, d, page, order, 8-bit, gamma
    (2, 1, 64, 8, "token", False, 0),
    (1, 4, 128, 16, "token", False, 0),
    (2, 4, 128, 16, "head", False, 7),
    (3, 5, 64, 32, "token", False, 3),
    (1, 8, 128, 64, "head", True, 7),
    (2, 2, 64, 16, "token", True, 16),
    (1, 16, 256, 128, "token", False, 1),
    (2, 3, 256, 8, "head", True, 6),
    (1, 1, 128, 1024, "token", True, 32),
    (1, 9, 128, 16, "token", False, 32),
    (1, 64, 64, 16, "token", False, 2),
    (5, 1, 256, 32, "token", True, 0),
]


@pytest.mark.parametrize("heads,group,d,page,order,eight,gamma", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_the_oracle(ctx, heads, group, d, page, order, eight, gamma, causal):
    print(f"attend heads={heads} group={group} d={d} page={page} {order} 8bit={eight} gamma={gamma} {causal}", flush=True)
    rng = np.random.RandomState(gamma + d)
    K = [gamma, 0, -1] + [int(k) for k in rng.randint(-1, gamma + 1, len(LENGTHS) - 3)]
    s = make(1 + d, LENGTHS, K, heads, group, d, page, order, eight)
    out, lse = call(ctx, s, causal)
    ctx.check()
    print("worst error over its bound: %.3f" % check(s, out, lse, causal))
    again, lse2 = call(ctx, s, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("length,gamma,heads,group,d,eight", [(5000, 0, 1, 1, 128, False), (9001, 3, 2, 4, 128, True),
                                                              (20000, 7, 1, 2, 64, False), (3333, 1, 1, 3, 256, True)])
def test_one_long_request_is_joined_from_many_pieces(ctx, length, gamma, heads, group, d, eight):
    print(f"attend length={length} gamma={gamma} heads={heads} d={d}", flush=True)
    s = make(3, [length], [gamma], heads, group, d, 16, "token", eight)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_long_and_short_requests_together(ctx):
    lengths = [12000, 0, 3, 0, 700, 64, 8000, 1, 2, 5]
    s = make(4, lengths, [1, 0, 1, -1, 0, 1, 0, 1, 1, 0], 1, 2, 128, 16)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_many_requests(ctx):
    rng = np.random.RandomState(8)
    s = make(5, rng.randint(0, 60, 1500), rng.randint(-1, 2, 1500), 1, 2, 64, 8)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_large_scores(ctx):
    """Scores of hundreds: one key takes all the weight, rows of every order of the maximum."""
    for spread in (30.0, 300.0):
        s = make(6, [200, 900, 31], [2, 0, 4], 2, 3, 128, 16, spread=spread)
        out, lse = call(ctx, s)
        ctx.check()
        check(s, out, lse)


def test_what_is_masked_has_no_effect(ctx):
    """NaN and infinities in unused places of pages, in free pages and, for the rows before them, in later drafts."""
    for eight in (False, True):
        for page, order in ((8, "token"), (64, "head")):
            s = make(7, [0, 13, 40, 127, 250], [3, 7, 5, 2, 6], 2, 2, 128, page, order, eight)
            used = torch.zeros(s["kc"].shape[:2], dtype=torch.bool)
            for b in range(5):
                for t in range(s["length"][b] + s["K"][b] + 1):
                    used[s["table"][b][t // page], t % page] = True
            nan = float("nan")
            for c in (s["kc"], s["vc"]):
                x = c.float()
                x[~used.cuda()] = nan
                c.copy_(x.to(c.dtype))
            out, lse = call(ctx, s)
            ctx.check()
            clean = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
            for name in ("kc", "vc"):
                clean[name] = torch.nan_to_num(s[name].float()).to(s[name].dtype)
            check(clean, out, lse)
            # a draft's own value or key is NaN or infinite: the rows before it are as they were
            for bad in ([nan] if eight else [nan, float("inf"), -float("inf")]):
                for name in ("kc", "vc"):
                    t2 = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in clean.items()}
                    for b, i in ((1, 4), (2, 5), (4, 1)):
                        t = s["length"][b] + i
                        x = t2[name].float()
                        x[s["table"][b][t // page], t % page, 1, 3:9] = bad
                        t2[name] = x.to(t2[name].dtype)
                    out2, lse2 = call(ctx, t2)
                    ctx.check()
                    for b, i in ((1, 4), (2, 5), (4, 1)):
                        lo, hi = s["offs"][b], s["offs"][b] + i
                        assert torch.equal(out2[lo:hi], out[lo:hi]) and torch.equal(lse2[lo:hi], lse[lo:hi])
                        assert torch.equal(out2[lo:s["offs"][b + 1], :2], out[lo:s["offs"][b + 1], :2])
                    if name == "vc":
                        # what sees it, and only at its places, is not finite
                        lo = s["offs"][1] + 4
                        assert not torch.isfinite(out2[lo:s["offs"][2], 2:, 3:9]).any()
                        assert torch.equal(out2[lo:s["offs"][2], 2:, 9:], out[lo:s["offs"][2], 2:, 9:])


def test_rows_of_no_request_are_left_as_they_were(ctx):
    s = make(9, [10, 20], [1, 0], 1, 2, 64, 8)
    q = torch.randn((9, 2, 64), device="cuda").to(torch.bfloat16)
    q[1:3], q[6:7] = s["q"][:2], s["q"][2:]
    s["q"], s["offs"] = q, np.array([1, 6])
    out, lse = call(ctx, s)
    ctx.check()
    rest = [0, 3, 4, 5, 7, 8]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()
    want, wl = oracle.attend(f64(q), f64(s["kc"]), f64(s["vc"]), s["table"], s["length"], s["K"], s["offs"],
                             scale=s["scale"])
    for r in (1, 2, 6):
        assert np.allclose(f64(out[r]), want[r], atol=0.05) and np.allclose(f64(lse[r]), wl[r], atol=1e-4)


def test_defaults_are_the_dense_layout(ctx):
    s = make(10, [5, 33, 64], [3, 3, 3], 2, 2, 128, 16)
    a, _ = call(ctx, s)
    b = ctx.attend(s["q"], s["kc"], s["vc"], dev(s["table"]), dev(s["length"]), 3)
    ctx.check()
    assert torch.equal(a, b)


def test_a_strided_result(ctx):
    s = make(11, [5, 70], [2, 1], 2, 2, 64, 16)
    a, _ = call(ctx, s)
    out = torch.full((4, 5, 72), 7.0, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)[..., 8:]
    got, _ = call(ctx, s, out=out)
    ctx.check()
    assert torch.equal(got, a)


def test_bad_numbers_are_flagged_and_the_rest_is_right(ctx):
    s = make(12, [10, 20, 30], [1, 1, 1], 1, 2, 64, 8)
    good, _ = call(ctx, s)
    for field, b, value, word in (("K", 1, 5, "verify length"), ("K", 0, -2, "verify length"), ("length", 1, -1, "cache length"),
                                  ("length", 2, 10 ** 6, "cache length"), ("length", 2, 2 ** 31 - 1, "cache length"),
                                  ("offs", 1, 5, "row out of range"), ("offs", 0, -1, "row out of range")):
        t = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
        t[field][b] = value
        out, _ = call(ctx, t, gamma=1)
        with pytest.raises(dk.DSparkError, match=word):
            ctx.check()
        for o in set(range(3)) - {b}:
            assert torch.equal(out[2 * o:2 * o + 2], good[2 * o:2 * o + 2]), (field, b, o)
        if field != "K" or value < 0:
            assert (out[2 * b:2 * b + 2] == 7).all()
    for bad in (99, -1, 2 ** 31 - 1):
        t = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
        t["table"][1][0] = bad
        out, _ = call(ctx, t, gamma=1)
        with pytest.raises(dk.DSparkError, match="page id"):
            ctx.check()
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])


def test_offsets_beyond_32_bits(ctx):
    """Pages whose places pass 2^32 bytes in the cache."""
    heads, d, page, n_pages = 2, 128, 64, 150_000                # 4.9 GB a cache
    kc = torch.empty((n_pages, page, heads, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    s = make(13, [150, 3], [2, 1], heads, 2, d, page)
    small = s["table"].copy()
    far = np.array([n_pages - 1, 70_000, 3, 140_001, 131_072, 9])
    for i, p in enumerate(sorted(set(small[small >= 0]))):
        kc[far[i]], vc[far[i]] = s["kc"][p], s["vc"][p]
        s["table"][small == p] = far[i]
    near, _ = call(ctx, {**s, "table": small})
    out, _ = call(ctx, {**s, "kc": kc, "vc": vc})
    ctx.check()
    assert torch.equal(out, near)
    slot = dev([int(far[0]) * page + 63, int(far[1]) * page])
    x = torch.randn((2, heads, d), device="cuda").to(torch.bfloat16)
    ctx.cache_write(x, -x, slot, kc, vc)
    ctx.check()
    assert torch.equal(kc[far[0], 63], x[0]) and torch.equal(vc[far[1], 0], -x[1])


def test_refusals(ctx):
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    c = bf(4, 8, 2, 64)
    good = dict(q=bf(2, 4, 64), kcache=c, vcache=c, table=i(2, 2), length=i(2), gamma=0)
    ctx.attend(**good)
    for change, error in ((dict(gamma=-1), dk.DSparkError), (dict(gamma=33, t_offsets=i(2)), dk.DSparkError),
                          (dict(gamma=1), dk.DSparkError), (dict(q=bf(2, 3, 64)), dk.DSparkError),
                          (dict(q=bf(2, 4, 128)), ValueError), (dict(q=bf(2, 130, 64)), dk.DSparkError),
                          (dict(q=torch.zeros(2, 4, 64, device="cuda")), TypeError),
                          (dict(q=bf(2, 4, 68)[..., 2:66]), dk.DSparkError), (dict(q=bf(2, 4, 66)[..., :64]), dk.DSparkError),
                          (dict(kcache=c.half(), vcache=c.half()), TypeError), (dict(vcache=bf(4, 8, 2, 128)), ValueError),
                          (dict(table=i(3, 2)), ValueError), (dict(length=i(2).long()), TypeError),
                          (dict(K=i(1)), ValueError), (dict(t_offsets=i(1)), ValueError), (dict(scale=0.0), dk.DSparkError),
                          (dict(scale=float("inf")), dk.DSparkError), (dict(scale=float("nan")), dk.DSparkError),
                          (dict(k_scale=torch.ones(2, device="cuda")), dk.DSparkError),
                          (dict(k_scale=torch.ones(3, device="cuda")), ValueError),
                          (dict(out=bf(1, 4, 64).expand(2, 4, 64)), dk.DSparkError), (dict(out=bf(2, 4, 32)), ValueError),
                          (dict(lse=torch.zeros(2, 3, device="cuda")), ValueError),
                          (dict(kcache=bf(4, 12, 2, 64), vcache=bf(4, 12, 2, 64)), dk.DSparkError),
                          (dict(kcache=bf(4, 8, 2, 96), vcache=bf(4, 8, 2, 96), q=bf(2, 4, 96)), dk.DSparkError)):
        with pytest.raises(error):
            ctx.attend(**{**good, **change})
    assert ctx.attend(**{**good, "q": bf(0, 4, 64), "t_offsets": i(2), "K": i(2) - 1}).shape[0] == 0
    ctx.check()


def test_captured_and_replayed(ctx):
    """Pages, write and attention of a step in one graph; lengths and verify lengths change between the replays."""
    page, heads, d, B, G = 16, 2, 128, 5, 4
    s = make(14, [300, 0, 31, 47, 1000], [3] * B, heads, 2, d, page)
    n_pages = s["kc"].shape[0]
    st = dict(length=dev(s["length"]), K=dev(s["K"]), table=dev(s["table"]), held=dev((s["table"] >= 0).sum(1)),
              free=dev(np.zeros(n_pages)), n_free=dev([0]))
    rows = (torch.randn((B * G, heads, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    k, v = rows
    outs = [torch.empty((n,), dtype=torch.int32, device="cuda") for n in (B + 1, B * G, B * G, B * G)]
    out = torch.zeros_like(s["q"])
    kc, vc = s["kc"].clone(), s["vc"].clone()

    def step():
        ctx.pages_reserve(st["K"], st["length"], st["table"], st["held"], st["free"], st["n_free"], page, n_pages, out=outs)
        ctx.cache_write(k, v, outs[3], kc, vc)
        ctx.attend(s["q"], kc, vc, st["table"], st["length"], G - 1, K=st["K"], t_offsets=outs[0], out=out)

    def eager(K, length):
        kc.copy_(s["kc"])
        vc.copy_(s["vc"])
        out.zero_()
        st["K"].copy_(dev(K))
        st["length"].copy_(dev(length))
        step()
        torch.cuda.synchronize()
        return out.clone(), kc.clone()

    plans = [(s["K"], s["length"]), ([0, 3, 1, -1, 2], [299, 0, 2, 47, 1000]), ([-1] * B, s["length"])]
    want = [eager(*p) for p in plans]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in (0, 1, 2, 0, 1):
        kc.copy_(s["kc"])
        vc.copy_(s["vc"])
        out.zero_()
        st["K"].copy_(dev(plans[n][0]))
        st["length"].copy_(dev(plans[n][1]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n][0]) and torch.equal(kc, want[n][1]), n
    ctx.check()


def test_two_contexts_on_two_streams(ctx):
    other = dk.Context(0)
    try:
        a, b = make(15, [4000, 90], [3, 0], 2, 2, 128, 16), make(16, [2000, 9], [1, 2], 2, 2, 128, 16)
        wa, wb = call(ctx, a)[0], call(ctx, b)[0]
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(3):
            with torch.cuda.stream(s1):
                ga = call(ctx, a)[0]
            with torch.cuda.stream(s2):
                gb = call(other, b)[0]
            torch.cuda.synchronize()
            assert torch.equal(ga, wa) and torch.equal(gb, wb)
        other.check()
        ctx.check()
    finally:
        other.close()
