"""GPU: penalties, biases and masks (dspark_constrain) against the float64 oracle.

Tolerance of an entry, all in float32: half a step of every rounding.  The
division or product by rep, freq c, the two differences, and a bias sum of m
terms: 2^-24 (5 + m) times the sum of the magnitudes |l1| + freq c + pres + sum
|bias| that they form, where l1 = l rep or l / rep.  Masked entries and rows
that no rule touches are exact.
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


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def words_of(allowed):
    n, V = allowed.shape
    bits = np.zeros((n, -(-V // 32) * 32), dtype=np.uint8)
    bits[:, :V] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def make(seed, B, n_pos, V, hist, n_bias, with_mask, K=None):
    rng = np.random.RandomState(seed)
    s = dict(B=B, n_pos=n_pos, V=V)
    s["K"] = np.full(B, n_pos - 1) if K is None else np.array(K)
    s["n_hist"] = rng.randint(0, hist + 1, B)
    s["n_hist"][0] = hist
    s["n_prompt"] = (s["n_hist"] * rng.rand(B)).astype(int)
    s["hist"] = (rng.rand(B, max(hist, 1)) ** 3 * V).astype(int)
    s["tokens"] = (rng.rand(B, max(n_pos - 1, 1)) ** 3 * V).astype(int)
    if n_pos > 3:
        s["tokens"][:, 2] = s["tokens"][:, 0]                    # a token drafted twice
    if n_pos > 1:
        s["tokens"][0, 0] = s["hist"][0, 0]                      # one of the history
    s["rep"] = (0.8 + rng.rand(B)).astype(np.float32)
    s["freq"], s["pres"] = rng.randn(2, B).astype(np.float32)
    s["bias_n"] = rng.randint(0, n_bias + 1, B)
    s["bias_id"] = np.sort((rng.rand(B, n_bias) ** 2 * V).astype(int), 1)
    if n_bias > 1:
        s["bias_id"][:, 1] = s["bias_id"][:, 0]                  # an id given twice
        s["bias_id"][0, -1] = V - 1
        s["bias_n"][0] = n_bias
    s["bias_val"] = (rng.randn(B, n_bias) * 5).astype(np.float32)
    s["allowed"] = rng.rand(B, n_pos, V) < rng.rand(B, n_pos, 1) if with_mask else None
    if with_mask:
        s["allowed"][0, 0] = False
        s["allowed"][-1, -1] = True
    s["x"] = rng.randn(B, n_pos, V).astype(np.float32) * 4
    return s


def want_of(s, x):
    out, tol = [], []
    for b in range(s["B"]):
        n, p = s["K"][b] + 1, min(s["n_prompt"][b], s["n_hist"][b])
        nb = s["bias_n"][b]
        bias = list(zip(s["bias_id"][b][:nb], s["bias_val"][b][:nb].astype(np.float64)))
        h = s["hist"][b]
        rep, freq, pres = [float(s[k][b]) for k in ("rep", "freq", "pres")]
        how = dict(prompt=h[:p], written=h[p:s["n_hist"][b]], drafts=s["tokens"][b])
        allowed = None if s["allowed"] is None else s["allowed"][b][:n]
        out.append(oracle.constrain(x[b][:n], **how, rep=rep, freq=freq, pres=pres, bias=bias, allowed=allowed))
        # magnitudes: every term of the sum positive
        size = oracle.constrain(np.abs(x[b][:n]), **how, rep=min(rep, 1 / rep), freq=-abs(freq), pres=-abs(pres),
                                bias=[(t, abs(v)) for t, v in bias])
        tol.append(2.0 ** -24 * (5 + nb) * size)
        touched = oracle.constrain(np.zeros((n, s["V"])), **how, freq=-1.0, bias=[(t, 1.0) for t, _ in bias]) > 0
        for t in how["prompt"]:
            touched[:, t] = True
        tol[-1][~touched] = 0
        if allowed is not None:
            tol[-1][~allowed] = 0
    return out, tol


def arguments(s):
    kw = dict(hist=dev(s["hist"])[:, :max(1, s["hist"].shape[1])], n_hist=dev(s["n_hist"]), n_prompt=dev(s["n_prompt"]),
              rep=dev(s["rep"], np.float32), freq=dev(s["freq"], np.float32), pres=dev(s["pres"], np.float32))
    if s["n_pos"] > 1:
        kw["tokens"] = dev(s["tokens"])
    if s["bias_id"].shape[1]:
        kw["bias"] = (dev(s["bias_id"]), dev(s["bias_val"], np.float32), dev(s["bias_n"]))
    return kw


def compare(got, want, tol):
    for b, (w, t) in enumerate(zip(want, tol)):
        g = got[b].double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(w)), b
        inf = ~np.isfinite(w)
        assert np.array_equal(g[inf & ~np.isnan(w)], w[inf & ~np.isnan(w)])
        assert (np.abs(g - w)[~inf] <= t[~inf]).all(), (b, np.abs(g - w)[~inf].max())


CASES = [  # B, n_pos, V, history, biases, mask
    (1, 1, 1, 1, 0, False),
    (1, 1, 1000, 5, 1, True),
    (3, 8, 1024, 300, 7, True),
    (2, 8, 50257, 3000, 40, True),
    (5, 33, 8191, 100, 2, False),
    (4, 2, 8193, 0, 300, True),
    (2, 17, 16388, 40000, 0, True),
    (70, 4, 32003, 50, 3, True),
]


@pytest.mark.parametrize("B,n_pos,V,hist,n_bias,with_mask", CASES)
@pytest.mark.parametrize("bf16", [True, False])
def test_packed_rows_match_the_oracle(ctx, B, n_pos, V, hist, n_bias, with_mask, bf16):
    print(f"constrain B={B} n_pos={n_pos} V={V} hist={hist} bias={n_bias} mask={with_mask} bf16={bf16}", flush=True)
    rng = np.random.RandomState(V)
    s = make(V, B, n_pos, V, hist, n_bias, with_mask, K=rng.randint(0 if B == 1 else -1, n_pos, B))
    wide = -(-V // 8) * 8 + 8
    offs = np.concatenate([[0], np.cumsum(s["K"] + 1)]) + 1       # a row of no request on both sides
    x = torch.full((offs[-1] + 1, wide), 9.0)
    for b in range(B):
        x[offs[b]:offs[b + 1], :V] = torch.from_numpy(s["x"][b, :s["K"][b] + 1])
    x = x.cuda().to(torch.bfloat16 if bf16 else torch.float32)
    mask = None
    if with_mask:
        m = np.zeros((len(x), V), dtype=bool)
        for b in range(B):
            m[offs[b]:offs[b + 1]] = s["allowed"][b, :s["K"][b] + 1]
        mask = dev(words_of(m))
    out = torch.full((len(x), wide), 7.0, device="cuda")
    got = ctx.constrain(x[:, :V], n_pos, K=dev(s["K"]), t_offsets=dev(offs), mask=mask, out=out[:, :V], **arguments(s))
    ctx.check()
    xs = [x[offs[b]:offs[b + 1], :V].double().cpu().numpy() for b in range(B)]
    want, tol = want_of(s, xs)
    compare([got[offs[b]:offs[b + 1]] for b in range(B)], want, tol)
    assert (out[[0, -1]] == 7).all() and (out[:, V:] == 7).all()
    if not bf16:                                                  # in place: the same values
        ctx.constrain(x[:, :V], n_pos, K=dev(s["K"]), t_offsets=dev(offs), mask=mask, out=x[:, :V], **arguments(s))
        ctx.check()
        assert torch.equal(x[1:-1, :V], got[1:-1]) and (x[[0, -1]] == 9).all() and (x[:, V:] == 9).all()


@pytest.mark.parametrize("position_major", [False, True])
def test_strided_rows_of_the_draft(ctx, position_major):
    """The padded layout, request-major or position-major, more positions than n_pos, no drafts counted."""
    B, n_pos, V = 6, 3, 5003
    s = make(21, B, n_pos, V, 200, 5, True)
    s["tokens"] = [[] for _ in range(B)]
    shape = (n_pos + 1, B, 5008) if position_major else (B, n_pos + 1, 5008)
    x, out = torch.full(shape, 9.0, device="cuda"), torch.full(shape, 7.0, device="cuda")
    if position_major:
        x, out = x.transpose(0, 1), out.transpose(0, 1)
    x[:, :n_pos, :V] = torch.from_numpy(s["x"]).cuda()
    mask = np.zeros((B, n_pos + 1, V), dtype=bool)
    mask[:, :n_pos] = s["allowed"]
    kw = arguments(dict(s, tokens=np.zeros((B, n_pos - 1))))
    kw.pop("tokens")
    words = dev(words_of(mask.reshape(-1, V))).view(B, n_pos + 1, -1)
    got = ctx.constrain(x[:, :, :V], n_pos, mask=words, out=out[:, :, :V], **kw)
    ctx.check()
    want, tol = want_of(s, s["x"])
    compare(got[:, :n_pos], want, tol)
    assert (out[:, n_pos:] == 7).all() and (out[:, :, V:] == 7).all()


def test_nothing_to_apply_is_a_conversion(ctx):
    x = (torch.randn((5, 1000), device="cuda") * 9).to(torch.bfloat16)
    offs = dev([0, 3])
    got = ctx.constrain(x, 3, K=dev([2, 1]), t_offsets=offs)
    assert torch.equal(got, x.float())
    ctx.check()


def test_values_that_are_not_finite(ctx):
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[-float("inf"), low, float("nan"), float("inf"), 1.0, -1e30, -1.1e30, 0.0]], device="cuda")
    got = ctx.constrain(x, 1, t_offsets=dev([0]), rep=dev([2.0], np.float32), hist=dev([[0, 1, 3, 7]]), n_hist=dev([4]))
    ctx.check()
    m = np.float32(dk.MASKED)
    assert got[0, [0, 1, 5, 6]].tolist() == [m] * 4 and torch.isnan(got[0, 2]) and got[0, 3] == float("inf")
    assert got[0, 4] == 1 and got[0, 7] == 0
    xb = x.to(torch.bfloat16)
    xb[0, 1] = torch.finfo(torch.bfloat16).min
    mask = dev([[0b11111011]])
    got = ctx.constrain(xb, 1, t_offsets=dev([0]), mask=mask)
    assert got[0, [0, 1, 2]].tolist() == [m] * 3 and got[0, 3] == float("inf")
    none = ctx.constrain(xb, 1, t_offsets=dev([0]), mask=mask * 0)
    assert (none == m).all()
    ctx.check()


def test_bad_numbers_are_flagged(ctx):
    x = torch.zeros((4, 64), device="cuda")
    base = dict(n_pos=2, K=dev([1, 1]), t_offsets=dev([0, 2]), hist=dev([[1, 2], [3, 4]]), n_hist=dev([2, 2]),
                freq=dev([1, 1], np.float32))
    good = ctx.constrain(x, **base)
    ctx.check()
    bias = lambda ids, n=(2, 2): (dev(ids), torch.zeros((2, 2), device="cuda"), dev(n))
    for change, word, same in ((dict(K=dev([2, 1])), "verify length", True), (dict(K=dev([1, -2])), "verify length", None),
                               (dict(t_offsets=dev([0, 3])), "row out of range", None),
                               (dict(t_offsets=dev([-1, 2])), "row out of range", None),
                               (dict(n_hist=dev([2, 3])), "history", True), (dict(n_hist=dev([2, -1])), "history", None),
                               (dict(hist=dev([[1, 2], [64, 4]])), "token id", None),
                               (dict(hist=dev([[1, 2], [3, -1]])), "token id", None),
                               (dict(tokens=dev([[0], [2 ** 31 - 1]])), "token id", None),
                               (dict(bias=bias([[1, 2], [4, 3]])), "ascending", True),
                               (dict(bias=bias([[1, 64], [4, 5]])), "token id", True),
                               (dict(bias=bias([[1, 2], [4, 5]], (3, 0))), "bias length", True),
                               (dict(rep=dev([1.0, 0.0], np.float32)), "repetition", True),
                               (dict(rep=dev([1.0, np.nan], np.float32)), "repetition", True),
                               (dict(rep=dev([np.inf, 1.0], np.float32)), "repetition", True)):
        got = ctx.constrain(x, **{**base, **change})
        with pytest.raises(dk.DSparkError, match=word):
            ctx.check()
        if same:
            assert torch.equal(got, good), change


def test_refusals(ctx):
    x = torch.zeros((2, 3, 64), device="cuda")
    i = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    f = lambda *n: torch.zeros(n, device="cuda")
    for args, kw, error in (((x, 4), {}, ValueError), ((x, 0), {}, dk.DSparkError), ((x.half(), 3), {}, TypeError),
                            ((x[0], 3), {}, ValueError), ((x, 3), dict(K=i(3)), ValueError),
                            ((f(2, 3, 66)[:, :, :64], 3), {}, dk.DSparkError), ((f(2, 3, 68)[:, :, 1:65], 3), {}, dk.DSparkError),
                            ((f(1, 3, 64).expand(2, 3, 64), 3), {}, dk.DSparkError),
                            ((x, 3), dict(out=f(2, 3, 32)), ValueError), ((x, 3), dict(out=f(2, 1, 64).expand(2, 3, 64)), dk.DSparkError),
                            ((x, 3), dict(hist=i(3, 4), n_hist=i(2)), ValueError), ((x, 3), dict(hist=i(2, 4), n_hist=i(3)), ValueError),
                            ((x, 3), dict(hist=i(2, 4)), TypeError), ((x, 3), dict(tokens=i(2, 1)), ValueError),
                            ((x, 3), dict(rep=f(3)), ValueError), ((x, 3), dict(rep=i(2)), TypeError),
                            ((x, 3), dict(bias=(i(2, 4), f(2, 3), None)), ValueError),
                            ((x, 3), dict(mask=i(2, 3, 1)), ValueError), ((x, 3), dict(mask=i(2, 2, 2)), ValueError),
                            ((x, 3), dict(mask=f(2, 3, 2)), TypeError),
                            ((f(40, 64), 34), dict(t_offsets=i(1)), dk.DSparkError),
                            ((x, 3), dict(mask=i(2, 1, 2).expand(2, 3, 2)), dk.DSparkError)):
        with pytest.raises(error):
            ctx.constrain(*args, **kw)
    assert ctx.constrain(f(0, 64), 3, t_offsets=i(2), K=i(2) - 1).shape == (0, 64)
    ctx.check()


def test_captured_and_replayed(ctx):
    B, n_pos, V = 3, 4, 9001
    s = make(31, B, n_pos, V, 500, 9, True)
    offs = np.arange(B) * n_pos
    x = torch.zeros((B * n_pos, 9008), device="cuda")
    x[:, :V] = torch.from_numpy(s["x"]).reshape(-1, V)
    mask = dev(words_of(s["allowed"].reshape(-1, V)))
    out = torch.zeros_like(x)
    kw = dict(K=dev(s["K"]), t_offsets=dev(offs), mask=mask, out=out[:, :V], **arguments(s))
    step = lambda: ctx.constrain(x[:, :V], n_pos, **kw)
    want = []
    for k in (3, 0, 2):
        kw["K"].fill_(k)
        out.zero_()
        step()
        torch.cuda.synchronize()
        want.append(out.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n, k in ((0, 3), (1, 0), (2, 2), (0, 3)):
        kw["K"].fill_(k)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n])
    ctx.check()
