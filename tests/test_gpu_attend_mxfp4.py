"""GPU: attention over a 4-bit paged cache (dspark_attend_mxfp4) against float64.

The cache's values are exact in bf16, weights are split in two: the bound is
that of a bf16 cache (2^-8 of the result, 2^-15 of the weights), as
worst_error() of attend_reference has it (and 2^-60 of the largest value, since
0 is among the values and is 0 exactly).
"""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from attend_reference import worst_error
from test_gpu_attend import LENGTHS, dev
from test_gpu_rope import refused, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def make(seed, length, K, heads, group, d, page, order="token", spread=1.5):
    """Books, a cache of random codes and powers, queries between other columns."""
    rng = np.random.RandomState(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    length, K = np.array(length), np.array(K)
    held = -(-(length + K + 1) // page)
    n_pages = int(held.sum()) + 2
    table = np.full((len(length), int(held.max()) + 1), -1)
    ids = rng.permutation(n_pages)
    at = 0
    for b in range(len(length)):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    shape = (n_pages, page, heads, d // 2) if order == "token" else (n_pages, heads, page, d // 2)

    def cache():
        x = torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8)
        return x if order == "token" else x.permute(0, 2, 1, 3)

    def power():
        return torch.randint(122, 127, (n_pages, heads, page, d // 32), generator=g, device="cuda").to(torch.uint8)

    wide = torch.randn((int((K + 1).sum()), heads * group + 2, d), generator=g, device="cuda").mul_(spread).to(torch.bfloat16)
    return dict(q=wide[:, 1:-1], kc=cache(), vc=cache(), kp=power(), vp=power(), table=table, length=length, K=K,
                offs=np.concatenate([[0], np.cumsum(K + 1)]), scale=d ** -0.5)


def call(ctx, s, causal=True, **kw):
    out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    kw = {**dict(K=dev(s["K"]), t_offsets=dev(s["offs"]), out=out, lse=lse), **kw}
    ctx.attend(s["q"], s["kc"], s["vc"], dev(s["table"]), dev(s["length"]), max(0, int(s["K"].max())), causal=causal,
               scale=s["scale"], k_scale=s["kp"], v_scale=s["vp"], **kw)
    return kw["out"], kw["lse"]


def decoded(s):
    """The same books over the values that the cache stands for."""
    t = dict(s, ks=None, vs=None)
    for c, p in (("kc", "kp"), ("vc", "vp")):
        t[c] = torch.from_numpy(values(s[c], s[p])).float()
    return t


def check(s, out, lse, causal=True):
    worst = worst_error(decoded(s), out, lse, causal, 2.0 ** -15, 2.0 ** -60)
    assert worst <= 1.0, worst
    return worst


CASES = [  # heads, group, d, page, order, gamma
    (2, 1, 64, 8, "token", 0),
    (1, 4, 128, 16, "token", 0),
    (2, 4, 128, 16, "head", 7),
    (3, 5, 64, 32, "token", 3),
    (1, 8, 128, 64, "head", 7),
    (2, 2, 64, 16, "token", 16),
    (1, 16, 256, 128, "token", 1),
    (2, 3, 256, 8, "head", 6),
    (1, 1, 128, 1024, "token", 32),
    (1, 64, 64, 16, "token", 2),
    (5, 1, 256, 32, "token", 0),
]


@pytest.mark.parametrize("heads,group,d,page,order,gamma", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_float64(ctx, heads, group, d, page, order, gamma, causal):
    print(f"attend mxfp4 heads={heads} group={group} d={d} page={page} {order} gamma={gamma} {causal}", flush=True)
    rng = np.random.RandomState(gamma + d)
    K = [gamma, 0, -1] + [int(k) for k in rng.randint(-1, gamma + 1, len(LENGTHS) - 3)]
    s = make(1 + d, LENGTHS, K, heads, group, d, page, order)
    out, lse = call(ctx, s, causal)
    ctx.check()
    print("worst error over its bound: %.3f" % check(s, out, lse, causal))
    again, lse2 = call(ctx, s, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("length,gamma,heads,group,d", [(5000, 0, 1, 1, 128), (9001, 3, 2, 4, 128), (20000, 7, 1, 2, 64),
                                                        (3333, 1, 1, 3, 256), (6000, 7, 2, 8, 128)])
def test_one_long_request_is_joined_from_many_pieces(ctx, length, gamma, heads, group, d):
    print(f"attend mxfp4 length={length} gamma={gamma} heads={heads} d={d}", flush=True)
    s = make(3, [length], [gamma], heads, group, d, 16)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_the_same_result_as_over_a_bf16_cache_of_the_same_values(ctx):
    for d, order in ((64, "token"), (128, "head"), (256, "token")):
        s = make(11, [300, 0, 1200, 31], [3, 0, 7, 2], 2, 3, d, 16, order)
        out, lse = call(ctx, s)
        k, v = [torch.from_numpy(values(s[c], s[p])).float().cuda().to(torch.bfloat16) for c, p in (("kc", "kp"), ("vc", "vp"))]
        want = torch.zeros_like(out)
        wl = torch.zeros_like(lse)
        ctx.attend(s["q"], k, v, dev(s["table"]), dev(s["length"]), 7, K=dev(s["K"]), t_offsets=dev(s["offs"]), scale=s["scale"],
                   out=want, lse=wl)
        ctx.check()
        # the same exact products in another order of sums
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        assert (lse - wl).abs().max() < 1e-4


def test_powers_far_apart(ctx):
    """Blocks of 2^-60 beside blocks of 2^50: nothing is lost where a row sees the small ones alone."""
    for d in (64, 128, 256):
        s = make(5, [40, 200, 3], [2, 0, 1], 2, 2, d, 8)
        s["vp"][:, :, :, 0] -= 60
        s["vp"][:, 1, :, -1] += 50
        s["kp"][:, :, :, 1] -= 30
        out, lse = call(ctx, s)
        ctx.check()
        check_blocks(s, out, lse, d)


def check_blocks(s, out, lse, d):
    """Each block of 32 values against its own bound."""
    for b in range(d // 32):
        t = decoded(s)
        at = slice(32 * b, 32 * b + 32)
        vc = torch.zeros_like(t["vc"])
        vc[..., at] = t["vc"][..., at]
        part = torch.zeros_like(out)
        part[..., at] = out[..., at]
        assert worst_error(dict(t, vc=vc), part, lse, True, 2.0 ** -15, 2.0 ** -60) <= 1.0


@pytest.mark.parametrize("step", [-3, -1, 1, 3])
def test_powers_that_rise_and_fall_along_a_request(ctx, step):
    """From token to token, by 2^100 in all; values stay below 2^100."""
    for d, page in ((64, 16), (128, 8), (128, 32), (256, 16)):
        s = make(15, [70, 8, 333], [3, 0, 1], 2, 4, d, page)
        for b, (n, k) in enumerate(zip(s["length"], s["K"])):
            for t in range(n + k + 1):
                s["vp"][s["table"][b][t // page], :, t % page] = int(np.clip(110 + step * (t // 3), 30, 170))
        s["vp"][:, 1, :, 0] += 40
        out, lse = call(ctx, s)
        ctx.check()
        check_blocks(s, out, lse, d)
        # a NaN among them reaches who sees it
        t2 = dict(s, vp=s["vp"].clone())
        t2["vp"][s["table"][2][4], 1, 2, 1] = 255
        t2["vp"][s["table"][0][(s["length"][0] + 2) // page], 0, (s["length"][0] + 2) % page, 0] = 255
        out2, _ = call(ctx, t2)
        nan = torch.zeros_like(out, dtype=torch.bool)
        nan[s["offs"][2]:, 4:, 32:64] = True
        nan[2:4, :4, :32] = True
        assert torch.isnan(out2[nan]).all() and torch.isfinite(out2[~nan]).all()
        # (a block that is NaN has no power: sums may be in another order)
        assert ((out2 - out)[~nan].abs() <= 2.0 ** -7 * out[~nan].abs()).all()


def test_loud_drafts_leave_the_rows_before_them_alone(ctx):
    """Later drafts whose values are 2^60 larger or smaller: rows that do not see them are as they were."""
    for d, page in ((64, 8), (128, 16), (256, 32)):
        for up in (60, -60):
            s = make(16, [40, 0, 31, 700], [7, 5, 3, 6], 2, 3, d, page)
            out, lse = call(ctx, s)
            check(s, out, lse)
            for b in range(4):
                t = s["length"][b] + 3
                s["vp"][s["table"][b][t // page], :, t % page] += up % 256
            out2, lse2 = call(ctx, s)
            ctx.check()
            check_blocks(s, out2, lse2, d)
            for b in range(4):
                lo = s["offs"][b]
                assert torch.equal(lse2[lo:lo + 3], lse[lo:lo + 3])
                assert ((out2 - out)[lo:lo + 3].abs() <= 2.0 ** -7 * out[lo:lo + 3].abs()).all()


def test_large_scores(ctx):
    for spread in (30.0, 300.0):
        s = make(6, [200, 900, 31], [2, 0, 4], 2, 3, 128, 16, spread=spread)
        out, lse = call(ctx, s)
        ctx.check()
        check(s, out, lse)


def test_what_is_masked_has_no_effect(ctx):
    """Any bytes in unused places of pages and free pages; NaN blocks in later drafts reach the rows that see them alone."""
    for d, page, order in ((64, 8, "token"), (128, 64, "head"), (256, 16, "token")):
        s = make(7, [0, 13, 40, 127, 250], [3, 7, 5, 2, 6], 2, 2, d, page, order)
        out, lse = call(ctx, s)
        check(s, out, lse)
        used = torch.zeros((s["kc"].shape[0], page), dtype=torch.bool)
        for b in range(5):
            for t in range(s["length"][b] + s["K"][b] + 1):
                used[s["table"][b][t // page], t % page] = True
        un = ~used.cuda()
        for name in ("kp", "vp"):
            s[name].masked_fill_(un[:, None, :, None], 255)
        for name in ("kc", "vc"):
            s[name].masked_fill_(un[:, :, None, None], 0xFF)
        out2, lse2 = call(ctx, s)
        ctx.check()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        for name in ("kp", "vp"):
            t2 = dict(s, **{name: s[name].clone()})
            for b, i in ((1, 4), (2, 5), (4, 1)):
                t = s["length"][b] + i
                t2[name][s["table"][b][t // page], 1, t % page, 1] = 255
            out2, lse2 = call(ctx, t2)
            ctx.check()
            for b, i in ((1, 4), (2, 5), (4, 1)):
                lo, hi = s["offs"][b], s["offs"][b + 1]
                assert torch.equal(out2[lo:lo + i], out[lo:lo + i]) and torch.equal(lse2[lo:lo + i], lse[lo:lo + i])
                assert torch.equal(out2[lo:hi, :2], out[lo:hi, :2])
                if name == "vp":
                    assert torch.isnan(out2[lo + i:hi, 2:, 32:64]).all()
                    assert torch.equal(out2[lo + i:hi, 2:, :32], out[lo + i:hi, 2:, :32])
                    assert torch.equal(out2[lo + i:hi, 2:, 64:], out[lo + i:hi, 2:, 64:])
                else:
                    assert torch.isnan(out2[lo + i:hi, 2:]).all()
        # a NaN block that every row sees
        t2 = dict(s, vp=s["vp"].clone())
        t2["vp"][s["table"][4][0], 0, 3, 0] = 255
        out2, _ = call(ctx, t2)
        lo, hi = s["offs"][4], s["offs"][5]
        assert torch.isnan(out2[lo:hi, :2, :32]).all() and torch.equal(out2[lo:hi, :, 32:], out[lo:hi, :, 32:])
        assert torch.equal(out2[:lo], out[:lo])


def test_rows_of_no_request_are_left_as_they_were(ctx):
    s = make(9, [10, 20], [1, 0], 1, 2, 64, 8)
    q = torch.randn((9, 2, 64), device="cuda").to(torch.bfloat16)
    q[1:3], q[6:7] = s["q"][:2], s["q"][2:]
    s["q"], s["offs"] = q, np.array([1, 6])
    out, lse = call(ctx, s)
    ctx.check()
    rest = [0, 3, 4, 5, 7, 8]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()


def test_a_bad_page_is_flagged(ctx):
    for bad in (-1, 10 ** 6):
        s = make(2, [50, 20], [1, 0], 1, 2, 64, 8)
        s["table"][0, 3] = bad
        call(ctx, s)
        with pytest.raises(dk.DSparkError, match="page"):
            ctx.check()


def test_refusals(ctx):
    s = make(2, [50, 20], [1, 0], 1, 2, 64, 8)
    refused(lambda: call(ctx, dict(s, kp=None)), "k_scale")
    refused(lambda: call(ctx, dict(s, vp=s["kp"])), "powers")
    refused(lambda: call(ctx, dict(s, vp=s["vp"][:-1])), "v_scale")
    refused(lambda: call(ctx, dict(s, kp=torch.ones(1, device="cuda"))), "k_scale")
    refused(lambda: call(ctx, dict(s, q=s["q"][..., :32])), "q must")
    refused(lambda: ctx.attend(s["q"], s["kc"], s["vc"], dev(s["table"]), dev(s["length"]), 1, K=dev(s["K"]),
                               t_offsets=dev(s["offs"]), k_scale=s["kp"], v_scale=s["vp"], scale=0.0), "scale")
    lib, h = ctx.lib, ctx._h
    p = s["kc"].data_ptr()
    cache = lambda f, *rest: f(h, None, 1, 1, 64, 8, 4, p, 64, 64, p, 64, 64, p, p, p, 256, 32, 32, *rest)
    assert cache(lib.dspark_cache_write, dk.DSPARK_MXFP4, None, None) == dk.DSPARK_EINVAL
    assert b"dspark_cache_write_mxfp4" in lib.dspark_last_error(h)
    ctx.check()


def test_captured_and_replayed_over_growing_lengths(ctx):
    s = make(13, [100, 7, 900], [2, 0, 5], 2, 4, 128, 16)
    table, length, K, offs = [dev(s[k]) for k in ("table", "length", "K", "offs")]
    out, lse = torch.zeros_like(s["q"]), torch.zeros(s["q"].shape[:2], device="cuda")

    def step():
        ctx.attend(s["q"], s["kc"], s["vc"], table, length, 5, K=K, t_offsets=offs, k_scale=s["kp"], v_scale=s["vp"], out=out,
                   lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lengths in ([100, 7, 900], [3, 0, 450], [105, 0, 1]):
        length.copy_(dev(lengths))
        s["q"].mul_(-1)
        step()
        want = out.clone(), lse.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    ctx.check()
