"""GPU: the 4-bit cache's writes (dspark_cache_write_mxfp4) and rows of a cache
back as bf16 (dspark_cache_read), bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from test_gpu_rope import caches, codes_of, f64, i32, refused, rows, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


CASES = [  # rows, heads, d, page, order
    (1, 1, 64, 8, "token"),
    (5, 3, 128, 16, "head"),
    (33, 2, 256, 64, "token"),
    (200, 5, 64, 1024, "head"),
    (77, 1, 128, 32, "token"),
]


@pytest.mark.parametrize("n,h,d,page,order", CASES)
def test_written_values_and_rows_read_back(ctx, n, h, d, page, order):
    print(f"mxfp4 n={n} heads={h} d={d} page={page} {order}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.RandomState(n)
    n_pages = n // page + 2
    slot = rng.permutation(n_pages * page)[:n]
    k, v = rows(g, n, h, d), rows(g, n, h, d, False)
    k[0, 0, :32] = 0                                     # a block of nothing
    v *= torch.exp2(torch.randint(-60, 60, (n, h, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
    kc, vc, ks, vs = caches("mxfp4", n_pages, page, h, d, order)
    before = [x.clone() for x in (kc, vc, ks, vs)]
    if n > 4:
        slot[2] = -1
    ctx.cache_write(k, v, i32(slot), kc, vc, ks, vs)
    ctx.check()
    live = slot >= 0
    at = (slot[live] // page, slot[live] % page)
    for x, cache, power in ((k, kc, ks), (v, vc, vs)):
        code, byte = oracle.to_mxfp4(f64(x)[live])
        assert np.array_equal(codes_of(cache)[at], code)
        assert np.array_equal(power.cpu().numpy().transpose(0, 2, 1, 3)[at], byte)
    rest = np.ones((n_pages, page), dtype=bool)
    rest[at] = False
    for a, b in zip(before[:2], (kc, vc)):
        assert np.array_equal(a.cpu().numpy()[rest], b.cpu().numpy()[rest])
    for a, b in zip(before[2:], (ks, vs)):
        assert np.array_equal(a.cpu().numpy().transpose(0, 2, 1, 3)[rest], b.cpu().numpy().transpose(0, 2, 1, 3)[rest])
    # back: in another order, rows twice, rows of no slot left as they were
    ask = np.concatenate([rng.permutation(slot[live]), slot[live][:2], [-1]])
    out = [torch.full((len(ask), h + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")[:, :h] for _ in range(2)]
    got = ctx.cache_read(kc, vc, i32(ask), ks, vs, out=out)
    ctx.check()
    for y, cache, power in zip(got, (kc, vc), (ks, vs)):
        want = values(cache, power)[ask[:-1] // page, ask[:-1] % page]
        assert np.array_equal(f64(y)[:-1], want) and (y[-1] == 7).all()
    new = ctx.cache_read(kc, vc, i32(ask), ks, vs)
    assert all(torch.equal(a[:-1], b[:-1]) and (b[-1] == 0).all() for a, b in zip(got, new))


def test_every_bf16_value(ctx):
    """All bf16 bit patterns, beside a value that sets their block's power: borders, subnormals, infinities, NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    for top in (0.0, 6.0, 1.75, 1.0, 448.0, 3e38):
        x = torch.zeros((65536 // 31 + 1) * 31, dtype=torch.bfloat16)
        x[:65536] = bits
        x = torch.cat([x.view(-1, 31), torch.full((len(x) // 31, 1), top, dtype=torch.bfloat16)], 1)
        x = torch.cat([x, x[:len(x) % 2]]).reshape(-1, 1, 64).cuda()
        n = len(x)
        pages = -(-n // 64)
        kc, vc, ks, vs = caches("mxfp4", pages, 64, 1, 64, "token")
        ctx.cache_write(x, -x, i32(np.arange(n)), kc, vc, ks, vs)
        k, v = ctx.cache_read(kc, vc, i32(np.arange(n)), ks, vs)
        ctx.check()
        code, byte = oracle.to_mxfp4(f64(x))
        assert np.array_equal(codes_of(kc).reshape(-1, 1, 64)[:n], code)
        assert np.array_equal(ks.cpu().numpy().reshape(-1, 1, 2)[:n], byte)
        want = oracle.from_mxfp4(code, byte)
        assert np.array_equal(f64(k), want, equal_nan=True) and np.array_equal(f64(v), -want, equal_nan=True)


def test_powers_of_every_byte_come_back(ctx):
    """Caches that another program filled: powers from 2^-126 on, 255 for NaN."""
    kc, vc, ks, vs = caches("mxfp4", 32, 8, 1, 64, "head")
    kc.copy_(torch.arange(32 * 8 * 32, device="cuda").to(torch.uint8).view(32, 8, 1, 32))
    byte = torch.arange(256, device="cuda").to(torch.uint8)
    byte[byte < 1] = 1
    byte[(byte > 252) & (byte < 255)] = 252
    ks.copy_(byte.view(32, 1, 8, 1).expand(32, 1, 8, 2))
    k, _ = ctx.cache_read(kc, vc, i32(np.arange(256)), ks, vs)
    ctx.check()
    want = values(kc, ks).reshape(256, 1, 64)
    tiny = np.abs(want) < 2.0 ** -126
    got = f64(k)
    assert np.array_equal(got[~tiny], want[~tiny], equal_nan=True)
    assert (np.abs(got[tiny] - want[tiny]) <= 2.0 ** -127).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["token", "head"])
def test_rows_of_the_other_caches_back(ctx, kv, order):
    g = torch.Generator(device="cuda").manual_seed(5)
    for n, h, d, page in ((1, 1, 64, 8), (90, 3, 128, 16), (41, 2, 256, 128)):
        kc, vc, ks, vs = caches(kv, n // page + 2, page, h, d, order)
        k, v = rows(g, n, h, d), rows(g, n, h, d)
        slot = np.random.RandomState(n).permutation((n // page + 2) * page)[:n]
        ctx.cache_write(k, v, i32(slot), kc, vc, ks, vs)
        got = ctx.cache_read(kc, vc, i32(slot), ks, vs)
        ctx.check()
        for y, x, cache, scale in zip(got, (k, v), (kc, vc), (ks, vs)):
            if kv == "bf16":
                assert torch.equal(y, x)
                continue
            raw = cache.float().cpu()[torch.from_numpy(slot // page), torch.from_numpy(slot % page)]
            assert torch.equal(y.cpu(), (raw * scale.cpu()[:, None]).to(torch.bfloat16))
    # no scales: those are 1
    if kv == "e4m3":
        got = ctx.cache_read(kc, vc, i32(slot))
        raw = kc.float().cpu()[torch.from_numpy(slot // page), torch.from_numpy(slot % page)]
        assert torch.equal(got[0].cpu(), raw.to(torch.bfloat16))


def test_bad_slots_are_flagged_and_left(ctx):
    kc, vc, ks, vs = caches("mxfp4", 2, 8, 2, 64, "token")
    for bad in (16, -2, 2 ** 31 - 1, -2 ** 31):
        out = [torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ctx.cache_read(kc, vc, i32([0, bad, 15]), ks, vs, out=out)
        with pytest.raises(dk.DSparkError, match="slot"):
            ctx.check()
        assert (out[0][1] == 7).all() and (out[1][1] == 7).all() and not (out[0][2] == 7).any()
        x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
        a, b, c, d = [t.clone() for t in (kc, vc, ks, vs)]
        ctx.cache_write(x, x, i32([-1, bad, -1]), a, b, c, d)
        with pytest.raises(dk.DSparkError, match="slot"):
            ctx.check()
        assert torch.equal(a, kc) and torch.equal(b, vc) and torch.equal(c, ks) and torch.equal(d, vs)


def test_refusals(ctx):
    kc, vc, ks, vs = caches("mxfp4", 2, 8, 2, 64, "token")
    slot = i32([0, 1])
    x = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    refused(lambda: ctx.cache_write(x, x, slot, kc, vc), "k_scale")
    refused(lambda: ctx.cache_write(x, x, slot, kc, vc, torch.ones(2, device="cuda"), vs), "k_scale")
    refused(lambda: ctx.cache_write(x, x, slot, kc, vc, ks.transpose(1, 2).contiguous(), vs), "k_scale")
    refused(lambda: ctx.cache_write(x, x, slot, kc, vc, ks, ks), "powers")
    refused(lambda: ctx.cache_write(x, x, slot, kc, vc[:1], ks, vs), "kcache")
    refused(lambda: ctx.cache_write(x[..., :32], x[..., :32], slot, kc, vc, ks, vs), "k and v")
    refused(lambda: ctx.cache_read(kc, vc, slot, ks, vs, out=(x, x)), "different")
    refused(lambda: ctx.cache_read(kc, vc, slot, ks, vs, out=(x, x[:1])), "k and v")
    refused(lambda: ctx.cache_read(kc, vc, slot, ks, vs, out=(x, x[:1].expand(2, 2, 64))), "overlap")
    refused(lambda: ctx.cache_read(kc, vc, slot.long(), ks, vs), "row_slot")
    b = caches("bf16", 2, 8, 2, 64, "token")
    refused(lambda: ctx.cache_read(b[0], b[1], slot, torch.ones(2, device="cuda")), "scales")
    refused(lambda: ctx.cache_read(b[0], b[1], slot, out=(b[0][0, :2], x)), "different")
    got = ctx.cache_read(kc, vc, slot[:0], ks, vs)
    assert got[0].shape == (0, 2, 64)
    ctx.cache_write(x[:0], x[:0], slot[:0], kc, vc, ks, vs)
    # the other types' names of the same bytes
    k2 = ctx.cache_read(kc.view(torch.float4_e2m1fn_x2), vc.view(torch.float4_e2m1fn_x2), slot, ks.view(torch.float8_e8m0fnu),
                        vs.view(torch.float8_e8m0fnu))
    assert torch.equal(k2[0], ctx.cache_read(kc, vc, slot, ks, vs)[0])
    ctx.check()
