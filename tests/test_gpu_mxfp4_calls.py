"""GPU: rotary and 4-bit calls at the ends of what is allowed: one projection's
columns, broadcast inputs, 8192 heads, caches that lie within each other, shared
pages, the largest batch, nobody taking part."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import dev
from test_gpu_attend_mxfp4 import call, check, make
from test_gpu_rope import caches, frequencies, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("order", ["token", "head"])
def test_columns_of_one_projection_in_place(ctx, order):
    """Queries, keys and values lie in one tensor; heads of a row together, or rows of a head."""
    n, hq, h, d = 41, 6, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((n, hq + 2 * h, d), generator=g, device="cuda").to(torch.bfloat16)
    if order == "head":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    split = lambda t: (t[:, :hq], t[:, hq:hq + h], t[:, hq + h:])
    q, k, v = split(x)
    pos, slot = i32(np.arange(n) * 311 - 1), i32(np.arange(n)[::-1].copy())
    freq, _ = frequencies(64)
    want_q, want_k = ctx.rope(q.contiguous(), k.contiguous(), pos, freq)
    y = x.clone(memory_format=torch.preserve_format)
    yq, yk, yv = split(y)
    ctx.rope(yq, yk, pos, freq, q_out=yq, k_out=yk)
    ctx.check()
    assert torch.equal(yq[1:], want_q[1:]) and torch.equal(yk[1:], want_k[1:])
    assert torch.equal(yq[0], q[0]) and torch.equal(yk[0], k[0]) and torch.equal(yv, v)
    a, b = caches("mxfp4", 8, 8, h, d, order), caches("mxfp4", 8, 8, h, d, order)
    ctx.rope_write(q.contiguous(), k.contiguous(), v.contiguous(), pos, slot, freq, *a)
    z = x.clone(memory_format=torch.preserve_format)
    zq, zk, zv = split(z)
    ctx.rope_write(zq, zk, zv, pos, slot, freq, *b, q_out=zq)
    ctx.check()
    assert torch.equal(zq[1:], want_q[1:]) and torch.equal(zq[0], q[0])
    assert torch.equal(zk, k) and torch.equal(zv, v)
    assert all([torch.equal(s, t) for s, t in zip(a, b)])


def test_broadcast_inputs(ctx):
    """One row's or one head's values given to many."""
    n, h, d = 30, 4, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    one_row = torch.randn((1, h, d), generator=g, device="cuda").to(torch.bfloat16)
    one_head = torch.randn((n, 1, d), generator=g, device="cuda").to(torch.bfloat16)
    q, k = one_row.expand(n, h, d), one_head.expand(n, h, d)
    pos, (freq, _) = i32(np.arange(n) * 5), frequencies(64)
    got = ctx.rope(q, k, pos, freq, interleaved=True)
    want = ctx.rope(q.contiguous(), k.contiguous(), pos, freq, interleaved=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    slot = i32(np.arange(n))
    for kv in ("bf16", "e4m3", "mxfp4"):
        a, b = caches(kv, 4, 8, h, d, "token"), caches(kv, 4, 8, h, d, "token")
        ctx.rope_write(None, k, q, pos, slot, freq, *a)
        ctx.rope_write(None, k.contiguous(), q.contiguous(), pos, slot, freq, *b)
        assert all([s is None or torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b)])
    a, b = caches("mxfp4", 4, 8, h, d, "head"), caches("mxfp4", 4, 8, h, d, "head")
    ctx.cache_write(k, q, slot, *a)
    ctx.cache_write(k.contiguous(), q.contiguous(), slot, *b)
    ctx.check()
    assert all([torch.equal(s, t) for s, t in zip(a, b)])


@pytest.mark.parametrize("hq,h,d", [(8192, 0, 16), (5000, 3192, 32), (1, 8191, 24)])
def test_the_most_heads(ctx, hq, h, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((3, hq + h, d), generator=g, device="cuda").to(torch.bfloat16)
    pos, (freq, _) = i32([7, -1, 100000]), frequencies(16)
    got = ctx.rope(x[:, :hq], x[:, hq:] if h else None, pos, freq)
    # every head as a row of its own
    rows = x.view(3 * (hq + h), 1, d)
    want, _ = ctx.rope(rows, None, pos.repeat_interleave(hq + h), freq)
    ctx.check()
    want = want.view(3, hq + h, d)
    assert torch.equal(got[0], want[:, :hq]) and (not h or torch.equal(got[1], want[:, hq:]))
    with pytest.raises(dk.DSparkError, match="8192"):
        ctx.rope(torch.zeros((1, 8193, 16), dtype=torch.bfloat16, device="cuda"), None, pos[:1], freq)


def test_caches_that_lie_within_one_tensor(ctx):
    """Keys and values of a page side by side; the types torch has for 4-bit values and powers."""
    s = make(3, [70, 5, 333], [3, 0, 7], 2, 4, 128, 16)
    want, want_lse = call(ctx, s)
    both = torch.stack([s["kc"], s["vc"]], 1)            # [n_pages][2][page][heads][d / 2]
    t = dict(s, kc=both[:, 0], vc=both[:, 1])
    got, lse = call(ctx, t)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    t = dict(s, kc=both[:, 0].view(torch.float4_e2m1fn_x2), vc=both[:, 1].view(torch.float4_e2m1fn_x2),
             kp=s["kp"].view(torch.float8_e8m0fnu), vp=s["vp"].view(torch.float8_e8m0fnu))
    got, lse = call(ctx, t)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    slot = i32([0, 17, -1, 40])
    a = ctx.cache_read(s["kc"], s["vc"], slot, s["kp"], s["vp"])
    b = ctx.cache_read(both[:, 0], both[:, 1], slot, s["kp"], s["vp"])
    # into columns of one tensor, rows of a head together
    wide = torch.full((5, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    c = ctx.cache_read(s["kc"], s["vc"], slot, s["kp"], s["vp"], out=(wide[:, :2], wide[:, 3:5]))
    ctx.check()
    live = torch.tensor([0, 1, 3], device="cuda")
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x[live], z[live]) and (z[2] == 7).all()
    assert (wide[:, 2] == 7).all()


def test_pages_that_requests_share(ctx):
    """Three requests over one prefix: the same ids in their tables."""
    s = make(4, [200, 200, 200], [2, 2, 2], 2, 2, 64, 32)
    s["table"][1:, :6] = s["table"][0, :6]               # 192 tokens
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_the_largest_batch(ctx):
    rng = np.random.RandomState(5)
    s = make(5, rng.randint(0, 40, 4096), rng.randint(-1, 1, 4096), 1, 1, 64, 8)
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_nobody_takes_part_and_no_rows(ctx):
    s = make(6, [20, 0, 300], [0, 0, 0], 2, 2, 128, 16)
    out = torch.full_like(s["q"], 7)
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    call(ctx, dict(s, K=np.array([-1] * 3)), K=dev([-1] * 3), t_offsets=dev([0] * 4), out=out, lse=lse)
    assert (out == 7).all() and (lse == 7).all()
    call(ctx, dict(s, q=s["q"][:0], K=np.array([-1] * 3)), K=dev([-1] * 3), t_offsets=dev([0] * 4), out=out[:0], lse=lse[:0])
    kc, vc, kp, vp = s["kc"], s["vc"], s["kp"], s["vp"]
    x = torch.zeros((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    none = i32([])
    before = [t.clone() for t in (kc, vc, kp, vp)]
    ctx.cache_write(x, x, none, kc, vc, kp, vp)
    k, v = ctx.cache_read(kc, vc, none, kp, vp)
    assert k.shape == v.shape == (0, 2, 128)
    pos = i32([-1, -1, -1])
    y = torch.ones((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    freq, _ = frequencies(128)
    ctx.rope_write(None, y, y, pos, i32([0, 1, 2]), freq, kc, vc, kp, vp)
    ctx.check()
    assert all([torch.equal(a, b) for a, b in zip(before, (kc, vc, kp, vp))])


@pytest.mark.parametrize("heads,group,d", [(96, 1, 64), (40, 3, 128), (1, 64, 256)])
def test_many_heads(ctx, heads, group, d):
    s = make(7, [100, 0, 37], [2, 0, 1], heads, group, d, 8, "head")
    out, lse = call(ctx, s)
    ctx.check()
    check(s, out, lse)


def test_single_entries_with_arbitrary_strides(ctx):
    s = make(8, [13], [0], 1, 1, 64, 16)
    want, lse = call(ctx, s)
    t = dict(s, kc=torch.as_strided(s["kc"], s["kc"].shape, (s["kc"].stride(0), s["kc"].stride(1), 1, 1)))
    t["q"] = torch.as_strided(s["q"].contiguous(), (1, 1, 64), (1, 3, 1))
    got, lse2 = call(ctx, t)
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    x = torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16)
    y = torch.as_strided(x.clone(), (1, 1, 64), (5, 7, 1))
    freq, _ = frequencies(32)
    a, _ = ctx.rope(x, None, i32([9]), freq)
    ctx.rope(y, None, i32([9]), freq, q_out=y)
    ctx.check()
    assert torch.equal(a, y)
