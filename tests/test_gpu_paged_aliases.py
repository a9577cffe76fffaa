"""GPU: arrays given twice to the calls that write a paged cache or read it back
are refused where one's bytes would be the other's."""
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_rope import caches, frequencies, i32, refused, rows

pytestmark = pytest.mark.gpu

PAGES, PAGE, HEADS, D, N = 4, 8, 2, 64, 5


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


@pytest.fixture
def kqv():
    g = torch.Generator(device="cuda").manual_seed(3)
    return rows(g, N, HEADS, D, False), rows(g, N, HEADS, D, False), rows(g, N, HEADS, D, False)


SLOT = [0, 9, 17, 31, 4]


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "mxfp4"])
def test_one_array_for_keys_and_values_is_refused(ctx, kqv, kv):
    q, k, v = kqv
    kc, vc, ks, vs = caches(kv, PAGES, PAGE, HEADS, D, "token")
    before = kc.clone()
    pos, slot, (freq, _) = i32(range(N)), i32(SLOT), frequencies(D)
    refused(lambda: ctx.cache_write(k, v, slot, kc, kc, ks, vs), "different arrays")
    refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, kc, kc, ks, vs), "different arrays")
    refused(lambda: ctx.rope_write(None, k, k, pos, slot, freq, kc, kc, ks, vs), "different arrays")
    ctx.check()
    assert torch.equal(kc.view(torch.uint8), before.view(torch.uint8))


def test_one_array_for_rows_that_are_the_same(ctx, kqv):
    """Keys that are the values too: the bytes are the same, written twice."""
    _, k, v = kqv
    slot = i32(SLOT)
    for kv in ("bf16", "e4m3"):
        a, b = caches(kv, PAGES, PAGE, HEADS, D, "token"), caches(kv, PAGES, PAGE, HEADS, D, "token")
        ctx.cache_write(k, k, slot, a[0], a[0], a[2], a[2])
        ctx.cache_write(k, v, slot, b[0], b[1], b[2], b[2])
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
        wide = torch.cat([k, v], 1)                      # the same first row, other strides
        refused(lambda: ctx.cache_write(k, wide[:, :HEADS], slot, a[0], a[0], a[2], a[2]), "different arrays")
    refused(lambda: ctx.cache_write(k, k, slot, a[0], a[0], a[2], a[3]), "different arrays")
    ctx.check()


def as_rows(t):
    """The first bytes of an array as bf16 rows."""
    n = N * HEADS * D
    flat = torch.as_strided(t, (t.numel(),), (1,)).view(torch.bfloat16)
    assert flat.numel() >= n
    return flat[:n].view(N, HEADS, D)


def test_results_over_caches_and_powers_are_refused(ctx, kqv):
    q, k, v = kqv
    pos, slot, (freq, _) = i32(range(N)), i32(SLOT), frequencies(D)
    for kv in ("bf16", "e4m3", "mxfp4"):
        c = caches(kv, 20 * PAGES, PAGE, HEADS, D, "token")
        arrays = c if kv == "mxfp4" else c[:2]
        for t in arrays:
            refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, *c, q_out=as_rows(t)), "q_out")
            refused(lambda: ctx.cache_read(c[0], c[1], slot, *c[2:], out=(as_rows(t), q)), "different")
            refused(lambda: ctx.cache_read(c[0], c[1], slot, *c[2:], out=(q, as_rows(t))), "different")
        refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, *c, q_out=k), "q_out")
        refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, *c, q_out=v), "q_out")
        refused(lambda: ctx.cache_read(c[0], c[1], slot, *c[2:], out=(q, q)), "different")
    ctx.check()


def test_powers_over_a_cache_are_refused(ctx, kqv):
    q, k, v = kqv
    pos, slot, (freq, _) = i32(range(N)), i32(SLOT), frequencies(D)
    kc, vc, ks, vs = caches("mxfp4", PAGES, PAGE, HEADS, D, "token")
    shape = ks.shape
    for cache in (kc, vc):
        over = cache.reshape(-1)[:ks.numel()].view(shape)
        assert over.data_ptr() == cache.data_ptr()
        for powers in ((over, vs), (ks, over)):
            refused(lambda: ctx.cache_write(k, v, slot, kc, vc, *powers), "powers")
            refused(lambda: ctx.rope_write(q, k, v, pos, slot, freq, kc, vc, *powers), "powers")
            refused(lambda: ctx.cache_read(kc, vc, slot, *powers), "powers")
    ctx.check()
