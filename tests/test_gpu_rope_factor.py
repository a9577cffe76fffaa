"""GPU: the rotary factor reaches keys of 8 and 4 bits in float64.

A stretched context's factor, 0.1 ln s + 1, is off by up to 2^-25 of it as a
float32.  Here pairs are turned by angles that bring a key between the two
borders that lie where the factor is the double and where it is that float:
factor x cos f = border factor / middle, middle halfway between the two.  The
distance of the border, 2^-27 of the key and more, is far above what the turn in float64
loses (2^-50), so the stored value has to be the oracle's.  (Its value, for a zero may
have either sign: cos of the float64 next to pi / 2 is 6e-17, and the angle is
off by up to 2^-51 pi / 2 = 7e-16; times 7 both are far below the first border.)
"""
import math

import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from test_gpu_rope import bound, caches, f64, i32, refused, values

pytestmark = pytest.mark.gpu

STRETCHES = [3.0, 6.0, 10.0, 40.0]
E4M3_BORDERS = [1 + (2 * m + 1) / 16 for m in range(8)]          # between the levels 1 + m / 8
E2M1_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def factors(stretch):
    """The factor, the float32 next to it, and what lies halfway."""
    _, factor = dk.rope_frequencies(64, 500000.0, "yarn", stretch, trained=4096)
    near = float(np.float32(factor))
    assert abs(near / factor - 1) > 2.0 ** -27
    return factor, near, (factor + near) / 2


def angles(x, borders, middle):
    """Radians that bring x middle to the borders, 32 pairs: the largest possible turned value in both of every block."""
    f = [math.acos(borders[i % len(borders)] / (x * middle)) for i in range(32)]
    f[0] = f[16] = 0.0
    f[1] = f[17] = math.pi / 2
    return np.array(f)


def keys(x, inter):
    """One row, one head of 64: pairs (x, 0)."""
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    if inter:
        k[0, 0, 0::2] = x
    else:
        k[0, 0, :32] = x
    return k.cuda()


def write(ctx, k, freq, factor, inter, kv, scale=None):
    c = caches(kv, 1, 8, 1, 64, "token")
    if kv == "e4m3":
        c = (*c[:2], scale, scale)
    ctx.rope_write(None, k, k, i32([1]), i32([3]), torch.from_numpy(freq).cuda(), *c, interleaved=inter, factor=factor)
    ctx.check()
    return c


@pytest.mark.parametrize("stretch", STRETCHES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scale", [None, 0.5])
def test_e4m3_keys_beside_a_border(ctx, stretch, inter, scale):
    factor, near, middle = factors(stretch)
    freq, k = angles(2.0, E4M3_BORDERS, middle), keys(2.0, inter)
    s = 1.0 if scale is None else scale
    want, other = [oracle.to_e4m3(oracle.rope(f64(k), [1], freq, inter, f) / s) for f in (factor, near)]
    assert (want != other).sum() == 28                   # all but the four pairs that are no border's
    c = write(ctx, k, freq, factor, inter, "e4m3", None if scale is None else torch.full((1,), scale, device="cuda"))
    assert np.array_equal(f64(c[0])[0, 3], want[0])
    assert np.array_equal(f64(c[1])[0, 3], oracle.to_e4m3(f64(k) / s)[0])


@pytest.mark.parametrize("stretch", STRETCHES)
@pytest.mark.parametrize("inter", [False, True])
def test_mxfp4_keys_beside_a_border(ctx, stretch, inter):
    factor, near, middle = factors(stretch)
    freq, k = angles(5.0, E2M1_BORDERS, middle), keys(5.0, inter)
    (want, power), (other, _) = [oracle.to_mxfp4(oracle.rope(f64(k), [1], freq, inter, f)) for f in (factor, near)]
    assert (power == 127).all() and (want != other).sum() == 28
    kc, _, kp, _ = write(ctx, k, freq, factor, inter, "mxfp4")
    assert np.array_equal(kp.cpu().numpy()[0, :, 3], power[0])
    assert np.array_equal(values(kc, kp)[0, 3], oracle.from_mxfp4(want, power)[0])


@pytest.mark.parametrize("stretch", STRETCHES)
@pytest.mark.parametrize("inter", [False, True])
def test_mxfp4_power_beside_a_border(ctx, stretch, inter):
    """The largest key of a block on either side of 7: its power is 1 or 2."""
    factor, near, middle = factors(stretch)
    freq = np.full(32, math.pi / 3)
    freq[0] = math.acos(7 / (6.5 * middle))
    k = keys(1.0, inter)
    k[0, 0, 0] = 6.5
    (want, power), (_, other) = [oracle.to_mxfp4(oracle.rope(f64(k), [1], freq, inter, f)) for f in (factor, near)]
    assert power[0, 0, 0] != other[0, 0, 0]
    kc, _, kp, _ = write(ctx, k, freq, factor, inter, "mxfp4")
    assert np.array_equal(kp.cpu().numpy()[0, :, 3], power[0])
    assert np.array_equal(values(kc, kp)[0, 3], oracle.from_mxfp4(want, power)[0])


def test_bf16_rows_take_the_factor_as_it_is(ctx):
    """Rows whose factor is the double: what is stored is what rope leaves, within half a step of the exact value."""
    factor, _, _ = factors(40.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((200, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    freq, _ = dk.rope_frequencies(64, device="cuda")
    pos = np.arange(200) * 37
    _, turned = ctx.rope(None, k, i32(pos), freq, factor=factor)
    kc, vc, _, _ = caches("bf16", 25, 8, 2, 64, "token")
    ctx.rope_write(None, k, k, i32(pos), i32(np.arange(200)), freq, kc, vc, factor=factor)
    ctx.check()
    assert torch.equal(kc.reshape(200, 2, 64), turned)
    want = oracle.rope(f64(k), pos, freq.cpu().numpy(), False, factor)
    N, extra = bound(f64(k), pos, freq.cpu().numpy(), False, factor)
    assert (np.abs(f64(turned) - want) <= 2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -24 * N + extra).all()


def test_factors_that_no_float32_holds_are_refused(ctx):
    k = keys(1.0, False)
    freq = torch.zeros(32, dtype=torch.float64, device="cuda")
    c = caches("mxfp4", 1, 8, 1, 64, "token")
    for factor in (1e39, -1e39, 1e300, float("inf"), float("nan")):
        refused(lambda: ctx.rope(k, None, i32([1]), freq, factor=factor), "factor")
        refused(lambda: ctx.rope_write(None, k, k, i32([1]), i32([3]), freq, *c, factor=factor), "factor")
    ctx.check()
