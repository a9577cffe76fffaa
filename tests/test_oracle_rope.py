"""Pins of the oracle's rotary positions and 4-bit values, and of the binding's
frequencies: closed forms, invariants, values worked out by hand."""
import math

import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk


def test_a_quarter_turn_by_hand():
    x = np.zeros((1, 1, 6))
    x[0, 0] = [1, 2, 3, 4, 5, 6]
    f = [math.pi / 2, math.pi]
    half = oracle.rope(x, [1], f)                        # pairs (1, 3), (2, 4); 5 and 6 stay
    assert np.allclose(half[0, 0], [-3, -2, 1, -4, 5, 6], atol=1e-15)
    pairs = oracle.rope(x, [1], f, interleaved=True)     # pairs (1, 2), (3, 4)
    assert np.allclose(pairs[0, 0], [-2, 1, -3, -4, 5, 6], atol=1e-15)
    assert np.allclose(oracle.rope(x, [0], f, factor=0.5)[0, 0], [0.5, 1, 1.5, 2, 5, 6])
    assert np.isnan(oracle.rope(x, [-1], f)).all()


def test_lengths_stay_and_products_go_by_the_distance():
    r = np.random.RandomState(1)
    f = 10000.0 ** (-np.arange(8) / 8)
    q, k = r.randn(1, 1, 16), r.randn(1, 1, 16)
    for inter in (False, True):
        at = lambda x, t: oracle.rope(x, [t], f, inter)[0, 0]
        assert np.allclose(np.linalg.norm(at(q, 977)), np.linalg.norm(q))
        assert np.allclose(at(q, 1000) @ at(k, 993), at(q, 50) @ at(k, 43), atol=1e-12)


def test_far_positions_keep_their_angle():
    """2^30 steps of 2 pi / 2^20 are whole turns: nothing moves, though the angle is 6.4e3 turns of 2^17."""
    x = np.arange(1.0, 3.0).reshape(1, 1, 2)
    f = [float(np.longdouble(2) * np.pi) / 2 ** 20]
    assert np.allclose(oracle.rope(x, [1 << 30], f), x, atol=1e-6)


def test_mxfp4_values_by_hand():
    block = np.zeros(32)
    block[:12] = [6.0, 0.25, 0.26, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 5.01, 0.0, -0.1]
    codes, power = oracle.to_mxfp4(block)
    assert power == 127
    want = [6, 0, 0.5, 1, -1, 2, 2, -4, 4, 6, 0, 0]      # borders go to the even code
    assert np.array_equal(oracle.from_mxfp4(codes, power)[:12], want)


@pytest.mark.parametrize("top,e,back", [(7.0, 0, 6), (7.01, 1, 8), (8.0, 1, 8), (3.5, -1, 3), (3.6, 0, 4), (6.0, 0, 6),
                                        (1e-38, -120, 0), (0.0, 0, 0), (float("inf"), 125, 6 * 2.0 ** 125),
                                        (7 * 2.0 ** 125, 125, 6 * 2.0 ** 125)])
def test_mxfp4_powers_by_hand(top, e, back):
    block = np.zeros(32)
    block[5] = -top
    codes, power = oracle.to_mxfp4(block)
    assert power == e + 127
    assert oracle.from_mxfp4(codes, power)[5] == -back


def test_every_mxfp4_value_is_off_by_half_a_step_at_most():
    r = np.random.RandomState(2)
    x = r.randn(4000, 32) * np.exp(r.randn(4000, 1) * 5)
    codes, power = oracle.to_mxfp4(x)
    unit = 2.0 ** (power.astype(float) - 127)
    a = np.abs(x) / unit
    assert a.max() <= 7 and (a.max(1) > 3.5).all()       # no smaller power would do
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(oracle.from_mxfp4(codes, power) - x) <= unit * step / 2).all()
    codes, power = oracle.to_mxfp4(np.where(np.arange(64) == 40, np.nan, 1.0))
    assert list(power) == [125, 255] and np.isnan(oracle.from_mxfp4(codes, power)[32:]).all()


def test_plain_and_linear_frequencies():
    f, factor = dk.rope_frequencies(8, 10000.0)
    assert f.dtype == torch.float64 and factor == 1.0
    assert np.allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-14)
    g, factor = dk.rope_frequencies(8, 10000.0, "linear", 4.0)
    assert np.allclose(g, f / 4, rtol=1e-15) and factor == 1.0


def test_ntk_frequencies_stretch_the_slowest_pair_alone():
    f, _ = dk.rope_frequencies(64, 10000.0)
    g, factor = dk.rope_frequencies(64, 10000.0, "ntk", 8.0)
    assert g[0] == 1 and np.isclose(g[-1], f[-1] / 8, rtol=1e-13) and factor == 1.0
    assert (g[1:] < f[1:]).all() and (torch.diff(g / f) < 0).all()


def test_parts_go_by_turns():
    f, _ = dk.rope_frequencies(128, 500000.0)
    g, factor = dk.rope_frequencies(128, 500000.0, "parts", 8.0, trained=8192)
    turns = 8192 * f / (2 * math.pi)
    assert factor == 1.0
    assert torch.equal(g[turns >= 4], f[turns >= 4]) and np.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    for i in np.flatnonzero(((turns > 1) & (turns < 4)).numpy()):
        w = (float(turns[i]) - 1) / 3
        assert np.isclose(g[i], f[i] * (w + (1 - w) / 8), rtol=1e-13)


def test_yarn_mixes_over_the_pairs():
    f, _ = dk.rope_frequencies(128, 10000.0)
    g, factor = dk.rope_frequencies(128, 10000.0, "yarn", 16.0, trained=4096)
    assert np.isclose(factor, 0.1 * math.log(16) + 1)
    # the pair that turns n times within 4096 positions: 64 ln(4096 / 2 pi n) / ln 10000
    lo, hi = [64 * math.log(4096 / (2 * math.pi * n)) / math.log(10000) for n in (32, 1)]
    lo, hi = math.floor(lo), math.ceil(hi)
    assert (lo, hi) == (20, 46)
    for j in range(64):
        w = min(1, max(0, (j - lo) / (hi - lo)))
        assert np.isclose(g[j], f[j] * (1 - w) + f[j] / 16 * w, rtol=1e-13)


@pytest.mark.parametrize("args", [(7,), (0,), (8, 1.0), (8, float("inf")), (8, 1e4, "linear", 0.5), (8, 1e4, None, 2.0),
                                  (8, 1e4, "other", 2.0), (8, 1e4, "yarn", 2.0), (8, 1e4, "parts", 2.0, 0),
                                  (8, 1e4, "parts", 2.0, 100, 4.0, 1.0), (2, 1e4, "ntk", 2.0)])
def test_frequencies_that_are_none_are_refused(args):
    with pytest.raises(ValueError):
        dk.rope_frequencies(*args)
