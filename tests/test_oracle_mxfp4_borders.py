"""Pins of the oracle's MXFP4 rounding at every border (CPU): between two
levels, and where a block's power steps; the neighbours of each on both sides."""
import math

import numpy as np
import pytest

import oracle

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# border, the level that a tie goes to: the even one of codes i and i + 1
BORDERS = [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0)]


def value(x, e):
    """What x of a block whose largest value is 6 2^e becomes."""
    block = np.zeros(32)
    block[3], block[17] = 6 * 2.0 ** e, x
    codes, power = oracle.to_mxfp4(block)
    assert power == e + 127
    return oracle.from_mxfp4(codes, power)[17]


@pytest.mark.parametrize("e", [-120, -3, 0, 1, 77, 125])
@pytest.mark.parametrize("sign", [1, -1])
def test_borders_between_levels(e, sign):
    unit = sign * 2.0 ** e
    for i, (border, even) in enumerate(BORDERS):
        assert border == (LEVELS[i] + LEVELS[i + 1]) / 2 and LEVELS.index(even) % 2 == 0
        assert value(border * unit, e) == even * unit
        below, above = math.nextafter(border, 0) * unit, math.nextafter(border, 7) * unit
        assert value(below, e) == LEVELS[i] * unit and value(above, e) == LEVELS[i + 1] * unit
    for level in LEVELS:
        assert value(level * unit, e) == level * unit


@pytest.mark.parametrize("e", [-119, -3, 0, 1, 77, 124])
def test_borders_between_powers(e):
    """7 2^e is the largest that 2^e holds: it becomes 6 2^e, what lies above it belongs to the next power."""
    for x, want in ((math.nextafter(7.0, 0), (e, 6.0)), (7.0, (e, 6.0)), (math.nextafter(7.0, 8), (e + 1, 8.0)),
                    (3.5, (e - 1, 3.0)), (math.nextafter(3.5, 4), (e, 4.0))):
        block = np.zeros(32)
        block[9] = -x * 2.0 ** e
        codes, power = oracle.to_mxfp4(block)
        assert power == want[0] + 127
        assert oracle.from_mxfp4(codes, power)[9] == -want[1] * 2.0 ** e
