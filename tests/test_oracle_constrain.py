"""Pins of the logit-constraint oracle (CPU): a row worked by hand, and the
identities that follow from the definition."""
import numpy as np

import oracle


def test_by_hand():
    #          0    1    2    3    4    5     6
    l = [[1.0, -1.0, 2.0, -2.0, 0.5, 4.0, -8.0]] * 3
    allowed = np.ones((3, 7), dtype=bool)
    allowed[1, 4] = allowed[2] = False
    got = oracle.constrain(l, prompt=[0, 1], written=[2, 3, 2], drafts=[6, 2], rep=2.0, freq=0.25, pres=0.5,
                           bias=[(0, 3.0), (5, -1.0), (5, -1.0)], allowed=allowed)
    assert got[0].tolist() == [0.5 + 3, -2.0, 1 - 0.5 - 0.5, -4 - 0.25 - 0.5, 0.5, 2.0, -8.0]
    assert got[1].tolist() == [3.5, -2.0, 0.0, -4.75, oracle.MASKED, 2.0, -16 - 0.25 - 0.5]
    assert (got[2] == oracle.MASKED).all()


def test_identities():
    rng = np.random.RandomState(0)
    l = rng.randn(4, 50) * 3
    assert np.array_equal(oracle.constrain(l), l)
    assert np.array_equal(oracle.constrain(l, prompt=[1, 2], written=[3], drafts=[4, 4, 4]), l)
    # a draft counts for the rows behind it alone, and as a written token does
    a = oracle.constrain(l, drafts=[7, 9, 7], rep=1.3, freq=0.2, pres=0.1)
    assert np.array_equal(a[0], l[0])
    assert np.array_equal(a[3], oracle.constrain(l[3:], written=[7, 9, 7], rep=1.3, freq=0.2, pres=0.1)[0])
    # low values become the masked value, NaN stays
    x = oracle.constrain([[-np.inf, -3.4e38, np.nan, np.inf]])
    assert x[0, 0] == x[0, 1] == oracle.MASKED and np.isnan(x[0, 2]) and x[0, 3] == np.inf
