"""Pin of the page oracle (CPU): pages held must hold the tokens cached."""
import oracle


def test_reserve_refuses_tokens_without_a_page():
    go = lambda K, n, held: oracle.pages_reserve([K], [n], [[0, 1, -1]], [held], [3, 2], 2, 8, 9) is not None
    assert go(0, 8, 1) and go(-1, 16, 2) and go(-1, 0, 0)
    assert not go(0, 9, 1) and not go(-1, 17, 2) and not go(-1, 1, 0)
