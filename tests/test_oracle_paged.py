"""Pins of the paged-cache oracle (CPU): hand-worked page books, the e4m3
rounding against torch's type and against its own definition on borders, the
attention against torch's float64 softmax over the tokens in sequence order."""
import numpy as np
import pytest
import torch

import oracle


def test_reserve_by_hand():
    # request 0 holds one page of 8 with 6 tokens and takes 3 rows; request 1
    # is new with 2 rows; request 2 sits out
    table = np.array([[5, -1, -1], [-1, -1, -1], [2, 7, -1]])
    got = oracle.pages_reserve([2, 1, -1], [6, 0, 9], table, [1, 0, 2], [9, 4, 3, 0], 3, 8, 7)
    offs, req, pos, slot, table, held, top = got
    assert offs.tolist() == [0, 3, 5, 5]
    assert req.tolist() == [0, 0, 0, 1, 1, -1, -1]
    assert pos.tolist() == [6, 7, 8, 0, 1, -1, -1]
    # pops 3, then 4
    assert slot.tolist() == [46, 47, 24, 32, 33, -1, -1]
    assert table.tolist() == [[5, 3, -1], [4, -1, -1], [2, 7, -1]]
    assert held.tolist() == [2, 1, 2] and top == 1


def test_reserve_refuses_what_does_not_fit():
    args = dict(table=[[0, -1]], held=[1], free_list=[3, 1], page_size=8)
    fits = lambda K, n, free, rows: oracle.pages_reserve([K], [n], args["table"], args["held"], args["free_list"], free,
                                                         8, rows) is not None
    assert fits(3, 4, 0, 4) and fits(4, 4, 1, 5)
    assert not fits(4, 4, 0, 5)          # the pool is empty
    assert not fits(4, 4, 1, 4)          # five rows in four places
    assert not fits(8, 8, 2, 16)         # a third page has no place in the table
    assert not fits(-2, 4, 2, 4) and not fits(0, -1, 2, 4)


def test_commit_by_hand():
    table = np.array([[5, 3, 1], [4, 6, -1], [2, 7, 8]])
    length, held, free, top = oracle.pages_commit([6, 8, 9], [1, -1, 4], table, [3, 2, 3], [9] + [0] * 7, 1, 8,
                                                  finished=[0, 0, 1])
    assert length.tolist() == [8, 8, 0] and held.tolist() == [1, 1, 0]
    assert top == 7 and free.tolist() == [9, 3, 1, 6, 2, 7, 8, 0]


def test_commit_by_hand_limits():
    table = np.array([[5, 3, 1], [4, 6, -1]])
    length, held, free, top = oracle.pages_commit([6, 8], [1, -1], table, [3, 2], [9, 0, 0, 0], 1, 8)
    assert length.tolist() == [8, 8] and held.tolist() == [1, 1]
    assert free.tolist() == [9, 3, 1, 6] and top == 4
    assert oracle.pages_commit([6, 8], [1, -1], table, [3, 2], [9, 0, 0], 1, 8) is None     # full
    assert oracle.pages_commit([6], [2], table[:1], [1], [9, 0], 1, 8) is None               # too few pages held


def test_what_is_reserved_comes_back():
    rng = np.random.RandomState(3)
    B, page, cols, n_pages = 7, 8, 9, 60
    ids = rng.permutation(n_pages)
    length = rng.randint(0, 50, B)
    held = -(-length // page)
    table = np.full((B, cols), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.concatenate([ids[at:], np.full(at, -1)])
    K = rng.randint(0, 17, B)
    offs, req, pos, slot, t2, h2, top = oracle.pages_reserve(K, length, table, held, free, n_pages - at, page, 200)
    assert len(set(slot[:offs[-1]].tolist())) == offs[-1]
    _, h3, f3, top3 = oracle.pages_commit(length, np.full(B, -1), t2, h2, free, top, page)
    assert h3.tolist() == held.tolist() and top3 == n_pages - at
    assert set(f3[:top3].tolist()) == set(free[:top3].tolist())


def test_e4m3_levels_are_the_type():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(oracle.e4m3_levels(), codes.view(torch.float8_e4m3fn).double().numpy())


def test_e4m3_rounding():
    lv = oracle.e4m3_levels()
    mid = (lv[1:] + lv[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, lv[:-1], lv[1:])
    assert np.array_equal(oracle.to_e4m3(mid), even)
    assert np.array_equal(oracle.to_e4m3(np.nextafter(mid, 0)), lv[:-1])
    assert np.array_equal(oracle.to_e4m3(np.nextafter(mid, 1e9)), lv[1:])
    assert np.array_equal(oracle.to_e4m3(-lv), -lv)
    assert oracle.to_e4m3(1e9) == 448 and oracle.to_e4m3(-np.inf) == -448 and np.isnan(oracle.to_e4m3(np.nan))
    x = np.random.RandomState(1).randn(5000) * 50
    x32 = x.astype(np.float32)
    want = torch.from_numpy(x32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.to_e4m3(x32), want)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_against_a_softmax_over_the_sequence(causal):
    rng = np.random.RandomState(5)
    page, H, Hq, D, n_pages = 8, 2, 6, 16, 12
    length, K = np.array([0, 13]), np.array([2, 4])
    offs = np.array([0, 3])
    table = rng.permutation(n_pages)[:6].reshape(2, 3)
    kc, vc = rng.randn(n_pages, page, H, D), rng.randn(n_pages, page, H, D)
    ks, vs = rng.rand(H) + 0.5, rng.rand(H) + 0.5
    q = rng.randn(8, Hq, D)
    out, lse = oracle.attend(q, kc, vc, table, length, K, offs, causal=causal, scale=0.3, k_scale=ks, v_scale=vs)
    for b in range(2):
        k = kc[table[b]].reshape(-1, H, D) * ks[:, None]
        v = vc[table[b]].reshape(-1, H, D) * vs[:, None]
        for i in range(K[b] + 1):
            n = length[b] + (i if causal else K[b]) + 1
            for h in range(Hq):
                s = torch.from_numpy(0.3 * k[:n, h // 3] @ q[offs[b] + i, h])
                want = torch.softmax(s, 0).numpy() @ v[:n, h // 3]
                assert np.allclose(out[offs[b] + i, h], want, rtol=1e-12, atol=1e-13)
                assert abs(lse[offs[b] + i, h] - torch.logsumexp(s, 0).item()) < 1e-12
