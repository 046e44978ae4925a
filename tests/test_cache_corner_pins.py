"""The oracle's order of protected tokens, by hand."""

import numpy as np

from oracle import cache_oracle as co


def test_the_newest_of_the_protected_stay():
    n, page = 6, 4
    table = np.array([[1, 0]])
    p, at = co.slots(table[0], n, page)
    k = np.zeros((2, page, 1, 1))
    k[p, at, 0, 0] = np.arange(n)
    cache = {"k": k, "v": k, "k_exp": None, "v_exp": None}
    w, pos = np.zeros((2, page, 1)), np.zeros((2, page, 1), int)
    w[p, at, 0] = [1, np.inf, 2, 3, np.nan, 0]
    pos[p, at, 0] = [0, 7, 19, 17, 18, 16]
    kept = lambda budget, sinks, recent: sorted(  # noqa: E731
        co.evict(cache, table, [n], w, pos, [20], budget, sinks, recent)[2][p, at, 0][:budget])
    assert kept(1, 1, 4) == [19] and kept(2, 1, 4) == [18, 19] and kept(4, 1, 4) == [16, 17, 18, 19]
    assert kept(5, 1, 4) == [0, 16, 17, 18, 19]    # the first token, then +infinity
    assert kept(2, 0, 1) == [7, 19] and kept(3, 1, 1) == [0, 7, 19] and kept(5, 0, 0) == [0, 7, 16, 17, 19]
