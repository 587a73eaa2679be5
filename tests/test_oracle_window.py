"""Pins of oracle.window: the plain forms at their limits, small cases worked out by hand, and planted
mistakes that have to show."""
import numpy as np
import pytest

from gen import trees
from oracle import attention as oatt
from oracle import chunk as och
from oracle import window as ow


def problem(rng, lens, hq=4, hkv=2, dim=8):
    need = [(n + 15) // 16 for n in lens]
    order = rng.permutation(sum(need) + 2)
    table = np.zeros((len(lens), max(need)), dtype=np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pools = rng.standard_normal((2, sum(need) + 2, 16, hkv, dim))
    return pools[0], pools[1], table


@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (1, 1 << 30), (40, 40), (65, 0)])
def test_a_window_that_reaches_all_is_plain_attention(window, sinks):
    rng = np.random.default_rng(1)
    prefix, new = [30, 0, 7], [5, 20, 1]
    k, v, table = problem(rng, [p + n for p, n in zip(prefix, new)])
    off = np.concatenate(([0], np.cumsum(new)))
    q = rng.standard_normal((off[-1], 4, 8))
    for a, b in zip(ow.chunk_attention(q, k, v, table, prefix, off, window, sinks),
                    och.chunk_attention(q, k, v, table, prefix, off)):
        assert np.allclose(a, b, rtol=1e-13, atol=1e-13)
    parents = trees.padded([trees.random_recursive(rng, n) for n in new], 20)
    q = rng.standard_normal((3, 20, 4, 8))
    out = ow.tree_attention(q, k, v, table, prefix, parents, window, sinks)[0]
    assert np.allclose(out, oatt.tree_attention(q, k, v, table, prefix, parents, 16), rtol=1e-12, atol=1e-12)


def test_a_window_of_one_token_returns_its_value():
    rng = np.random.default_rng(2)
    k, v, table = problem(rng, [25])
    q = rng.standard_normal((4, 4, 8))
    out = ow.chunk_attention(q, k, v, table, [21], [0, 4], 1, 0)[0]
    for i in range(4):
        t = 21 + i
        assert np.array_equal(out[i], np.repeat(v[table[0, t // 16], t % 16], 2, axis=0))


def test_what_is_seen_in_a_small_case():
    assert np.flatnonzero(ow.seen_by_chunk(5, 3, 3, 1)[0]).tolist() == [0, 3, 4, 5]
    assert np.flatnonzero(ow.seen_by_chunk(5, 3, 3, 1)[2]).tolist() == [0, 5, 6, 7]
    assert np.flatnonzero(ow.seen_by_chunk(0, 3, 1, 2)[2]).tolist() == [0, 1, 2]
    # root 0, children 1 and 2, 3 below 2, 4 below 3; prefix of 4
    seen = ow.seen_by_tree(4, [-1, 0, 0, 2, 3], 3, 1)
    assert np.flatnonzero(seen[0]).tolist() == [0, 2, 3, 4]
    assert np.flatnonzero(seen[1]).tolist() == [0, 3, 4, 5]
    assert np.flatnonzero(seen[3]).tolist() == [0, 4, 6, 7]          # positions 4, 5, 6
    assert np.flatnonzero(seen[4]).tolist() == [0, 6, 7, 8]          # the root has left the window
    # a sink among the tree's own positions: the root at position 1
    seen = ow.seen_by_tree(1, [-1, 0, 1, 2], 2, 2)
    assert np.flatnonzero(seen[3]).tolist() == [0, 1, 3, 4]


def test_a_chain_is_a_chunk():
    rng = np.random.default_rng(3)
    for S, n, w, s in ((9, 12, 5, 2), (0, 12, 4, 6), (33, 3, 20, 0)):
        assert np.array_equal(ow.seen_by_tree(S, list(range(-1, n - 1)), w, s), ow.seen_by_chunk(S, n, w, s))
        k, v, table = problem(rng, [S + n])
        q = rng.standard_normal((n, 4, 8))
        a = ow.chunk_attention(q, k, v, table, [S], [0, n], w, s)[0]
        b = ow.tree_attention(q[None], k, v, table, [S], np.arange(-1, n - 1)[None], w, s)[0][0]
        assert np.array_equal(a, b)


def test_every_node_is_its_root_path_as_a_chunk():
    rng = np.random.default_rng(4)
    S, n, w, s = 10, 17, 6, 3
    parents = trees.random_recursive(rng, n)
    seen = ow.seen_by_tree(S, parents, w, s)
    for i in range(n):
        path = [i]
        while path[-1]:
            path.append(int(parents[path[-1]]))
        path = path[::-1]
        want = ow.seen_by_chunk(S, len(path), w, s)[-1]
        assert np.array_equal(seen[i, :S], want[:S])
        assert np.array_equal(np.flatnonzero(seen[i, S:]), sorted(p for p, on in zip(path, want[S:]) if on))


def test_planted_mistakes_show():
    """A window one token wider, sinks one fewer, and node indices in place of depths."""
    good = ow.seen_by_chunk(40, 6, 8, 3)
    assert not np.array_equal(good, ow.seen_by_chunk(40, 6, 9, 3))
    assert not np.array_equal(good, ow.seen_by_chunk(40, 6, 8, 2))
    star = [-1] + [0] * 9                                             # every node a child of the root
    assert not np.array_equal(ow.seen_by_tree(40, star, 4, 1), ow.seen_by_tree(40, list(range(-1, 9)), 4, 1))
    assert ow.seen_by_tree(40, star, 4, 0)[:, 40].all()
