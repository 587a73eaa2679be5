"""Attention with a sliding window and sinks over a paged cache, float64, by definition.

A row at position P sees, of the tokens that plain causal (or tree) attention lets it see, those
at positions p with P - p < window or p < sinks.  A cached or chunk token's position is its
logical index; tree node i's is S + depth(i), S the prefix length and the root's depth 0.
"""
from __future__ import annotations

import numpy as np

from . import chunk as och


def seen_by_chunk(S: int, n: int, window: int, sinks: int) -> np.ndarray:
    """[n][S + n]: whether new token i sees logical token t."""
    P = S + np.arange(n)[:, None]
    t = np.arange(S + n)[None]
    return (t <= P) & ((P - t < window) | (t < sinks))


def seen_by_tree(S: int, parents, window: int, sinks: int) -> np.ndarray:
    """[N][S + N] for a tree of N nodes (parents[0] = -1): whether node i sees logical token t."""
    N = len(parents)
    depth = np.zeros(N, dtype=np.int64)
    family = np.eye(N, dtype=bool)
    for i in range(1, N):
        depth[i] = depth[parents[i]] + 1
        family[i] |= family[parents[i]]
    P = (S + depth)[:, None]
    pos = np.concatenate((np.arange(S), S + depth))[None]
    allowed = np.concatenate((np.ones((N, S), dtype=bool), family), axis=1)
    return allowed & ((P - pos < window) | (pos < sinks))


def _tokens(pages, table, t):
    return pages[table[t // och.PS], t % och.PS]


def _rows(q, seen, k_pages, v_pages, table):
    """attend() of rows q [n][H][D], each over the tokens it sees; no other token is looked at."""
    out, spread, reach = np.empty(q.shape), np.empty(q.shape), np.empty(q.shape[:2])
    for i in range(len(q)):
        t = np.flatnonzero(seen[i])
        K, V = _tokens(k_pages, table, t), _tokens(v_pages, table, t)
        out[i], spread[i], reach[i] = och.attend(q[i], K, V, np.ones(len(t), dtype=bool))
    return out, spread, reach


def chunk_attention(q, k_pages, v_pages, page_table, prefix_lens, offsets, window: int, sinks: int):
    """Packed rows q [T][Hq][D] over float64 pools [P][16][Hkv][D]; (out, spread, reach) as in
    oracle.chunk, NaN where a row belongs to no sequence."""
    T, H, D = q.shape
    res = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    for b in range(len(prefix_lens)):
        o0, o1, S = int(offsets[b]), int(offsets[b + 1]), int(prefix_lens[b])
        part = _rows(q[o0:o1], seen_by_chunk(S, o1 - o0, window, sinks), k_pages, v_pages, np.asarray(page_table[b]))
        for whole, x in zip(res, part):
            whole[o0:o1] = x
    return res


def tree_attention(q, k_pages, v_pages, page_table, prefix_lens, parents, window: int, sinks: int):
    """Trees q [B][N][Hq][D]; parent rows may be padded with -2, whose output rows are zeros."""
    B, N, H, D = q.shape
    res = np.zeros((B, N, H, D)), np.zeros((B, N, H, D)), np.zeros((B, N, H))
    for b in range(B):
        n = int((np.asarray(parents[b]) > -2).sum())
        seen = seen_by_tree(int(prefix_lens[b]), [int(x) for x in parents[b][:n]], window, sinks)
        for whole, x in zip(res, _rows(q[b, :n], seen, k_pages, v_pages, np.asarray(page_table[b]))):
            whole[b, :n] = x
    return res
