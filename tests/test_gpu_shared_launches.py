"""Shared prefixes where the groups' rows and the sequences' own are two launches side by side, and trees of few rows in
every form that AUTO takes of them."""
import numpy as np
import pytest
import torch

from chunk_util import check_attention
from test_gpu_window import (TIMEOUT, ints, run_chunk_shared, run_chunk_window, run_tree_shared, shared_tree_problem,  # noqa: F401
                             ts)
from window_util import chunk64, make_shared, tree64

pytestmark = pytest.mark.gpu
pools = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


def launches(ts, call):  # noqa: F811
    before = ts.launch_count()
    res = call()
    return res, ts.launch_count() - before


# ------------------------------------------------------------------------------ two launches

def two_launch_chunks(device, e4m3, seed):
    rng = np.random.default_rng([seed, 3])
    groups = [(1000, [int(x) for x in rng.integers(100, 900, 21)]), (0, [400]), (513, [int(x) for x in rng.integers(60, 300, 18)])]
    B = sum(len(own) for _, own in groups)
    return make_shared(device, groups, [1 + b % 3 if b % 7 else 0 for b in range(B)], 32, 8, 128, "bf16", e4m3, seed=seed)


@pools
@pytest.mark.parametrize("graph", [False, True], ids=["calls", "graph"])
def test_each_of_many_calls_finds_its_own_plan(ts, cuda_device, e4m3, graph):  # noqa: F811
    """Calls over one workspace with nothing waited for between them, each of other lengths and groups than the one before:
    ranges, shares or counters of an earlier call would give other rows.  Each is compared with a call on its own."""
    p, go, sl = two_launch_chunks(cuda_device, e4m3, 51)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)
    ws = torch.empty(ts.chunk_shared_workspace_bytes(prob, sl.shape[0]), dtype=torch.uint8, device=cuda_device)
    ws.fill_(0xa5)
    full, n = torch.tensor(p.prefix, dtype=torch.int32), 10
    settings = []
    for i in range(n):                                         # within the tokens that are there
        lens = full - ints([(7 * i + 11 * b) % 60 for b in range(len(p.prefix))], "cpu")
        starts = go + ints([0, -(i % 4), i % 5, 0], cuda_device)   # more of them in the group that shares nothing
        settings.append((lens.to(cuda_device), ints([(1000, 640, 64)[i % 3], 0, (450, 0, 320)[i % 3]], cuda_device), starts))
    lens, shared, starts = (torch.empty_like(x) for x in settings[0])
    out = torch.empty_like(p.q)

    def call():
        ts.tree_chunk_attn_shared(p.q, p.k_pages, p.v_pages, p.page_table, lens, p.chunk_offsets, starts, shared, out,
                                  workspace=ws, **p.scales())

    def load(i):
        for dst, src in zip((lens, shared, starts), settings[i]):
            dst.copy_(src)

    load(0)
    _, count = launches(ts, call)
    assert count == 4, "not the form with two attention launches"
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
    for turn in range(3):
        got = []
        for i in range(n):
            load(i)
            out.fill_(3.0)
            g.replay() if graph else call()
            got.append(out.clone())
        torch.cuda.synchronize()
        assert ts.read_status(ws) == 0
        for i in range(n):
            p.prefix_lens, sl2, go2 = settings[i][0], settings[i][1], settings[i][2]
            want, status = run_chunk_shared(ts, p, go2, sl2)
            rows = slice(p.chunk_offsets[0].item(), p.chunk_offsets[-1].item())
            assert status == 0 and torch.equal(got[i][rows], want[rows])
            if turn == 0 and i < 3:
                p.prefix = p.prefix_lens.tolist()
                check_attention(want[rows], *chunk64(p), max(p.prefix) + 3, 128, "bf16", True)


# ------------------------------------------------------------------------------ trees of few rows

def inner(offsets, lens):
    """The groups between the first and the last, whose sequences then share nothing."""
    return offsets[1:-1].contiguous(), lens[1:-1].contiguous()


# trees behind shared prefixes in units of 8 or 16 rows: groups, nodes, N, hq, hkv, dim, whether the first and last group are
# left out, kernels of a call: the prologue, the plan, the attention (twice where the groups' rows are a launch of their own)
# and the merge
FEW_TREES = [
    ([(130, [5, 0])], [4, 2], 4, 8, 2, 128, False, 4),
    ([(64, [1, 70, 0])], [2, 1, 2], 2, 8, 2, 64, False, 4),
    ([(300, [0, 9])], [1, 1], 1, 32, 2, 128, False, 4),
    ([(40, [30, 0]), (700, list(range(0, 300, 20))), (257, list(range(0, 900, 60))), (128, [0] * 5), (90, [8, 9, 60])],
     [1, 4, 3, 2, 4] * 8, 4, 32, 8, 128, True, 5),
    ([(40, [30, 0]), (700, list(range(0, 300, 20))), (257, list(range(0, 900, 60))), (128, [0] * 5), (90, [8, 9, 60])],
     [1, 2, 2] * 13 + [1], 2, 16, 4, 64, True, 5),
    ([(64, [0] * 7), (1999, [3 * b for b in range(20)]), (0, [5])], [3, 4, 1, 2] * 7, 4, 16, 8, 128, False, 5),
    ([(70, [9]), (1000, [7 * b for b in range(38)]), (66, [3])], [1] * 40, 1, 64, 4, 64, True, 5),
]


@pools
@pytest.mark.parametrize("case", FEW_TREES, ids=lambda c: f"{len(c[0])}g-{len(c[1])}x{c[2]}x{c[3]}-d{c[5]}-{c[7]}k")
def test_trees_of_few_rows_behind_shared_prefixes(ts, cuda_device, case, e4m3):  # noqa: F811
    """Against the definition, with padding rows whose queries are NaN, and to the bit whatever ran in between."""
    groups, sizes, N, hq, hkv, dim, cut, kernels = case
    p, q, parents, go, sl = shared_tree_problem(cuda_device, groups, sizes, N, hq, hkv, dim, "bf16", e4m3, sum(sizes))
    assert len(sizes) == go[-1].item()
    if cut:
        go, sl = inner(go, sl)
    prob = ts.attn_problem(q, p.k_pages, p.page_table)
    kv = ts.DTYPE_E4M3 if e4m3 else ts.DTYPE_BF16
    own = torch.empty(ts.attn_shared_workspace_bytes(prob, kv, sl.shape[0]), dtype=torch.uint8, device=cuda_device)
    out, count = launches(ts, lambda: ts.tree_attn_verify_shared(q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, parents,
                                                                 go, sl, workspace=own, **p.scales()))
    assert ts.read_status(own) == 0 and count == kernels
    ref, spread, reach = tree64(p, q, parents.cpu().numpy())
    check_attention(out, ref, spread, reach, max(S + n for S, n in zip(p.prefix, p.new)), dim, "bf16", True)
    other, go2, sl2 = two_launch_chunks(cuda_device, e4m3, 53)
    for turn in range(6):
        if turn % 2:
            run_chunk_shared(ts, other, go2, sl2)
        again, status = run_tree_shared(ts, p, q, parents, go, sl)
        assert status == 0 and torch.equal(again, out)


@pools
def test_trees_of_few_rows_replay_from_a_graph(ts, cuda_device, e4m3):  # noqa: F811
    """Two launches over trees: lengths, trees and shares change between the replays."""
    groups, sizes, N, hq, hkv, dim = FEW_TREES[3][:6]
    p, q, parents, go, sl = shared_tree_problem(cuda_device, groups, sizes, N, hq, hkv, dim, "bf16", e4m3, 55)
    prob = ts.attn_problem(q, p.k_pages, p.page_table)
    kv = ts.DTYPE_E4M3 if e4m3 else ts.DTYPE_BF16
    ws = torch.empty(ts.attn_shared_workspace_bytes(prob, kv, sl.shape[0]), dtype=torch.uint8, device=cuda_device)
    out = torch.empty_like(q)

    def call():
        ts.tree_attn_verify_shared(q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, parents, go, sl, out, workspace=ws,
                                   **p.scales())

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    lens, nodes = sl.tolist(), list(sizes)
    for turn in range(4):
        q.normal_()
        sl.copy_(ints([max(0, x - 64 * turn) for x in lens], cuda_device))
        sizes = [max(1, n - (b + turn) % 2) for b, n in enumerate(nodes)]
        rows = [[-1] + [max(0, i - 1 - turn % 2) for i in range(1, n)] + [-2] * (N - n) for n in sizes]
        parents.copy_(ints(rows, cuda_device))
        p.new = sizes
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert ts.read_status(ws) == 0
        assert torch.equal(got, run_tree_shared(ts, p, q, parents, go, sl)[0])
        ref, spread, reach = tree64(p, q, parents.cpu().numpy())
        check_attention(got, ref, spread, reach, max(S + n for S, n in zip(p.prefix, p.new)), dim, "bf16", True)


# ------------------------------------------------------------------------------ limits

@pools
@pytest.mark.parametrize("kind", ["chunks", "trees"])
def test_waits_that_run_out_in_two_launches_leave_the_next_call_right(ts, cuda_device, kind, e4m3):  # noqa: F811
    if kind == "chunks":
        p, go, sl = two_launch_chunks(cuda_device, e4m3, 57)
        call = lambda: run_chunk_shared(ts, p, go, sl)  # noqa: E731
    else:
        p, q, parents, go, sl = shared_tree_problem(cuda_device, *FEW_TREES[3][:6], "bf16", e4m3, 57)
        call = lambda: run_tree_shared(ts, p, q, parents, go, sl)  # noqa: E731
    want, status = call()
    assert status == 0
    for limit in (1, 500, 1500, 3000, 8000, 25000):
        ts.set_wait_limit_ns(limit)
        try:
            got, status = call()
        finally:
            ts.set_wait_limit_ns(0)
        assert status in (0, TIMEOUT) and (limit > 1 or status == TIMEOUT)
        if status == 0:
            assert torch.equal(got, want)
        got, status = call()
        assert status == 0 and torch.equal(got, want)


@pools
@pytest.mark.parametrize("sequences,kernel", [(40, 0), (3, 0), (40, 5), (40, 1)], ids=["two", "one", "units", "simt"])
def test_a_batch_without_new_tokens_writes_nothing(ts, cuda_device, sequences, kernel, e4m3):  # noqa: F811
    """Rows that no sequence owns, as in a captured call whose sequences have all ended; then one sequence has a token."""
    p, go, sl = make_shared(cuda_device, [(100, [b for b in range(sequences)])], [1] * sequences, 32, 8, 128, "bf16", e4m3, seed=59)
    p.chunk_offsets.zero_()
    for out, status in (run_chunk_shared(ts, p, go, sl, kernel), run_chunk_window(ts, p, 50, 2, kernel)):
        assert status == 0 and (out == 3).all()
    p.chunk_offsets[2:] = 1
    p.new = [int(b == 1) for b in range(sequences)]
    for (out, status), window in ((run_chunk_shared(ts, p, go, sl, kernel), (1 << 30, 0)), (run_chunk_window(ts, p, 50, 2, kernel), (50, 2))):
        assert status == 0 and (out[1:] == 3).all()
        check_attention(out[:1], *chunk64(p, *window), 200, 128, "bf16", kernel != 1)
