"""Windows and shared prefixes on the GPU where a program can go wrong with them: values that are not finite, bad
lengths, pages and groups, graphs, streams, limits, and a serving run with all of the cache's calls."""
import numpy as np
import pytest
import torch

from gen import trees

from chunk_util import Problem, check_attention, make
from test_gpu_window import (BAD_LENGTH, BAD_PAGE, BAD_PARENT, TIMEOUT, check_chunk_shared, check_chunk_window, ints, kv_dtype,
                             on_tensor_cores, run_chunk_shared, run_chunk_window, run_tree_shared, run_tree_window,
                             shared_tree_problem, tree_problem, ts, types)  # noqa: F401
from window_util import chunk64, drop_pages, make_shared, tree64

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def put(p, b, t, what, value, h=1, d=5):
    """A value into K or V of logical token t of sequence b: an element, or over 8-bit pools a NaN code (for a NaN) or the
    token's scale."""
    page, at = int(p.page_table[b, t // 16]), t % 16
    pages, scales = (p.k_pages, p.k_scales) if what == "k" else (p.v_pages, p.v_scales)
    if scales is None:
        pages[page, at, h, d] = value
    elif value != value:
        pages.view(torch.uint8)[page, at, h, d] = 0x7f
    else:
        scales[page, h, at] = value


def dt(p):
    return "bf16" if p.q.dtype == torch.bfloat16 else "f32"


# ------------------------------------------------------------------------------ values that are not finite

WINDOWED = [
    # prefix, new, hq, hkv, dim, window, sinks
    ([100, 130], [1, 1], 8, 2, 128, 40, 3),                    # 4 rows of a unit
    ([90, 300], [5, 12], 8, 8, 64, 37, 0),                     # a few tokens of one head each
    ([200, 61], [3, 2], 20, 4, 128, 70, 5),
    ([150, 20], [60, 100], 8, 2, 128, 50, 2),
]


@types
@pytest.mark.parametrize("case", WINDOWED, ids=lambda c: f"{sum(c[1])}x{c[2]}-d{c[4]}")
@pytest.mark.parametrize("what", ["v", "k"])
def test_a_nan_reaches_the_rows_whose_window_holds_it(ts, cuda_device, case, what, dtype, e4m3, kernel):  # noqa: F811
    """NaN just behind the first row's window, in it, in the last row's alone, among the new tokens and in a sink."""
    prefix, new, hq, hkv, dim, window, sinks = case
    p = make(cuda_device, prefix, new, hq, hkv, dim, dtype, e4m3, seed=sum(prefix))
    for b, (S, n) in enumerate(zip(prefix, new)):
        spots = [S - window, S - window + 1 + b, S - window + n // 2, S + n // 2, sinks]
        for i, t in enumerate(spots):
            if 0 <= t < S + n:
                put(p, b, t, what, NAN, h=i % hkv, d=(7 * i) % dim)
    out, status = run_chunk_window(ts, p, window, sinks, kernel)
    assert status == 0
    check_attention(out, *chunk64(p, window, sinks), window + sinks, dim, dtype, on_tensor_cores(ts, p, kernel))


@types
@pytest.mark.parametrize("bad", [INF, -INF])
def test_an_infinity_outside_the_window_reaches_nobody(ts, cuda_device, bad, dtype, e4m3, kernel):  # noqa: F811
    for prefix, new, hq, hkv in (([100], [1], 8, 2), ([100], [9], 8, 2), ([100], [40], 4, 1)):
        p = make(cuda_device, prefix, new, hq, hkv, 128, dtype, e4m3, seed=3)
        window, sinks, n = 33, 2, new[0]
        for t in (100 - window, 3, 2):                         # of no row
            put(p, 0, t, "v", bad, h=0)
            put(p, 0, t, "k", bad, h=0)
        assert check_chunk_window(ts, p, window, sinks, kernel) == 0
        t = 100 + n // 2                                       # of the rows from n / 2 on
        clean, _ = run_chunk_window(ts, p, window, sinks, kernel)
        put(p, 0, t, "v", bad, h=0)
        out, _ = run_chunk_window(ts, p, window, sinks, kernel)
        G = hq // hkv
        touched = torch.zeros_like(out, dtype=torch.bool)
        touched[n // 2:, :G, :] = True
        if not e4m3:
            touched[n // 2:, :G] = False
            touched[n // 2:, :G, 5] = True
        assert not torch.isfinite(out[touched]).all()
        assert torch.isfinite(out[~touched]).all()
        assert (out[~touched].float() - clean[~touched].float()).abs().max() <= 2.0 ** -7 * clean.float().abs().max()


@types
def test_scores_of_minus_infinity_weigh_nothing_in_a_window(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    """The oldest tokens of the window and a sink: rows that see others take those alone."""
    for prefix, new, hq in (([200, 90], [1, 1], 8), ([200, 90], [6, 30], 4)):
        p = make(cuda_device, prefix, new, hq, 2, 128, dtype, e4m3, seed=5)
        p.q[:] = p.q.abs() * 0.2 + 0.01
        window, sinks = 64, 2
        for b, S in enumerate(prefix):
            for t in [0, *range(S - window + 1, S - window + 40)]:
                page, at = int(p.page_table[b, t // 16]), t % 16
                if e4m3:
                    p.k_pages.view(torch.uint8)[page, at] = 0x38
                    p.k_scales[page, :, at] = -INF
                else:
                    p.k_pages[page, at, :, 5] = -INF
        out, status = run_chunk_window(ts, p, window, sinks, kernel)
        for b, S in enumerate(prefix):                         # what weighs nothing may as well hold zeros in V
            for t in [0, *range(S - window + 1, S - window + 40)]:
                page, at = int(p.page_table[b, t // 16]), t % 16
                if e4m3:
                    p.k_scales[page, :, at] = -3e4
                else:
                    p.k_pages[page, at, :, 5] = -1e7 if dtype == "bf16" else -1e8
        assert status == 0
        ref, spread, _ = chunk64(p, window, sinks)
        for b, S in enumerate(prefix):
            for t in [0, *range(S - window + 1, S - window + 40)]:
                page, at = int(p.page_table[b, t // 16]), t % 16
                if e4m3:
                    p.k_scales[page, :, at] = 0
                else:
                    p.k_pages[page, at] = 0
        reach = chunk64(p, window, sinks)[2]
        check_attention(out, ref, spread, reach, window + sinks, 128, dtype, on_tensor_cores(ts, p, kernel))


@types
def test_a_nan_in_a_tree_reaches_the_nodes_that_see_it(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    for sizes, N, hq, window in (([7, 12], 12, 8, 30), ([3, 4], 4, 8, 6), ([40, 64], 64, 16, 9)):
        p, q, parents = tree_problem(cuda_device, [80, 33], sizes, N, hq, 4, 128, dtype, e4m3, N)
        for b, (S, n) in enumerate(zip(p.prefix, p.new)):
            put(p, b, S + n // 2, "v", NAN, h=0)
            put(p, b, S + n - 1, "v", NAN, h=1)
            put(p, b, S - window + 2, "v", NAN, h=2)
            put(p, b, S + 1, "k", NAN, h=3)
        out, status = run_tree_window(ts, p, q, parents, window, 1, kernel)
        assert status == 0
        check_attention(out, *tree64(p, q, parents.cpu().numpy(), window, 1), 160, 128, dtype, on_tensor_cores(ts, p, kernel))


@types
def test_a_nan_of_one_sequence_stays_with_it_and_a_shared_one_reaches_all(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    for new, hq in (([1, 1, 1], 8), ([3, 1, 2], 8), ([30, 1, 20], 4)):
        p, go, sl = make_shared(cuda_device, [(200, [10, 40, 0])], new, hq, 2, 128, dtype, e4m3, seed=7)
        put(p, 1, 205, "v", NAN, h=0, d=9)
        put(p, 0, 200 + 10 + new[0] - 1, "k", NAN, h=1)
        if new[2] > 1:
            put(p, 2, 200 + new[2] - 1, "v", NAN, h=1, d=60)
        out, status = run_chunk_shared(ts, p, go, sl, kernel)
        assert status == 0
        check_attention(out, *chunk64(p), 300, 128, dtype, on_tensor_cores(ts, p, kernel))
        put(p, 0, 70, "v", NAN, h=0, d=33)                     # in a page that all share
        put(p, 0, 5, "k", NAN, h=1)
        out, status = run_chunk_shared(ts, p, go, sl, kernel)
        assert status == 0
        check_attention(out, *chunk64(p), 300, 128, dtype, on_tensor_cores(ts, p, kernel))


@types
def test_queries_that_are_not_finite_spoil_their_own_rows(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    for new in ([1, 1, 1, 1], [3, 9, 30, 2]):
        p, go, sl = make_shared(cuda_device, [(130, [0, 9, 60, 30])], new, 8, 2, 128, dtype, e4m3, seed=9)
        row = [0, new[0], p.q.shape[0] - 1]
        p.q[row[0], 3, 5], p.q[row[1], 6, 100], p.q[row[2], 0, 0] = NAN, INF, -INF
        for out, (window, sinks) in ((run_chunk_shared(ts, p, go, sl, kernel)[0], (1 << 30, 0)),
                                     (run_chunk_window(ts, p, 50, 4, kernel)[0], (50, 4))):
            ref, spread, reach = chunk64(p, window, sinks)
            for r, h in zip(row, (3, 6, 0)):
                assert torch.isnan(out[r, h]).all()
                out[r, h] = 0
                ref[r, h] = spread[r, h] = reach[r, h] = 0
            check_attention(out, ref, spread, reach, 300, 128, dtype, on_tensor_cores(ts, p, kernel))


# ------------------------------------------------------------------------------ bad lengths, pages, groups

@types
def test_pages_outside_the_pool_count_as_zeros_where_a_row_sees_them(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    for new in ([1, 1], [5, 40]):
        p = make(cuda_device, [300, 100], new, 8, 2, 128, dtype, e4m3, seed=11)
        drop_pages(p, 100, 20)
        table = p.page_table.clone()
        for b, i in ((0, 1), (0, 17), (1, 3)):                 # a sink's, two of the windows'
            page = int(table[b, i])
            for pages in (p.k_pages, p.v_pages):
                (pages.view(torch.uint8) if e4m3 else pages)[page] = 0
            for s in (p.k_scales, p.v_scales):
                if s is not None:
                    s[page] = 1
        want, status = run_chunk_window(ts, p, 100, 20, kernel)
        assert status == 0
        for b, i, bad in ((0, 1, -1), (0, 17, p.k_pages.shape[0]), (1, 3, 1 << 30)):
            p.page_table[b, i] = bad
        got, status = run_chunk_window(ts, p, 100, 20, kernel)
        assert status == BAD_PAGE and torch.equal(got, want)


@types
def test_bad_prefix_lengths_give_zeros(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    for new in ([1, 1, 1], [3, 20, 7]):
        p, go, sl = make_shared(cuda_device, [(0, [60]), (70, [60, 70])], new, 8, 2, 64, dtype, e4m3, seed=13)
        off = p.chunk_offsets.tolist()
        for bad in (-1, (1 << 31) - 1, 16 * p.page_table.shape[1]):
            p.prefix_lens.copy_(ints(p.prefix, cuda_device))
            want = run_chunk_window(ts, p, 30, 2, kernel)[0], run_chunk_shared(ts, p, go, sl, kernel)[0]
            p.prefix_lens[1] = bad
            for (got, status), ref in zip((run_chunk_window(ts, p, 30, 2, kernel), run_chunk_shared(ts, p, go, sl, kernel)), want):
                assert status == BAD_LENGTH and (got[off[1]:off[2]] == 0).all()
                keep = torch.ones(got.shape[0], dtype=torch.bool, device=cuda_device)
                keep[off[1]:off[2]] = False
                tol = 2.0 ** -7 if dtype == "bf16" else 1e-5   # another order of sums where nothing is shared any more
                assert (got[keep].float() - ref[keep].float()).abs().max() <= tol * ref.float().abs().max()


@types
def test_groups_that_do_not_hold_share_nothing(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    p, go, sl = make_shared(cuda_device, [(100, [3, 0]), (300, [40, 9, 1]), (0, [70])], [2, 1, 1, 4, 1, 3], 8, 2, 128, dtype,
                            e4m3, seed=15)
    assert check_chunk_shared(ts, p, go, sl, kernel) == 0
    # 301 is no longer than the prefixes of 340, 309 and 301 tokens, and whole tiles of 64 end before their contents differ
    for lens, status in (([101, 300, 0], BAD_LENGTH), ([-1, 300, 0], BAD_LENGTH), ([100, 301, 0], 0), ([100, 302, 0], BAD_LENGTH),
                         ([(1 << 31) - 1, 300, 71], BAD_LENGTH), ([100, 300, -(1 << 31)], BAD_LENGTH)):
        assert check_chunk_shared(ts, p, go, ints(lens, cuda_device), kernel) == status
    for offsets in ([0, 3, 2, 6], [-1, 2, 5, 6], [0, 2, 5, 7], [0, 2, 1 << 30, 6], [6, 5, 2, 0]):
        assert check_chunk_shared(ts, p, ints(offsets, cuda_device), sl, kernel) == BAD_LENGTH
    assert check_chunk_shared(ts, p, ints([0, 0, 0, 0], cuda_device), sl, kernel) == 0          # no sequence in a group


@types
def test_offsets_out_of_order_touch_nothing_else(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    p, go, sl = make_shared(cuda_device, [(64, [10, 10, 10])], [10, 10, 10], 4, 1, 64, dtype, e4m3, seed=17)
    for offsets in ([0, 10, 400, 30], [-5, 10, 20, 30], [0, 20, 10, 30], [0, (1 << 31) - 1, -1, 30]):
        p.chunk_offsets.copy_(ints(offsets, cuda_device))
        for out, status in (run_chunk_window(ts, p, 20, 1, kernel), run_chunk_shared(ts, p, go, sl, kernel)):
            assert status & BAD_LENGTH
            kept = [t for t in range(30) if not any(0 <= a <= t < z <= 30 for a, z in zip(offsets, offsets[1:]))]
            assert (out[kept] == 3).all()


@types
def test_bad_trees_are_flagged(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    p, q, parents = tree_problem(cuda_device, [40, 50], [8, 8], 8, 8, 2, 64, dtype, e4m3, 21)
    parents[0, 3] = 5
    assert run_tree_window(ts, p, q, parents, 20, 1, kernel)[1] == BAD_PARENT
    go, sl = ints([0, 2], cuda_device), ints([0], cuda_device)
    assert run_tree_shared(ts, p, q, parents, go, sl, kernel)[1] == BAD_PARENT
    parents[0, 3] = 0
    p.prefix_lens[1] = -3
    out, status = run_tree_window(ts, p, q, parents, 20, 1, kernel)
    assert status == BAD_LENGTH and (out[1] == 0).all()
    out, status = run_tree_shared(ts, p, q, parents, go, sl, kernel)
    assert status == BAD_LENGTH and (out[1] == 0).all()


# ------------------------------------------------------------------------------ limits

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("sequences", [1023, 1024])
def test_the_most_entries_of_a_call(ts, cuda_device, sequences, e4m3):  # noqa: F811
    """1024 sequences and groups take the tensor cores, one more the CUDA cores."""
    lens = [70 + b % 50 for b in range(sequences)]
    p, go, sl = make_shared(cuda_device, [(64, [n - 64 for n in lens])], [1] * sequences, 4, 1, 64, "bf16", e4m3, seed=23)
    assert check_chunk_shared(ts, p, go, sl) == 0
    assert check_chunk_window(ts, p, 33, 3) == 0


def test_many_groups(ts, cuda_device):  # noqa: F811
    groups = [(64 + 16 * (g % 5), [g % 7, 0]) for g in range(300)]
    p, go, sl = make_shared(cuda_device, groups, [1, 2] * 300, 8, 2, 64, "bf16", seed=25)
    assert check_chunk_shared(ts, p, go, sl) == 0
    p, go, sl = make_shared(cuda_device, groups[:200], [1, 30] * 200, 8, 2, 64, "bf16", seed=25)
    assert check_chunk_shared(ts, p, go, sl) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_waits_that_run_out_leave_the_next_call_right(ts, cuda_device, e4m3):  # noqa: F811
    cases = []
    for groups, new, hq in (([(900, [100, 7, 300, 0])], [1, 1, 1, 1], 16), ([(700, [30, 0])], [70, 1], 16)):
        p, go, sl = make_shared(cuda_device, groups, new, hq, 2, 128, "bf16", e4m3, seed=27)
        cases.append(lambda p=p, go=go, sl=sl: run_chunk_shared(ts, p, go, sl))
        cases.append(lambda p=p: run_chunk_window(ts, p, 333, 5))
    for call in cases:
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


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_pool_larger_than_32_bit_offsets(ts, cuda_device, e4m3):  # noqa: F811
    pages = 300_000 if e4m3 else 280_000
    p, go, sl = make_shared(cuda_device, [(64, [100, 31])], [9, 1], 16, 8, 128, "bf16", e4m3, seed=29)
    want = [run_chunk_window(ts, p, 80, 3)[0], run_chunk_shared(ts, p, go, sl)[0]]
    small = p.k_pages.shape[0]
    for name in ("k", "v"):
        old = getattr(p, name + "_pages")
        big = torch.empty((pages,) + tuple(old.shape[1:]), dtype=old.dtype, device=cuda_device)
        big[pages - small:].view(torch.uint8).copy_(old.view(torch.uint8))
        setattr(p, name + "_pages", big)
        if e4m3:
            s = torch.empty((pages, 8, 16), device=cuda_device)
            s[pages - small:] = getattr(p, name + "_scales")
            setattr(p, name + "_scales", s)
    p.page_table += pages - small
    for (got, status), ref in zip((run_chunk_window(ts, p, 80, 3), run_chunk_shared(ts, p, go, sl)), want):
        assert status & ~BAD_PAGE == 0 and torch.equal(got, ref)


# ------------------------------------------------------------------------------ graphs and streams

@types
def test_captured_calls_replay_over_other_lengths_and_groups(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    """Two graphs of both calls, one workspace, replayed in turn with lengths, values and groups changed between."""
    for new in ([1, 1, 1, 1], [3, 1, 0, 40]):
        p, go, sl = make_shared(cuda_device, [(320, [100, 60, 30, 10])], new, 8, 2, 128, dtype, e4m3, seed=31)
        prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets, kernel=kernel)
        ws = torch.empty(max(ts.chunk_window_workspace_bytes(prob, 100, 5), ts.chunk_shared_workspace_bytes(prob, 1)),
                         dtype=torch.uint8, device=cuda_device)
        outs = [torch.full_like(p.q, 3.0) for _ in range(2)]
        args = (p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets)

        def step(**more):
            ts.tree_chunk_attn_window(*args, 100, 5, outs[0], workspace=ws, kernel=kernel, **more, **p.scales())
            ts.tree_chunk_attn_shared(*args, go, sl, outs[1], workspace=ws, kernel=kernel, **more, **p.scales())

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(stream=side)
        side.synchronize()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            graphs.append(g)
        for turn, g in enumerate(graphs * 2):
            p.q.normal_()
            own = [100 - 7 * turn, 60, 30 - turn, 10 - 3 * turn]   # within the tokens that are there
            p.prefix_lens.copy_(ints([320 + o for o in own], cuda_device))
            sl.copy_(ints([(320, 130, 0, 257)[turn]], cuda_device))
            for o in outs:
                o.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for o in outs:
                o.fill_(3.0)
            step(stream=side)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
            p.prefix = p.prefix_lens.tolist()
            for out, (window, sinks) in zip(got, ((100, 5), (1 << 30, 0))):
                check_attention(out, *chunk64(p, window, sinks), 500, 128, dtype, on_tensor_cores(ts, p, kernel))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_calls_at_once_with_a_workspace_each(ts, cuda_device, e4m3):  # noqa: F811
    p, go, sl = make_shared(cuda_device, [(900, [100, 5, 64, 0] * 4)], [1] * 16, 16, 2, 128, "bf16", e4m3, seed=33)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)
    want = [run_chunk_window(ts, p, 300, 4)[0], run_chunk_shared(ts, p, go, sl)[0]]
    args = (p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets)
    streams = [torch.cuda.Stream() for _ in range(4)]
    size = max(ts.chunk_window_workspace_bytes(prob, 300, 4), ts.chunk_shared_workspace_bytes(prob, 1))
    spaces = [torch.empty(size, dtype=torch.uint8, device=cuda_device) for _ in streams]
    outs = [[torch.empty_like(p.q) for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(6):
        for k, (st, ws) in enumerate(zip(streams, spaces)):
            if (i + k) % 2:
                ts.tree_chunk_attn_shared(*args, go, sl, outs[k][i], workspace=ws, stream=st, **p.scales())
            else:
                ts.tree_chunk_attn_window(*args, 300, 4, outs[k][i], workspace=ws, stream=st, **p.scales())
    torch.cuda.synchronize()
    assert all(torch.equal(outs[k][i], want[(i + k) % 2]) for k in range(4) for i in range(6))


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_serving_with_a_window_layer_and_a_layer_behind_a_shared_prompt(ts, cuda_device, e4m3):  # noqa: F811
    """Four samples of one prompt through a layer with a window and one without: the prompt once, its pages in all
    tables; then rounds of a draft tree (append, verify in both layers, accept, commit), and a decoded token.  The window
    layer's pages are given back as the window passes them."""
    hq, hkv, D, B, N, window, sinks = 8, 2, 128, 4, 10, 48, 4
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(8)
    prompt, pages_per = 176, 8
    shared_pages = prompt // 16
    pool = shared_pages + B * pages_per + 2
    order = torch.randperm(pool, generator=gen, device=cuda_device).to(torch.int32)
    table = torch.empty((B, shared_pages + pages_per), dtype=torch.int32, device=cuda_device)
    table[:, :shared_pages] = order[:shared_pages]
    table[:, shared_pages:] = order[shared_pages:shared_pages + B * pages_per].view(B, -1)
    f = (10000.0 ** (-torch.arange(0, D, 2, device=cuda_device) / D)).float()
    caches, tables = [], [table.clone(), table]
    for _ in range(2):
        if e4m3:
            c = dict(k_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device).to(torch.float8_e4m3fn),
                     v_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device).to(torch.float8_e4m3fn),
                     k_scales=torch.ones((pool, hkv, 16), device=cuda_device),
                     v_scales=torch.ones((pool, hkv, 16), device=cuda_device))
        else:
            c = dict(k_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device, dtype=torch.bfloat16),
                     v_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device, dtype=torch.bfloat16))
        caches.append(c)

    def append(layer, n, prefix, offsets, positions=None, rows=slice(None)):
        x = torch.randn((n, hq + 2 * hkv, D), generator=gen, device=cuda_device).to(torch.bfloat16)
        return ts.tree_chunk_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], page_table=tables[layer][rows].contiguous(),
                                    prefix_lens=prefix, chunk_offsets=offsets, positions=positions, inv_freq=f, **caches[layer])

    def problem(layer, q, prefix, new, offsets):
        c = caches[layer]
        return Problem(prefix.tolist(), new, q, c["k_pages"], c["v_pages"], c.get("k_scales"), c.get("v_scales"), tables[layer],
                       prefix, offsets)

    zero, go, sl = ints([0], cuda_device), ints([0, B], cuda_device), ints([prompt], cuda_device)
    for layer in range(2):                                     # the prompt, by the first sequence's table
        first = slice(0, 1)
        off = ints([0, prompt], cuda_device)
        q = append(layer, prompt, zero, off, rows=first)
        t1 = tables[layer][first].contiguous()
        c = caches[layer]
        args = (q, c["k_pages"], c["v_pages"], t1, zero, off)
        scales = {k: v for k, v in c.items() if "scales" in k}
        out = ts.tree_chunk_attn(*args, **scales) if layer else ts.tree_chunk_attn_window(*args, window, sinks, **scales)
        p = Problem([0], [prompt], q, c["k_pages"], c["v_pages"], c.get("k_scales"), c.get("v_scales"), t1, zero, off)
        check_attention(out, *chunk64(p, *((1 << 30, 0) if layer else (window, sinks))), prompt, D, "bf16", True)
    prefix = ints([prompt] * B, cuda_device)
    rng = np.random.default_rng(4)
    for turn in range(3):
        parents = np.stack([trees.random_recursive(rng, N) for _ in range(B)])
        depth = np.stack([trees.depths(x) for x in parents])
        par = ints(parents, cuda_device)
        off = ints(np.arange(B + 1) * N, cuda_device)
        pos = ints((prefix.cpu().numpy()[:, None] + depth).reshape(-1), cuda_device)
        logits = torch.randn((B, N, 50), generator=gen, device=cuda_device)
        tokens = logits.argmax(-1)[torch.arange(B)[:, None], torch.from_numpy(np.maximum(parents, 0))].to(torch.int32)
        path, length, _ = ts.tree_accept(logits, tokens, None, par, None, 0.0)
        for layer in range(2):
            q = append(layer, B * N, prefix, off, pos).view(B, N, hq, D)
            c = caches[layer]
            scales = {k: v for k, v in c.items() if "scales" in k}
            args = (q, c["k_pages"], c["v_pages"], tables[layer], prefix, par)
            out = ts.tree_attn_verify_shared(*args, go, sl, **scales) if layer else \
                ts.tree_attn_verify_window(*args, window, sinks, **scales)
            p = problem(layer, None, prefix, [N] * B, off)
            check_attention(out, *tree64(p, q, parents, *((1 << 30, 0) if layer else (window, sinks))), 400, D, "bf16", True)
            more = dict(page_table=tables[layer], prefix_lens=prefix, accept_path=path, accept_len=length)
            new = ts.tree_kv_commit_e4m3(**c, **more) if e4m3 else ts.tree_kv_commit(c["k_pages"], c["v_pages"], **more)
        prefix = new
        # the window layer gives back what the window has passed: entries that no row sees any more
        low = prefix.min().item() - window + 1
        tables[0][:, (sinks + 15) // 16:max(low // 16, 1)] = -7
    off = ints(np.arange(B + 1), cuda_device)
    for layer in range(2):
        q = append(layer, B, prefix, off)
        p = problem(layer, q, prefix, [1] * B, off)
        out, status = run_chunk_shared(ts, p, go, sl) if layer else run_chunk_window(ts, p, window, sinks)
        assert status == 0
        check_attention(out, *chunk64(p, *((1 << 30, 0) if layer else (window, sinks))), 400, D, "bf16", True)


# ------------------------------------------------------------------------------ few rows to a sequence

FEW = pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (8, 2, 64), (32, 2, 128), (16, 1, 64)])


@FEW
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_bad_pages_of_decoded_tokens(ts, cuda_device, hq, hkv, dim, e4m3):  # noqa: F811
    """Each page of a step and of a tile of 64 tokens bad in turn, several at once, through a window and behind a shared
    prefix: zeros in their place, and nothing else changes."""
    p, go, sl = make_shared(cuda_device, [(192, [100, 30, 230])], [1, 1, 1], hq, hkv, dim, "bf16", e4m3, seed=dim + hq)
    spots = [(0, 12), (0, 13), (0, 14), (0, 15), (1, 12), (1, 13), (2, 16), (2, 19), (2, 21), (2, 25)]   # own tokens
    table = p.page_table.clone()
    for b, i in spots:
        page = int(table[b, i])
        for pages, scales in ((p.k_pages, p.k_scales), (p.v_pages, p.v_scales)):
            (pages.view(torch.uint8) if e4m3 else pages)[page] = 0
            if scales is not None:
                scales[page] = 1
    calls = [lambda: run_chunk_window(ts, p, 230, 200), lambda: run_chunk_shared(ts, p, go, sl)]
    want = [call() for call in calls]
    assert all(status == 0 for _, status in want)
    for n, (b, i) in enumerate(spots):
        p.page_table[b, i] = (-1, p.k_pages.shape[0], -(1 << 31), (1 << 31) - 1)[n % 4]
        if n % 3 == 0 or n + 1 == len(spots):
            for call, (ref, _) in zip(calls, want):
                got, status = call()
                assert status == BAD_PAGE and torch.equal(got, ref)
    p.page_table[2, 5] = -1                                    # a shared page, of one sequence: the group reads the first's
    got, status = calls[1]()
    assert status == BAD_PAGE and torch.equal(got, want[1][0])


@FEW
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_a_prompt_among_decoded_tokens(ts, cuda_device, hq, hkv, dim, e4m3):  # noqa: F811
    """The mean decides for units of few rows, and one sequence has many of them."""
    G = hq // hkv
    n = 60 + 12 * G
    lens = [(37 * b) % 400 for b in range(n)]
    new = [0 if G == 16 and b % 5 == 0 else 1 for b in range(n)]   # a mean of up to 16 rows
    new[6], new[40] = 45, 0
    assert sum(new) * G <= 16 * n
    p = make(cuda_device, lens, new, hq, hkv, dim, "bf16", e4m3, seed=3 * dim + hq)
    assert check_chunk_window(ts, p, 70, 3) == 0
    p, go, sl = make_shared(cuda_device, [(128, lens[:50]), (0, lens[50:51]), (64, lens[51:])], new, hq, hkv, dim, "bf16", e4m3,
                            seed=5 * dim + hq)
    assert check_chunk_shared(ts, p, go, sl) == 0


@types
def test_the_same_call_gives_the_same_bits(ts, cuda_device, dtype, e4m3, kernel):  # noqa: F811
    """Whatever ran in between and however the launches fell together."""
    p, go, sl = make_shared(cuda_device, [(320, [(53 * b) % 300 for b in range(24)]), (640, [1, 200, 77])], [1, 2] * 13 + [1], 8, 2,
                            128, dtype, e4m3, seed=41)
    other = make(cuda_device, [700, 20], [3, 90], 8, 2, 128, dtype, e4m3, seed=43)
    want = [run_chunk_shared(ts, p, go, sl, kernel)[0], run_chunk_window(ts, p, 200, 4, kernel)[0]]
    for i in range(12):
        if i % 3 == 2:
            run_chunk_window(ts, other, 50, 1, kernel)
        assert torch.equal(run_chunk_shared(ts, p, go, sl, kernel)[0], want[0])
        assert torch.equal(run_chunk_window(ts, p, 200, 4, kernel)[0], want[1])


@pytest.mark.parametrize("dtype,e4m3", [("f32", False), ("f32", True), ("bf16", False)])
def test_more_entries_than_the_tensor_cores_take(ts, cuda_device, dtype, e4m3):  # noqa: F811
    """1300 sequences, some without new tokens, in 400 groups, some of them empty or of one sequence."""
    sizes = [(g * 7) % 5 for g in range(400)]
    sizes[-1] += 1300 - sum(sizes) if sum(sizes) < 1300 else 0
    groups = [(16 * (g % 9), [(11 * (g + k)) % 60 for k in range(n)]) for g, n in enumerate(sizes)]
    B = sum(sizes)
    new = [(b % 4) if b % 10 else 0 for b in range(B)]
    p, go, sl = make_shared(cuda_device, groups, new, 4, 1, 64, dtype, e4m3, seed=47)
    assert B > 700 and check_chunk_shared(ts, p, go, sl) == 0
    assert check_chunk_window(ts, p, 21, 2) == 0
