"""Shared prefixes where the groups' rows and the sequences' own are two launches side by side."""
import numpy as np
import pytest
import torch

from chunk_util import check_attention
from test_gpu_window import ints, run_chunk_shared, ts  # noqa: F401
from window_util import chunk64, make_shared

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
