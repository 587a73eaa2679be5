"""tree_chunk_attn_window, tree_attn_verify_window, tree_chunk_attn_shared and tree_attn_verify_shared on the
GPU, against oracle.window and the definition in 64 bits."""
import numpy as np
import pytest
import torch

from gen import trees
from oracle import window as ow

from chunk_util import check_attention, make
from window_util import chunk64, drop_pages, make_shared, rows64, tree64

pytestmark = pytest.mark.gpu

BAD_PARENT, BAD_PAGE, BAD_LENGTH, TIMEOUT = 1, 2, 4, 16


@pytest.fixture(scope="module")
def ts():
    import __graft_entry__
    __graft_entry__.build()
    import eagle_speculative_tree_gb300 as mod
    return mod


def ints(a, device):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(device)


def kv_dtype(ts, p):
    return ts.DTYPE_E4M3 if p.k_scales is not None else ts.DTYPE_BF16 if p.q.dtype == torch.bfloat16 else ts.DTYPE_F32


def on_tensor_cores(ts, p, kernel):
    return p.q.dtype == torch.bfloat16 and kernel != ts.KERNEL_SIMT


# kernels to run a type on: the CUDA cores take all, the tensor cores bf16 queries (in units of 256 rows, or by
# their number where the call chooses)
TYPES = [("f32", False, 0), ("f32", True, 0), ("bf16", False, 0), ("bf16", True, 0), ("bf16", False, 5), ("bf16", True, 5),
         ("bf16", False, 1), ("bf16", True, 1)]
TYPE_IDS = ["f32", "f32-e4m3", "bf16", "bf16-e4m3", "bf16-units", "bf16-e4m3-units", "bf16-simt", "bf16-e4m3-simt"]
types = pytest.mark.parametrize("dtype,e4m3,kernel", TYPES, ids=TYPE_IDS)


# ------------------------------------------------------------------------------ windows: chunks

def run_chunk_window(ts, p, window, sinks, kernel=0, fill=3.0):
    out = torch.full_like(p.q, fill)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets, kernel=kernel)
    ws = torch.empty(ts.chunk_window_workspace_bytes(prob, window, sinks), dtype=torch.uint8, device=p.q.device)
    ws.fill_(0xa5)                                             # what a workspace holds does not matter
    got = ts.tree_chunk_attn_window(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, window, sinks,
                                    out, workspace=ws, kernel=kernel, **p.scales())
    assert got is out
    return out, ts.read_status(ws)


def check_chunk_window(ts, p, window, sinks, kernel=0):
    out, status = run_chunk_window(ts, p, window, sinks, kernel)
    off = p.chunk_offsets.tolist()
    ref, spread, reach = chunk64(p, window, sinks)
    tokens = max(min(S + n, window + sinks) for S, n in zip(p.prefix, p.new))
    check_attention(out[off[0]:off[-1]], ref, spread, reach, tokens, p.q.shape[2], "bf16" if p.q.dtype == torch.bfloat16 else
                    "f32", on_tensor_cores(ts, p, kernel))
    assert (out[:off[0]] == 3).all() and (out[off[-1]:] == 3).all(), "a row of no sequence changed"
    return status


CHUNKS = [
    # prefix, new, hq, hkv, dim, window, sinks
    ([0], [1], 4, 1, 64, 1, 0),
    ([100], [1], 8, 2, 128, 1, 1),
    ([100, 3, 700], [1, 1, 1], 32, 8, 128, 64, 4),
    ([700, 40, 0, 513], [1, 9, 30, 0], 8, 2, 128, 33, 17),
    ([2000], [130], 12, 4, 64, 127, 0),
    ([0, 0, 90], [300, 17, 200], 4, 1, 128, 100, 3),
    ([0], [700], 4, 4, 64, 65, 64),                            # unit longer than the window
    ([1500], [260], 32, 32, 128, 20, 130),
    ([64, 128, 63, 65], [64, 1, 65, 3], 7, 1, 64, 64, 64),
    ([900, 901], [5, 6], 20, 4, 128, 1 << 30, 0),              # reaches all
    ([900, 10], [5, 60], 20, 4, 64, 5, 1 << 30),               # so do the sinks
    ([31] * 70, [1, 2, 0] * 23 + [5], 8, 2, 64, 16, 2),
    ([3000, 200], [1, 40], 64, 1, 128, 700, 5),                # 64 heads to a kv head
]


@types
@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: f"{sum(c[1])}x{c[2]}-d{c[4]}-w{c[5]}-s{c[6]}")
def test_chunk_window(ts, cuda_device, case, dtype, e4m3, kernel):
    prefix, new, hq, hkv, dim, window, sinks = case
    p = make(cuda_device, prefix, new, hq, hkv, dim, dtype, e4m3, seed=sum(new) + window % 1000, lead=2, tail=3)
    drop_pages(p, window, sinks)
    assert check_chunk_window(ts, p, window, sinks, kernel) == 0


@types
@pytest.mark.parametrize("window,sinks", [(1, 0), (15, 1), (16, 16), (17, 15), (48, 0), (63, 3), (64, 65), (129, 33), (300, 64)])
def test_chunk_window_borders(ts, cuda_device, window, sinks, dtype, e4m3, kernel):
    """Windows and sinks around pages and tiles, over prefixes around them."""
    prefix = [0, 15, 16, 17, 47, 63, 64, 65, 127, 128, 191, 200, 333]
    new = [3, 1, 2, 70, 1, 2, 1, 64, 1, 3, 5, 1, 9]
    p = make(cuda_device, prefix, new, 8, 2, 64, dtype, e4m3, seed=window, lead=1, tail=1)
    drop_pages(p, window, sinks)
    assert check_chunk_window(ts, p, window, sinks, kernel) == 0


# ------------------------------------------------------------------------------ windows: trees

def run_tree_window(ts, p, q, parents, window, sinks, kernel=0):
    out = torch.full_like(q, 3.0)
    prob = ts.attn_problem(q, p.k_pages, p.page_table, kernel=kernel)
    ws = torch.empty(ts.attn_window_workspace_bytes(prob, kv_dtype(ts, p), window, sinks), dtype=torch.uint8, device=q.device)
    ws.fill_(0xa5)
    ts.tree_attn_verify_window(q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, parents, window, sinks, out,
                               workspace=ws, kernel=kernel, **p.scales())
    return out, ts.read_status(ws)


def tree_problem(device, prefix, sizes, N, hq, hkv, dim, dtype, e4m3, seed, kind="random"):
    rng = np.random.default_rng([seed, 9])
    shape = {"random": lambda n: trees.random_recursive(rng, n), "chain": trees.chain, "star": trees.star}[kind]
    parents = trees.padded([shape(n) for n in sizes], N)
    p = make(device, prefix, sizes, hq, hkv, dim, dtype, e4m3, seed=seed)
    q = torch.from_numpy(rng.standard_normal((len(sizes), N, hq, dim)).astype(np.float32)).to(device).to(p.q.dtype)
    for b, n in enumerate(sizes):
        q[b, n:] = float("nan")                                # of padding rows nothing matters
    return p, q, ints(parents, device)


TREES = [
    # prefix, nodes, N, hq, hkv, dim, window, sinks, kind
    ([100], [8], 8, 32, 8, 128, 50, 4, "random"),
    ([0, 5, 200], [1, 16, 9], 16, 8, 2, 64, 7, 3, "random"),
    ([300, 77], [60, 64], 64, 64, 8, 128, 100, 4, "random"),
    ([130], [100], 100, 4, 1, 128, 20, 0, "chain"),            # a chain longer than the window
    ([3], [128], 128, 8, 2, 64, 5, 10, "chain"),               # sinks among the tree's own positions
    ([90, 64], [40, 65], 65, 28, 4, 128, 1, 0, "star"),
    ([1000, 1, 500], [33, 2, 20], 33, 32, 32, 64, 64, 65, "random"),
    ([700], [30], 30, 12, 4, 128, 1 << 30, 0, "random"),
]


@types
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{len(c[1])}x{c[2]}x{c[3]}-d{c[5]}-w{c[6]}-s{c[7]}-{c[8]}")
def test_tree_window(ts, cuda_device, case, dtype, e4m3, kernel):
    prefix, sizes, N, hq, hkv, dim, window, sinks, kind = case
    p, q, parents = tree_problem(cuda_device, prefix, sizes, N, hq, hkv, dim, dtype, e4m3, sum(sizes), kind)
    drop_pages(p, window, sinks)
    out, status = run_tree_window(ts, p, q, parents, window, sinks, kernel)
    assert status == 0
    ref, spread, reach = tree64(p, q, parents.cpu().numpy(), window, sinks)
    tokens = max(min(S + n, window + sinks + n) for S, n in zip(prefix, sizes))
    check_attention(out, ref, spread, reach, tokens, dim, dtype, on_tensor_cores(ts, p, kernel))


# ------------------------------------------------------------------------------ shared prefixes

def run_chunk_shared(ts, p, group_offsets, shared_lens, kernel=0):
    out = torch.full_like(p.q, 3.0)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets, kernel=kernel)
    ws = torch.empty(ts.chunk_shared_workspace_bytes(prob, shared_lens.shape[0]), dtype=torch.uint8, device=p.q.device)
    ws.fill_(0xa5)
    ts.tree_chunk_attn_shared(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, group_offsets,
                              shared_lens, out, workspace=ws, kernel=kernel, **p.scales())
    return out, ts.read_status(ws)


def check_chunk_shared(ts, p, group_offsets, shared_lens, kernel=0):
    out, status = run_chunk_shared(ts, p, group_offsets, shared_lens, kernel)
    off = p.chunk_offsets.tolist()
    ref, spread, reach = chunk64(p)
    check_attention(out[off[0]:off[-1]], ref, spread, reach, max(S + n for S, n in zip(p.prefix, p.new)), p.q.shape[2],
                    "bf16" if p.q.dtype == torch.bfloat16 else "f32", on_tensor_cores(ts, p, kernel))
    assert (out[:off[0]] == 3).all() and (out[off[-1]:] == 3).all(), "a row of no sequence changed"
    return status


SHARED = [
    # groups of (shared, own cached), new, hq, hkv, dim
    ([(64, [0, 0])], [1, 1], 8, 2, 128),
    ([(300, [5, 0, 100, 17])], [1, 1, 1, 1], 32, 8, 128),
    ([(63, [1, 2]), (64, [0, 9, 0]), (0, [40, 30]), (1000, [10])], [2, 3, 1, 0, 5, 1, 1, 4], 4, 1, 64),
    ([(128, [0] * 40), (191, [3] * 30)], [1] * 70, 8, 2, 64),
    ([(700, [20, 300, 1])], [130, 2, 64], 12, 4, 128),
    ([(2000, [0, 1, 2, 3, 4, 5])], [7, 1, 3, 2, 9, 1], 28, 4, 64),
    ([(512, [10, 20]), (640, [30, 40])], [300, 280, 1, 2], 8, 8, 128),
    ([(1600, list(range(33)))], [1] * 33, 64, 1, 128),
    ([(256, [0, 50, 0])], [0, 3, 0], 8, 2, 64),                # one sequence with new tokens
]


@types
@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"{len(c[0])}g-{sum(c[1])}x{c[2]}-d{c[4]}")
def test_chunk_shared(ts, cuda_device, case, dtype, e4m3, kernel):
    groups, new, hq, hkv, dim = case
    p, go, sl = make_shared(cuda_device, groups, new, hq, hkv, dim, dtype, e4m3, seed=sum(new), lead=2, tail=3)
    assert check_chunk_shared(ts, p, go, sl, kernel) == 0


@types
def test_chunk_shared_by_pages_of_equal_content(ts, cuda_device, dtype, e4m3, kernel):
    p, go, sl = make_shared(cuda_device, [(200, [3, 9, 0]), (70, [1, 1])], [2, 1, 4, 1, 30], 8, 2, 128, dtype, e4m3, seed=5,
                            copies=True)
    assert check_chunk_shared(ts, p, go, sl, kernel) == 0


@types
def test_groups_need_not_cover_the_batch(ts, cuda_device, dtype, e4m3, kernel):
    p, go, sl = make_shared(cuda_device, [(0, [40]), (150, [3, 9, 0]), (300, [8, 8]), (0, [7, 0])], [2, 1, 4, 1, 3, 2, 1, 9],
                            8, 2, 64, dtype, e4m3, seed=6, lead=1)
    assert check_chunk_shared(ts, p, go[1:-1].contiguous(), sl[1:-1].contiguous(), kernel) == 0
    # groups without sequences, at both ends and between
    go2 = torch.cat((go[1:2], go[1:3], go[2:3], go[2:4], go[3:4]))
    sl2 = ints([5, 150, 1 << 20, 64, 300, 0][:go2.shape[0] - 1], cuda_device)
    assert go2.tolist() == [1, 1, 4, 4, 4, 6, 6] and check_chunk_shared(ts, p, go2, sl2, kernel) == 0


def run_tree_shared(ts, p, q, parents, group_offsets, shared_lens, kernel=0):
    out = torch.full_like(q, 3.0)
    prob = ts.attn_problem(q, p.k_pages, p.page_table, kernel=kernel)
    ws = torch.empty(ts.attn_shared_workspace_bytes(prob, kv_dtype(ts, p), shared_lens.shape[0]), dtype=torch.uint8,
                     device=q.device)
    ws.fill_(0xa5)
    ts.tree_attn_verify_shared(q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, parents, group_offsets, shared_lens, out,
                               workspace=ws, kernel=kernel, **p.scales())
    return out, ts.read_status(ws)


def shared_tree_problem(device, groups, sizes, N, hq, hkv, dim, dtype, e4m3, seed):
    rng = np.random.default_rng([seed, 10])
    parents = trees.padded([trees.random_recursive(rng, n) for n in sizes], N)
    p, go, sl = make_shared(device, groups, sizes, hq, hkv, dim, dtype, e4m3, seed=seed)
    q = torch.from_numpy(rng.standard_normal((len(sizes), N, hq, dim)).astype(np.float32)).to(device).to(p.q.dtype)
    for b, n in enumerate(sizes):
        q[b, n:] = float("nan")
    return p, q, ints(parents, device), go, sl


SHARED_TREES = [
    # groups, nodes, N, hq, hkv, dim
    ([(64, [0, 3])], [8, 8], 8, 32, 8, 128),
    ([(300, [5, 0, 100])], [1, 16, 9], 16, 8, 2, 64),
    ([(700, [20, 30]), (100, [0, 0, 7])], [60, 64, 3, 1, 40], 64, 64, 8, 128),
    ([(1000, [0] * 20)], [5, 8, 1, 3] * 5, 8, 28, 4, 128),
    ([(129, [64, 1])], [128, 100], 128, 4, 4, 64),
]


@types
@pytest.mark.parametrize("case", SHARED_TREES, ids=lambda c: f"{len(c[0])}g-{len(c[1])}x{c[2]}x{c[3]}-d{c[5]}")
def test_tree_shared(ts, cuda_device, case, dtype, e4m3, kernel):
    groups, sizes, N, hq, hkv, dim = case
    p, q, parents, go, sl = shared_tree_problem(cuda_device, groups, sizes, N, hq, hkv, dim, dtype, e4m3, sum(sizes))
    out, status = run_tree_shared(ts, p, q, parents, go, sl, kernel)
    assert status == 0
    ref, spread, reach = tree64(p, q, parents.cpu().numpy())
    check_attention(out, ref, spread, reach, max(S + n for S, n in zip(p.prefix, p.new)), dim, dtype,
                    on_tensor_cores(ts, p, kernel))


# ------------------------------------------------------------------------------ few rows, long ragged ranges

@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (64, 4, 128), (16, 8, 64), (12, 1, 64)])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decoded_tokens_of_many_ragged_sequences(ts, cuda_device, hq, hkv, dim, e4m3):
    """Ranges of many units of odd numbers of tiles, so that their steps and ring stages fall to other warps each time;
    several calls, which have to agree to the bit."""
    rng = np.random.default_rng([hq, dim])
    prefix = [int(x) for x in rng.integers(0, 4000, 30)] + [0, 1, 63, 64, 2999]
    p = make(cuda_device, prefix, [1] * len(prefix), hq, hkv, dim, "bf16", e4m3, seed=dim)
    window, sinks = 1501, 70
    assert drop_pages(p, window, sinks) > 100
    assert check_chunk_window(ts, p, window, sinks) == 0
    first, _ = run_chunk_window(ts, p, window, sinks)
    for _ in range(5):
        assert torch.equal(run_chunk_window(ts, p, window, sinks)[0], first)


@pytest.mark.parametrize("hq,hkv,dim", [(32, 8, 128), (64, 4, 64)])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decoded_tokens_behind_shared_prefixes(ts, cuda_device, hq, hkv, dim, e4m3):
    rng = np.random.default_rng([hq, dim, 1])
    groups = [(1000, [int(x) for x in rng.integers(0, 900, 20)]), (3007, [int(x) for x in rng.integers(0, 300, 17)]),
              (130, [int(x) for x in rng.integers(0, 2500, 9)])]
    B = sum(len(own) for _, own in groups)
    p, go, sl = make_shared(cuda_device, groups, [1] * B, hq, hkv, dim, "bf16", e4m3, seed=dim)
    assert check_chunk_shared(ts, p, go, sl) == 0
    first, _ = run_chunk_shared(ts, p, go, sl)
    for _ in range(5):
        assert torch.equal(run_chunk_shared(ts, p, go, sl)[0], first)
