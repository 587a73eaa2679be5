"""Refusals of the calls with sliding windows and shared prefixes: every argument the host can check fails
with its error code before any launch.  Runs without a GPU (the fake device pointers are never read)."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import eagle_speculative_tree_gb300 as ts  # noqa: E402

FAKE = 0x10000
WS = FAKE * 256
BIG = 1 << 40
NULL, SHAPE, DTYPE, WORKSPACE, ALIGN, DEVICE = -1, -2, -3, -4, -6, -7


def chunk_shape(**kw):
    base = dict(batch=2, num_tokens=40, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16,
                max_pages_per_seq=64, num_pool_pages=200, dtype=ts.DTYPE_BF16, kv_dtype=ts.DTYPE_BF16)
    base.update(kw)
    return ts.ChunkProblem(**base).c_shape()


def tree_shape(**kw):
    base = dict(batch=2, num_nodes=8, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, max_pages_per_seq=129,
                num_pool_pages=200, dtype=ts.DTYPE_BF16)
    base.update(kw)
    return ts.AttnProblem(**base).c_shape()


def calls(chunk=None, tree=None, kv=ts.DTYPE_BF16, window=16, sinks=4, groups=2, ws=WS, wsb=BIG, **ptr):
    """Return codes of the four calls: chunk window, tree window, chunk shared, tree shared."""
    lib = ts.raw_library()
    names = ("q", "k", "v", "ks", "vs", "pt", "pl", "rows")
    a = [ptr.get(n, FAKE) for n in names]
    g = [ptr.get("go", FAKE), ptr.get("sl", FAKE)]
    out = [ptr.get("out", FAKE)]
    c, t = ctypes.byref(chunk or chunk_shape()), ctypes.byref(tree or tree_shape())
    return (lib.tree_chunk_attn_window(*a, *out, c, window, sinks, ws, wsb, None),
            lib.tree_attn_verify_window(*a, *out, t, kv, window, sinks, ws, wsb, None),
            lib.tree_chunk_attn_shared(*a, *g, *out, c, groups, ws, wsb, None),
            lib.tree_attn_verify_shared(*a, *g, *out, t, kv, groups, ws, wsb, None))


def sizes(chunk=None, tree=None, kv=ts.DTYPE_BF16, window=16, sinks=4, groups=2):
    lib = ts.raw_library()
    c, t = ctypes.byref(chunk or chunk_shape()), ctypes.byref(tree or tree_shape())
    return (lib.treespec_chunk_window_workspace_bytes(c, window, sinks),
            lib.treespec_attn_window_workspace_bytes(t, kv, window, sinks),
            lib.treespec_chunk_shared_workspace_bytes(c, groups), lib.treespec_attn_shared_workspace_bytes(t, kv, groups))


@pytest.mark.parametrize("name", ["q", "k", "v", "pt", "pl", "rows", "out"])
def test_null_pointers(name):
    assert calls(**{name: None}) == (NULL,) * 4


@pytest.mark.parametrize("name", ["go", "sl"])
def test_null_groups(name):
    assert calls(**{name: None})[2:] == (NULL,) * 2


@pytest.mark.parametrize("name", ["ks", "vs"])
def test_scales_are_needed_with_8_bit_pools(name):
    assert calls(chunk_shape(kv_dtype=ts.DTYPE_E4M3), kv=ts.DTYPE_E4M3, **{name: None}) == (NULL,) * 4
    assert calls(chunk_shape(kv_dtype=ts.DTYPE_E4M3), kv=ts.DTYPE_E4M3, **{name: FAKE + 4}) == (ALIGN,) * 4


@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
def test_alignment(name):
    assert calls(**{name: FAKE + 8}) == (ALIGN,) * 4


def test_workspace():
    assert calls(ws=None) == (WORKSPACE,) * 4 and calls(ws=WS + 64) == (WORKSPACE,) * 4


def test_windows_and_sinks():
    for kw in (dict(window=0), dict(window=-1), dict(window=-(1 << 31)), dict(sinks=-1), dict(sinks=-(1 << 31))):
        assert calls(**kw)[:2] == (SHAPE,) * 2 and sizes(**kw)[:2] == (0, 0)
    top = (1 << 31) - 1
    assert all(sizes(window=top, sinks=top)) and all(sizes(window=1, sinks=0))


def test_groups():
    for n in (0, -1, 1025, 1 << 30, -(1 << 31)):
        assert calls(groups=n)[2:] == (SHAPE,) * 2 and sizes(groups=n)[2:] == (0, 0)
    assert all(sizes(groups=1024))
    # the persistent form holds batch + groups entries
    full = dict(batch=1020, kernel=ts.KERNEL_TC_STREAM)
    assert all(sizes(chunk_shape(num_tokens=1020, **full), tree_shape(**full), groups=4)[2:])
    assert sizes(chunk_shape(num_tokens=1020, **full), tree_shape(**full), groups=5)[2:] == (0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(num_q_heads=30), SHAPE), (dict(num_kv_heads=0), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(page_size=32), SHAPE), (dict(max_pages_per_seq=0), SHAPE),
    (dict(num_pool_pages=0), SHAPE), (dict(dtype=ts.DTYPE_E4M3), DTYPE), (dict(kernel=ts.KERNEL_TC), SHAPE),
    (dict(kernel=9), SHAPE), (dict(num_q_heads=129, num_kv_heads=1), SHAPE),
    (dict(dtype=ts.DTYPE_F32, kernel=ts.KERNEL_TC_STREAM), DTYPE),
])
def test_bad_shapes(kw, code):
    kv = dict(kv_dtype=kw["dtype"]) if "dtype" in kw else {}
    bad = dict(chunk=chunk_shape(**kw, **kv), tree=tree_shape(**kw), kv=kw.get("dtype", ts.DTYPE_BF16))
    assert calls(**bad) == (code,) * 4
    assert sizes(**bad) == (0,) * 4


def test_pool_types():
    for q, kv in ((ts.DTYPE_BF16, ts.DTYPE_F32), (ts.DTYPE_F32, ts.DTYPE_BF16), (ts.DTYPE_BF16, 7), (ts.DTYPE_F32, -1)):
        bad = dict(chunk=chunk_shape(dtype=q, kv_dtype=kv), tree=tree_shape(dtype=q), kv=kv)
        assert calls(**bad) == (DTYPE,) * 4 and sizes(**bad) == (0,) * 4
    assert calls(tree=tree_shape(num_nodes=129))[1::2] == (SHAPE,) * 2


def test_a_null_shape():
    lib = ts.raw_library()
    assert lib.tree_chunk_attn_window(*[FAKE] * 9, None, 16, 0, WS, BIG, None) == NULL
    assert lib.tree_attn_verify_shared(*[FAKE] * 11, None, ts.DTYPE_BF16, 1, WS, BIG, None) == NULL
    assert lib.treespec_attn_window_workspace_bytes(None, 0, 16, 0) == 0


def test_valid_calls_stop_at_the_device_check():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert calls() == (DEVICE,) * 4
    assert calls(ks=None, vs=None) == (DEVICE,) * 4              # no scales over plain pools
    assert calls(chunk_shape(kv_dtype=ts.DTYPE_E4M3, dtype=ts.DTYPE_F32), tree_shape(dtype=ts.DTYPE_F32), ts.DTYPE_E4M3,
                 window=1 << 30, sinks=1 << 30) == (DEVICE,) * 4


def test_binding_refusals_name_the_argument():
    """Checks that the binding makes before it reaches the library (CPU tensors)."""
    import torch
    q, tq = torch.zeros(4, 8, 64), torch.zeros(1, 4, 8, 64)
    pool, table = torch.zeros(3, 16, 2, 64), torch.zeros(1, 2, dtype=torch.int32)
    ints = torch.zeros(2, dtype=torch.int32)
    for w in (0, -5):
        with pytest.raises(ValueError, match="window"):
            ts.tree_chunk_attn_window(q, pool, pool, table, ints[:1], ints, w)
    with pytest.raises(ValueError, match="sinks"):
        ts.tree_attn_verify_window(tq, pool, pool, table, ints[:1], table, 4, -1)
    with pytest.raises(TypeError):
        ts.tree_chunk_attn_window(q, pool, pool, table, ints[:1], ints, 4.5)
    with pytest.raises(ValueError, match="shared_lens"):
        ts.tree_chunk_attn_shared(q, pool, pool, table, ints[:1], ints, ints[:1], ints[:0])
    with pytest.raises(ValueError, match="group_offsets must be a tensor"):
        ts.tree_attn_verify_shared(tq, pool, pool, table, ints[:1], table, [0, 1], ints)
    for call in (lambda x: ts.tree_chunk_attn_window(x, pool, pool, table, ints[:1], ints, 4),
                 lambda x: ts.tree_chunk_attn_shared(x, pool, pool, table, ints[:1], ints, ints, ints[:1])):
        with pytest.raises(ValueError, match="q must be on a CUDA device"):
            call(q)
        with pytest.raises(ValueError, match="q must be float32 or bfloat16"):
            call(q.double())
        with pytest.raises(ValueError, match="q must be a tensor"):
            call(None)
    with pytest.raises(ValueError, match="unsupported"):
        ts.chunk_window_workspace_bytes(ts.ChunkProblem(1, 1, 3, 2, 64, 16, 1, 1, 0, 0), 4)
    with pytest.raises(ValueError, match="unsupported"):
        ts.attn_shared_workspace_bytes(ts.AttnProblem(1, 1, 2, 2, 64, 16, 1, 1, 0), 0, 0)
