"""Refusals of the chunk and 8-bit cache calls: every argument the host can check fails with its
error code before any launch.  Runs without a GPU (the fake device pointers are never read)."""
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


def options(**kw):
    base = dict(q_norm=FAKE, k_norm=FAKE, inv_freq=FAKE, positions=FAKE, norm_eps=1e-6, rope_scale=1.0, rot_dim=128,
                layout=ts.ROPE_HALF)
    base.update(kw)
    return ts.AppendOptions(**base)


def append(shape=None, opt=None, q=FAKE, k=FAKE, v=FAKE, out=FAKE, kp=FAKE, ks=None, vs=None, strides=None, pt=FAKE,
           off=FAKE, ws=WS, wsb=BIG):
    s = shape or chunk_shape()
    st = strides or (s.num_q_heads * s.head_dim, s.num_kv_heads * s.head_dim, s.num_kv_heads * s.head_dim)
    return ts.raw_library().tree_chunk_append(q, st[0], k, st[1], v, st[2], out, kp, FAKE, ks, vs, pt, FAKE, off,
                                              ctypes.byref(s), ctypes.byref(opt or options()), ws, wsb, None)


def attn(shape=None, q=FAKE, kp=FAKE, ks=None, vs=None, off=FAKE, out=FAKE, ws=WS, wsb=BIG):
    return ts.raw_library().tree_chunk_attn(q, kp, FAKE, ks, vs, FAKE, FAKE, off, out,
                                            ctypes.byref(shape or chunk_shape()), ws, wsb, None)


def no_device():
    import torch
    return not torch.cuda.is_available()


BAD_SHAPES = [
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(num_tokens=0), SHAPE), (dict(num_q_heads=30), SHAPE),
    (dict(num_kv_heads=0), SHAPE), (dict(num_q_heads=129, num_kv_heads=1), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(page_size=32), SHAPE), (dict(max_pages_per_seq=0), SHAPE), (dict(num_pool_pages=0), SHAPE),
    (dict(max_pages_per_seq=(1 << 26) + 1), SHAPE), (dict(num_tokens=1 << 30), SHAPE), (dict(dtype=7), DTYPE),
    (dict(dtype=ts.DTYPE_E4M3), DTYPE), (dict(kv_dtype=ts.DTYPE_F32), DTYPE), (dict(kernel=9), SHAPE),
    (dict(kernel=ts.KERNEL_TC_2SM), SHAPE),
]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_bad_shapes(kw, code):
    s = chunk_shape(**kw)
    assert append(s, strides=(1 << 20,) * 3) == code
    assert attn(s) == code
    assert ts.raw_library().treespec_chunk_attn_workspace_bytes(ctypes.byref(s)) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(out=None), NULL), (dict(off=None), NULL), (dict(kp=None), NULL),
    (dict(pt=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(v=FAKE + 4), ALIGN), (dict(kp=FAKE + 2), ALIGN),
    (dict(strides=(4095, 1024, 1024)), SHAPE), (dict(strides=(4096, 1024, 1023)), SHAPE),
    (dict(strides=(4097, 1024, 1024), out=FAKE * 3), ALIGN),
    (dict(strides=(6144, 1024, 1024)), SHAPE),                    # in place, but not packed
    (dict(ws=None), WORKSPACE), (dict(ws=WS + 64), WORKSPACE), (dict(wsb=8), WORKSPACE),
    (dict(opt=options(rot_dim=24)), SHAPE), (dict(opt=options(rot_dim=144)), SHAPE), (dict(opt=options(rot_dim=-16)), SHAPE),
    (dict(opt=options(layout=2)), SHAPE), (dict(opt=options(inv_freq=None)), NULL),
    (dict(opt=options(norm_eps=-1.0)), SHAPE), (dict(opt=options(norm_eps=float("nan"))), SHAPE),
    (dict(opt=options(rope_scale=float("inf"))), SHAPE), (dict(opt=options(k_norm=FAKE + 4)), ALIGN),
    (dict(shape=chunk_shape(kv_dtype=ts.DTYPE_E4M3)), NULL),
    (dict(shape=chunk_shape(kernel=ts.KERNEL_SIMT)), SHAPE),
])
def test_append_refusals(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(kp=None), NULL), (dict(off=None), NULL), (dict(out=None), NULL), (dict(q=FAKE + 8), ALIGN),
    (dict(out=FAKE + 8), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=WS + 128), WORKSPACE), (dict(wsb=255), WORKSPACE),
    (dict(shape=chunk_shape(kv_dtype=ts.DTYPE_E4M3)), NULL),
    (dict(shape=chunk_shape(kv_dtype=ts.DTYPE_E4M3), ks=FAKE, vs=FAKE + 4), ALIGN),
])
def test_attention_refusals(kw, code):
    if code == WORKSPACE and kw.get("wsb") and not no_device():
        pytest.skip("a device is present: the size is checked against its plan")
    rc = attn(**kw)
    assert rc == code or (kw.get("wsb") and rc == DEVICE)


def test_valid_calls_stop_at_the_device_check():
    if not no_device():
        pytest.skip("a device is present")
    assert append() == DEVICE
    assert append(strides=(8192, 2048, 1024), out=FAKE * 3) == DEVICE
    assert append(opt=options(rot_dim=0, inv_freq=None, q_norm=None, k_norm=None, positions=None)) == DEVICE
    assert attn() == DEVICE
    assert attn(chunk_shape(dtype=ts.DTYPE_F32, kv_dtype=ts.DTYPE_E4M3), ks=FAKE, vs=FAKE) == DEVICE
    assert attn(chunk_shape(kernel=ts.KERNEL_SIMT)) == DEVICE


def tree_shape(**kw):
    base = dict(batch=1, num_nodes=8, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, max_pages_per_seq=129,
                num_pool_pages=200, dtype=ts.DTYPE_BF16)
    base.update(kw)
    return ts.AttnProblem(**base).c_shape()


@pytest.mark.parametrize("kw,code", [
    (dict(num_nodes=129), SHAPE), (dict(num_nodes=0), SHAPE), (dict(batch=0), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(dtype=ts.DTYPE_E4M3), DTYPE), (dict(kernel=ts.KERNEL_TC), SHAPE), (dict(kernel=ts.KERNEL_TC_PAIR), SHAPE),
    (dict(num_q_heads=256, num_kv_heads=1, num_nodes=2), SHAPE),
])
def test_verify_e4m3_bad_shapes(kw, code):
    s = tree_shape(**kw)
    lib = ts.raw_library()
    assert lib.treespec_attn_e4m3_workspace_bytes(ctypes.byref(s)) == 0
    assert lib.tree_attn_verify_e4m3(*[FAKE] * 9, ctypes.byref(s), WS, BIG, None) == code


def test_verify_and_commit_e4m3_null_and_alignment():
    lib, s = ts.raw_library(), tree_shape()
    for i in range(9):
        args = [FAKE] * 9
        args[i] = None
        assert lib.tree_attn_verify_e4m3(*args, ctypes.byref(s), WS, BIG, None) == NULL
        assert lib.tree_kv_commit_e4m3(*args, ctypes.byref(s), WS, BIG, None) == NULL
    for i in (0, 3, 4):
        args = [FAKE] * 9
        args[i] = FAKE + 8
        assert lib.tree_attn_verify_e4m3(*args, ctypes.byref(s), WS, BIG, None) == ALIGN
    args = [FAKE] * 9
    args[2] = FAKE + 8
    assert lib.tree_kv_commit_e4m3(*args, ctypes.byref(s), WS, BIG, None) == ALIGN
    assert lib.tree_attn_verify_e4m3(*[FAKE] * 9, ctypes.byref(s), WS + 16, BIG, None) == WORKSPACE
    assert lib.tree_kv_commit_e4m3(*[FAKE] * 9, ctypes.byref(s), None, BIG, None) == WORKSPACE


def test_existing_calls_still_refuse_8_bit_pools():
    s = tree_shape(dtype=ts.DTYPE_E4M3)
    assert ts.raw_library().tree_attn_verify(*[FAKE] * 7, ctypes.byref(s), WS, BIG, None) == DTYPE
    assert ts.raw_library().tree_kv_commit(*[FAKE] * 7, ctypes.byref(s), WS, BIG, None) == DTYPE


def test_binding_refusals_name_the_argument():
    """Checks that the binding makes before it reaches the library (CPU tensors)."""
    import torch
    q = torch.zeros(4, 8, 64)
    pool = torch.zeros(3, 16, 2, 64)
    ints = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        ts.tree_chunk_attn(q.double(), pool, pool, table, ints[:1], ints)
    with pytest.raises(ValueError, match="q must be on"):
        ts.tree_chunk_attn(q, pool, pool, table, ints[:1], ints)
    with pytest.raises(ValueError, match="head_dim"):
        ts.chunk_problem(q, torch.zeros(3, 16, 2, 128), table, ints)
    with pytest.raises(ValueError, match="chunk_offsets"):
        ts.chunk_problem(q, pool, table, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_pages"):
        ts.tree_kv_commit_e4m3(pool, pool, pool, pool, table, ints, table, ints)
    with pytest.raises(ValueError, match="unsupported"):
        ts.chunk_attn_workspace_bytes(ts.ChunkProblem(1, 1, 3, 2, 64, 16, 1, 1, 0, 0))


def test_binding_names_an_argument_that_is_no_tensor():
    import torch
    q, pool = torch.zeros(4, 8, 64), torch.zeros(3, 16, 2, 64)
    table, offsets = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for name in ("q", "k_pages", "page_table", "chunk_offsets"):
        args = dict(q=q, k_pages=pool, page_table=table, chunk_offsets=offsets)
        args[name] = None
        with pytest.raises(ValueError, match=f"{name} must be a tensor, got NoneType"):
            ts.chunk_problem(**args)
    for call, n in ((ts.tree_chunk_attn, 6), (ts.tree_chunk_append, 8), (ts.tree_attn_verify_e4m3, 8)):
        with pytest.raises(ValueError, match="q must be a tensor, got list"):
            call(*[[1.0]] * n)
    with pytest.raises(ValueError, match="k_pages must be a tensor"):
        ts.tree_kv_commit_e4m3(*[None] * 8)
