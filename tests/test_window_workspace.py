"""Workspaces of the calls with sliding windows and shared prefixes, by the form that a shape takes, as the header states
them.  Runs without a GPU (152 SMs are assumed)."""
import __graft_entry__

__graft_entry__.build()
import eagle_speculative_tree_gb300 as ts  # noqa: E402

MB = 1e6


def chunks(batch, tokens, hq=32, hkv=8):
    return ts.ChunkProblem(batch=batch, num_tokens=tokens, num_q_heads=hq, num_kv_heads=hkv, head_dim=128, page_size=16,
                           max_pages_per_seq=64, num_pool_pages=2000, dtype=ts.DTYPE_BF16, kv_dtype=ts.DTYPE_BF16)


def states(p):
    return 8 * 130 * p.num_tokens * p.num_q_heads


def test_windows():
    few, many, wide = chunks(64, 64), chunks(64, 640), chunks(64, 64, 64, 2)
    assert 4 * MB < ts.chunk_window_workspace_bytes(few, 100, 4) < 6 * MB
    assert 38 * MB < ts.chunk_window_workspace_bytes(many, 100, 4) < 42 * MB
    assert 38 * MB < ts.chunk_window_workspace_bytes(wide, 100, 4) < 42 * MB   # 32 heads to a kv head


def test_shared_prefixes():
    small, two, many = chunks(2, 2), chunks(64, 64), chunks(64, 640)
    assert 4 * MB < ts.chunk_shared_workspace_bytes(small, 1) - states(small) < 6 * MB
    assert 43 * MB < ts.chunk_shared_workspace_bytes(two, 2) - states(two) < 47 * MB
    assert 38 * MB < ts.chunk_shared_workspace_bytes(many, 2) - states(many) < 42 * MB


def test_more_entries_than_the_tensor_cores_take():
    for groups, on_tensor_cores in ((24, True), (25, False)):
        p = chunks(1000, 1000)
        n = ts.chunk_shared_workspace_bytes(p, groups) - states(p)
        assert (n > 43 * MB) == on_tensor_cores
