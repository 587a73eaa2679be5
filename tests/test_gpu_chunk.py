"""tree_chunk_append, tree_chunk_attn, tree_attn_verify_e4m3 and tree_kv_commit_e4m3 on the GPU,
against oracle.chunk and oracle.attention in 64 bits."""
import numpy as np
import pytest
import torch

from gen import trees
from oracle import attention as oatt
from oracle import chunk as och
from oracle import kv_commit as okc

from chunk_util import U_BF16, U_E4M3, U_F32, causal64, check_attention, make, make_8bit, tree64

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_LENGTH = 2, 4


@pytest.fixture(scope="module")
def ts():
    import __graft_entry__
    __graft_entry__.build()
    import eagle_speculative_tree_gb300 as mod
    return mod


def ints(a, device):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(device)


# ------------------------------------------------------------------------------ append

def append_inputs(device, p, seed, rot, norm, fused=True):
    """q, k, v of the problem's rows (views of one projection's output) and the options."""
    rng = np.random.default_rng([seed, 5])
    T, hq, D = p.q.shape
    hkv = p.k_pages.shape[2]
    x = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, D)).astype(np.float32)).to(device).to(p.q.dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(device) if norm else None for _ in "qk"]
    f = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)).to(device) if rot else None
    return q, k, v, w[0], w[1], f


def check_append(ts, p, q, k, v, qw, kw, f, positions, layout, scale=1.0, eps=1e-6, in_place=False, **more):
    dev = p.q.device
    D, hq = q.shape[2], q.shape[1]
    e4m3 = p.k_scales is not None
    u = U_BF16 if q.dtype == torch.bfloat16 else U_F32
    host = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    hq64, hk64, hv64 = host(q), host(k), host(v)
    before = [t.clone() for t in (p.k_pages, p.v_pages)] + [None if s is None else s.clone() for s in (p.k_scales, p.v_scales)]
    q_before = q.clone() if in_place else torch.full_like(q.contiguous(), 7.0)
    q_out = q if in_place else q_before.clone()
    ws = torch.empty(ts.append_workspace_bytes(), dtype=torch.uint8, device=dev)
    got = ts.tree_chunk_append(q, k, v, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, q_out,
                               positions=positions, q_norm=qw, k_norm=kw, norm_eps=eps, inv_freq=f, rope=layout,
                               rope_scale=scale, workspace=ws, **p.scales(), **more)
    status = ts.read_status(ws)
    assert got is q_out
    f64 = () if f is None else f.double().cpu().numpy()
    rows, slots = och.append(hq64, hk64, hv64, p.page_table.cpu().numpy(), p.prefix_lens.cpu().numpy(),
                             p.chunk_offsets.cpu().numpy(), p.k_pages.shape[0],
                             positions=None if positions is None else positions.cpu().numpy(), q_norm=host(qw),
                             k_norm=host(kw), eps=eps, inv_freq=f64, interleaved=layout == ts.ROPE_INTERLEAVED,
                             rope_scale=scale)
    # a sum of D squares and its root: (D / 2 + 4) 2^-24; the products and the rotation: 8 more
    # roundings; cosine, sine and the angle's last bits: 2^-22 of either term of the rotation
    rel = (D / 2 + 12) * 2.0 ** -24 + 2.0 ** -22

    def slack(x):
        return 2 * abs(scale) * rel * np.abs(x).max(-1, keepdims=True) / max(min(abs(scale), 1), 1e-9)

    out = got.double().cpu().numpy()
    untouched = [t for t in range(q.shape[0]) if t not in rows]
    assert torch.equal(got[untouched], q_before[untouched])
    for t, ref in rows.items():
        assert (np.abs(out[t] - ref) <= slack(ref) + u * np.abs(ref)).all(), t
    written = np.zeros(p.k_pages.shape[:2], dtype=bool)
    for (page, at) in slots:
        written[page, at] = True
    for which, (pages, scales) in enumerate(((p.k_pages, p.k_scales), (p.v_pages, p.v_scales))):
        raw = lambda t: t.view(torch.uint8) if e4m3 else t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
        kept = torch.from_numpy(~written).to(dev)
        assert torch.equal(raw(pages)[kept], raw(before[which])[kept]), "a slot that belongs to no new token changed"
        if e4m3:
            s_new, s_old = (x.transpose(1, 2)[kept].view(torch.int32) for x in (scales, before[2 + which]))
            assert torch.equal(s_new, s_old)
            codes, sc = pages.view(torch.uint8).cpu().numpy(), scales.cpu().numpy().astype(np.float64)
        else:
            x64 = pages.double().cpu().numpy()
        for (page, at), kv in slots.items():
            ref = kv[which]
            if e4m3:
                big = np.abs(ref).max(-1)
                s = sc[page, :, at]
                assert (np.abs(s - np.maximum(big / 448, och.SCALE_MIN)) <= 2 * (rel + 2.0 ** -23) * s).all()
                back = och.e4m3_values()[codes[page, at]] * s[:, None]
                tol = (U_E4M3 * np.abs(ref) + 2.0 ** -10 * s[:, None]) * (1 + 2.0 ** -20) + 1.1 * slack(ref)
            else:
                back, tol = x64[page, at], u * np.abs(ref) + (slack(ref) if which == 0 else 0)
            assert (np.abs(back - ref) <= tol).all(), (which, page, at)
    return status


APPEND = [
    # prefix, new, hq, hkv, dim, dtype, e4m3, layout, rot, norm, fused
    ([2048], [1], 32, 8, 128, "bf16", False, 0, 128, False, True),
    ([0], [1], 4, 1, 64, "f32", False, 1, 64, True, True),
    ([5, 0, 31, 16], [3, 0, 17, 16], 8, 2, 128, "bf16", True, 0, 64, True, True),
    ([15, 100], [2, 33], 4, 4, 64, "f32", True, 1, 32, False, False),
    ([7, 9, 0], [130, 1, 64], 7, 1, 128, "bf16", False, 1, 80, True, True),
    ([3], [50], 64, 8, 64, "bf16", True, 0, 16, True, True),
    ([0] * 40, [1] * 40, 12, 4, 128, "f32", False, 0, 128, False, True),
    ([11, 4], [260, 140], 20, 4, 128, "bf16", True, 1, 0, True, True),     # no rotation
    ([1000], [400], 28, 4, 128, "bf16", False, 0, 96, True, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[5]}-{'e4m3' if c[6] else 'same'}-d{c[4]}-{sum(c[1])}x{c[2]}")
def test_append(ts, cuda_device, case):
    prefix, new, hq, hkv, dim, dtype, e4m3, layout, rot, norm, fused = case
    p = make(cuda_device, prefix, new, hq, hkv, dim, dtype, e4m3, seed=len(prefix) + sum(new), lead=2, tail=3)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 1, rot, norm, fused)
    assert check_append(ts, p, q, k, v, qw, kw, f, None, layout) == 0


def test_append_keys_normed_queries_not_and_scaled_rotation(ts, cuda_device):
    p = make(cuda_device, [40, 2], [9, 12], 8, 2, 128, "bf16", True, seed=3)
    q, k, v, _qw, kw, f = append_inputs(cuda_device, p, 2, 128, True)
    assert check_append(ts, p, q, k, v, None, kw, f / 8, None, 0, scale=1.25) == 0
    assert check_append(ts, p, q, k, v, kw, None, f, None, 1, scale=0.5, eps=0.0) == 0


def test_append_tree_positions_with_padding(ts, cuda_device):
    """A batch of padded trees: a node's position is its depth, padding rows are left out."""
    rng = np.random.default_rng(4)
    sizes, N, prefix = [5, 1, 16, 11], 16, [30, 0, 7, 250]
    parents = trees.padded([trees.random_recursive(rng, n) for n in sizes], N)
    pos = np.full((4, N), -1)
    for b, n in enumerate(sizes):
        for i in range(n):
            pos[b, i] = prefix[b] if i == 0 else pos[b, parents[b, i]] + 1
    # the page table ends after the tree's own nodes: the padding slots have no place at all
    p = make(cuda_device, prefix, sizes, 16, 4, 128, "bf16", True, seed=9, rows=None)
    p.q = torch.zeros((4 * N, 16, 128), dtype=torch.bfloat16, device=cuda_device)
    p.chunk_offsets = ints(np.arange(5) * N, cuda_device)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 3, 64, True)
    assert check_append(ts, p, q, k, v, qw, kw, f, ints(pos.reshape(-1), cuda_device), 0) == 0


def test_append_far_positions_keep_their_angle(ts, cuda_device):
    p = make(cuda_device, [0], [6], 2, 1, 64, "f32", seed=2)
    q, k, v, qw, kw, _ = append_inputs(cuda_device, p, 4, 64, False)
    f = torch.tensor([1.0, 0.9, 6.5, 1e-30, 0.0, 2.0 ** -126, 1e-42, 0.123] * 4, device=cuda_device)
    pos = ints([0, 1, 65536, 1048573, (1 << 30) + 7, (1 << 31) - 1], cuda_device)
    assert check_append(ts, p, q, k, v, qw, kw, f, pos, 0) == 0
    assert check_append(ts, p, q, k, v, qw, kw, -f, pos, 1) == 0


def test_append_in_place_queries(ts, cuda_device):
    p = make(cuda_device, [3, 70], [40, 5], 8, 2, 128, "bf16", seed=6, tail=2)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 5, 128, True, fused=False)
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0, in_place=True) == 0


@pytest.mark.parametrize("tokens", [1, 60])
def test_append_zero_and_non_finite_heads(ts, cuda_device, tokens):
    """An all-zero head keeps scale 2^-100 and codes 0; a head with a NaN or an infinity reads
    back as NaN throughout, its neighbours as they are."""
    p = make(cuda_device, [4], [tokens], 4, 4, 64, "f32", True, seed=8)
    q, k, v, *_ = append_inputs(cuda_device, p, 6, 0, False, fused=False)
    v[0, 0], v[0, 1, 5], v[0, 2, 63], k[0, 3, 0] = 0, float("inf"), float("nan"), float("-inf")
    ts.tree_chunk_append(q, k, v, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, **p.scales())
    page, at = int(p.page_table[0, 0]), 4
    kp, vp = p.pools64()
    assert (p.v_pages[page, at, 0].view(torch.uint8) == 0).all() and float(p.v_scales[page, 0, at]) == 2.0 ** -100
    assert np.isnan(vp[page, at, 1:3]).all() and np.isnan(kp[page, at, 3]).all()
    assert np.isfinite(vp[page, at, 3]).all() and np.isfinite(kp[page, at, :3]).all()


@pytest.mark.parametrize("tokens", [2, 300])
def test_append_refuses_bad_pages_and_lengths_row_by_row(ts, cuda_device, tokens):
    p = make(cuda_device, [10, 3, 20], [tokens] * 3, 4, 2, 64, "bf16", seed=1)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 7, 64, True)
    table = p.page_table.clone()
    p.page_table[0, 0] = -1
    p.page_table[1, 0] = p.k_pages.shape[0]
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0) == BAD_PAGE
    p.page_table = table
    p.prefix_lens[1] = -5
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0) == BAD_LENGTH
    p.prefix_lens[1] = table.shape[1] * 16 - 1                 # one row fits, the others run past the table
    table[1, -1] = table[1, 0]
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0) == BAD_LENGTH
    p.prefix_lens[1] = (1 << 31) - 1                           # positions past 32 bits
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0) == BAD_LENGTH
    p.prefix_lens[1] = 3
    p.chunk_offsets[2] = -7                                    # sequences 1 and 2 have no rows
    assert check_append(ts, p, q, k, v, qw, kw, f, None, 0) == BAD_LENGTH


# ------------------------------------------------------------------------------ attention

def attend(ts, p, kernel, out=None):
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets, kernel=kernel)
    ws = torch.full((ts.chunk_attn_workspace_bytes(prob),), 0xff, dtype=torch.uint8, device=p.q.device)
    if out is None:
        out = torch.full_like(p.q, float("nan"))
    got = ts.tree_chunk_attn(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, out, kernel=kernel,
                             workspace=ws, **p.scales())
    return got, ts.read_status(ws)


def check_chunk(ts, p, kernel, status=0):
    got, st = attend(ts, p, kernel)
    assert st == status
    kp, vp = p.pools64()
    ref = och.chunk_attention(p.q.double().cpu().numpy(), kp, vp, p.page_table.cpu().numpy(), p.prefix_lens.cpu().numpy(),
                              p.chunk_offsets.cpu().numpy())
    tokens = max(a + b for a, b in zip(p.prefix, p.new))
    dtype = "bf16" if p.q.dtype == torch.bfloat16 else "f32"
    check_attention(got, *ref, tokens, p.q.shape[2], dtype, dtype == "bf16")
    again, _ = attend(ts, p, kernel)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(got.view(bits), again.view(bits)), "the same call gave other bits"
    return got


ATTEND = [
    # prefix, new, hq, hkv, dim
    ([0], [1], 4, 1, 64),                                      # one token, nothing before it
    ([0, 1, 15, 16, 17], [1, 1, 1, 1, 1], 8, 2, 128),          # decoding around a page's end
    ([300, 0, 63, 64, 1000], [1] * 5, 32, 8, 128),
    ([0, 5, 130], [64, 65, 63], 4, 4, 128),
    ([0, 0, 0], [200, 1, 129], 8, 2, 64),                      # prompts
    ([127, 0, 40, 3], [33, 0, 0, 100], 8, 1, 128),             # empty sequences among them
    ([900], [260], 3, 1, 128),                                 # 3 heads share one
    ([10, 2000], [300, 2], 14, 2, 64),                         # 7 heads share one
    ([5], [40], 128, 1, 64),                                   # 128 heads share one
    ([50, 60], [20, 9], 65, 1, 128),                           # a token's heads fill half a tile and one more
    ([777] * 3, [16] * 3, 16, 16, 64),
    ([0], [700], 2, 2, 128),
]
KINDS = [("f32", False), ("bf16", False), ("f32", True), ("bf16", True)]


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"d{c[4]}-{c[2]}x{c[3]}-{max(c[0])}+{max(c[1])}")
@pytest.mark.parametrize("kernel", ["auto", "simt"])
def test_chunk_attention(ts, cuda_device, case, dtype, e4m3, kernel):
    prefix, new, hq, hkv, dim = case
    p = make(cuda_device, prefix, new, hq, hkv, dim, dtype, e4m3, seed=hq + sum(prefix), lead=1, tail=2, extra_pages=2)
    check_chunk(ts, p, ts.KERNEL_AUTO if kernel == "auto" else ts.KERNEL_SIMT)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
def test_chunk_attention_many_ragged_sequences(ts, cuda_device, dtype, e4m3):
    rng = np.random.default_rng(12)
    prefix = [int(x) for x in rng.integers(0, 900, 70)]
    new = [int(x) for x in rng.integers(0, 4, 70)]
    check_chunk(ts, make(cuda_device, prefix, new, 8, 2, 128, dtype, e4m3, seed=5), ts.KERNEL_AUTO)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("prefix,new", [([6000], [1]), ([3000, 0], [1, 1]), ([1500], [70])])
def test_chunk_attention_long_context_few_rows(ts, cuda_device, dtype, e4m3, prefix, new):
    check_chunk(ts, make(cuda_device, prefix, new, 8, 1, 128, dtype, e4m3, seed=15), ts.KERNEL_AUTO)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefix,new,hq,hkv", [
    ([20000], [1], 8, 1),                                      # one unit in more than 32 pieces
    ([20000] + [5] * 40, [1] * 41, 4, 1),                      # a long unit among short ones
    ([9000, 0, 700, 3], [1, 400, 3, 0], 16, 2),                # decoding beside a prompt
    ([3000] * 40, [2] * 40, 8, 8),                             # more units than SMs, each cut somewhere
])
def test_chunk_attention_cuts(ts, cuda_device, prefix, new, hq, hkv, e4m3):
    p = make(cuda_device, prefix, new, hq, hkv, 128, "bf16", e4m3, seed=17)
    check_chunk(ts, p, ts.KERNEL_TC_STREAM)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_attention_at_the_batch_limit(ts, cuda_device, e4m3):
    """1024 sequences run on the tensor cores, 1025 on CUDA cores; the explicit kernel is refused."""
    rng = np.random.default_rng(23)
    for B in (1024, 1025):
        prefix, new = rng.integers(0, 40, B).tolist(), rng.integers(0, 3, B).tolist()
        p = make(cuda_device, prefix, new, 4, 2, 64, "bf16", e4m3, seed=B)
        check_chunk(ts, p, ts.KERNEL_AUTO)
    with pytest.raises(ValueError):
        attend(ts, p, ts.KERNEL_TC_STREAM)
    p.q = p.q.float()
    if e4m3:
        with pytest.raises(ValueError):                        # float32 queries run on CUDA cores only
            attend(ts, p, ts.KERNEL_TC_STREAM)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(ts, cuda_device, e4m3):
    p = make(cuda_device, [2000, 300], [64, 70], 16, 2, 128, "bf16", e4m3, seed=19)
    ts.set_wait_limit_ns(1)
    try:
        _, st = attend(ts, p, ts.KERNEL_TC_STREAM)
    finally:
        ts.set_wait_limit_ns(0)
    assert st & 16
    check_chunk(ts, p, ts.KERNEL_TC_STREAM)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_values_reach_only_the_rows_that_see_them(ts, cuda_device, dtype, e4m3, bad):
    """Token 40 of a 70-token chunk holds a NaN or an infinity in V, token 55 in K: rows before
    them are what they are without them, whatever tile they share with them."""
    p = make(cuda_device, [100, 30], [70, 12], 8, 2, 128, dtype, e4m3, seed=21)
    clean, _ = attend(ts, p, ts.KERNEL_AUTO)
    for pages, scales, tok in ((p.v_pages, p.v_scales, 40), (p.k_pages, p.k_scales, 55)):
        pos = 100 + tok
        page, at = int(p.page_table[0, pos // 16]), pos % 16
        if e4m3:
            scales[page, 1, at] = bad
        else:
            pages[page, at, 1, 77] = bad
    got, st = attend(ts, p, ts.KERNEL_AUTO)
    assert st == 0
    same = torch.ones(82, 8, dtype=torch.bool, device=cuda_device)
    same[40:70, 4:] = False                                    # heads 4..7 read kv head 1
    assert torch.isfinite(got[same]).all()
    tol = (2 * U_BF16 if dtype == "bf16" else 1e-5) * clean.abs().amax().item()
    assert (got[same].double() - clean[same].double()).abs().max().item() <= tol
    seen = got[40:70, 4:, 77] if not e4m3 else got[40:70, 4:]
    assert not torch.isfinite(seen).any()
    if not e4m3 and bad != bad:                                # the other elements of V's rows are untouched
        assert torch.isfinite(got[40:55, 4:, :77]).all()


def test_chunk_attention_large_scores_and_equal_scores(ts, cuda_device):
    for dtype, e4m3 in KINDS:
        p = make(cuda_device, [200], [80], 4, 1, 128, dtype, e4m3, seed=31)
        p.q *= 40                                              # one key takes nearly all the weight
        check_chunk(ts, p, ts.KERNEL_AUTO)
        p.q.zero_()                                            # the mean of V
        check_chunk(ts, p, ts.KERNEL_AUTO)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
def test_scores_that_rise_along_the_sequence(ts, cuda_device, dtype, e4m3):
    """The running maximum grows at every tile: the accumulated rows are rescaled each time."""
    p = make(cuda_device, [700], [40], 8, 2, 128, dtype, e4m3, seed=33)
    ramp = torch.zeros(128, device=cuda_device)
    ramp[0] = 1
    p.q[:] = (p.q.float() * 0.05 + ramp * 20).to(p.q.dtype)
    for pos in range(740):
        page, at = int(p.page_table[0, pos // 16]), pos % 16
        if e4m3:
            p.k_scales[page, :, at] = 0.002 + 0.0004 * pos
            p.k_pages.view(torch.uint8)[page, at, :, 0] = 0x78   # 256
        else:
            p.k_pages[page, at, :, 0] = 0.1 * pos
    check_chunk(ts, p, ts.KERNEL_AUTO)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_e4m3_code_reads_as_its_value(ts, cuda_device, dtype, dim):
    """One row per token and equal scores over a single token: row 0 of each one-token sequence
    returns V itself.  256 sequences, V of sequence c filled with code c."""
    p = make(cuda_device, [0] * 256, [1] * 256, 2, 1, dim, dtype, True, seed=3)
    page = p.page_table[:, 0].long()
    codes = torch.arange(256, dtype=torch.uint8, device=cuda_device)
    p.v_pages.view(torch.uint8)[page, 0, 0, :] = codes[:, None]
    p.v_scales[page, 0, 0] = 0.75
    got, st = attend(ts, p, ts.KERNEL_AUTO)
    ref = och.e4m3_values()[:, None, None] * 0.75
    g = got.double().cpu().numpy()
    assert st == 0 and np.array_equal(np.isnan(g), np.broadcast_to(np.isnan(ref), g.shape))
    ok = ~np.isnan(ref[:, 0, 0])
    assert np.array_equal(g[ok], np.broadcast_to(ref, g.shape)[ok])   # at most 5 significant bits: exact
    # the same through K: scores 0.01 x code against a token of score 0, V one and zero
    p = make(cuda_device, [1] * 254, [1] * 254, 1, 1, dim, dtype, True, seed=4)
    page = p.page_table[:, 0].long()
    keep = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8, device=cuda_device)
    p.k_pages.view(torch.uint8)[page, :2] = 0
    p.v_pages.view(torch.uint8)[page, :2] = 0
    p.k_pages.view(torch.uint8)[page, 0, 0, 0] = keep
    p.v_pages.view(torch.uint8)[page, 0] = 0x38
    p.k_scales[page, 0, :2] = 0.01
    p.v_scales[page, 0, :2] = 1.0
    p.q.zero_()
    p.q[:, 0, 0] = dim ** 0.5 if dim == 64 else 11.3125
    check_chunk(ts, p, ts.KERNEL_AUTO)


def test_chunk_attention_bad_lengths_and_pages(ts, cuda_device):
    for dtype, e4m3 in KINDS:
        p = make(cuda_device, [40, 33, 64], [10, 20, 5], 8, 2, 128, dtype, e4m3, seed=41, tail=4)
        p.prefix_lens[1] = -3
        p.prefix[1] = -3
        check_chunk(ts, p, ts.KERNEL_AUTO, BAD_LENGTH)         # its rows are zeros
        p.prefix_lens[1] = p.page_table.shape[1] * 16 - 19
        check_chunk(ts, p, ts.KERNEL_AUTO, BAD_LENGTH)
        p.prefix_lens[1] = 33
        clean, _ = attend(ts, p, ts.KERNEL_AUTO)
        p.page_table[1, 1] = 1 << 30
        got, st = attend(ts, p, ts.KERNEL_AUTO)
        assert st == BAD_PAGE
        bits = torch.int16 if dtype == "bf16" else torch.int32
        keep = list(range(10)) + list(range(30, 39))
        assert torch.equal(got[keep].view(bits), clean[keep].view(bits)) and torch.isfinite(got[10:30]).all()


def test_chunk_attention_offsets_that_decrease(ts, cuda_device):
    """No read or write outside the rows; a sequence with bad offsets has no rows."""
    for dtype, e4m3 in KINDS:
        p = make(cuda_device, [40, 33, 64], [10, 20, 5], 8, 2, 128, dtype, e4m3, seed=43)
        clean, _ = attend(ts, p, ts.KERNEL_AUTO)
        p.chunk_offsets[:] = ints([0, 10, 400, 35], cuda_device)
        got, st = attend(ts, p, ts.KERNEL_AUTO)
        assert st == BAD_LENGTH
        bits = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(got[:10].view(bits), clean[:10].view(bits)) and torch.isnan(got[10:]).all()


def test_pool_larger_than_32_bit_offsets(ts, cuda_device):
    """Pages whose byte and element offsets pass 2^32."""
    for e4m3 in (False, True):
        pages, hkv = (300_000, 8) if e4m3 else (280_000, 8)
        p = make(cuda_device, [100, 31], [9, 1], 16, hkv, 128, "bf16", e4m3, seed=51)
        small = p.k_pages.shape[0]
        check_chunk(ts, p, ts.KERNEL_AUTO)
        want, _ = attend(ts, p, ts.KERNEL_AUTO)
        for name in ("k", "v"):
            old = getattr(p, name + "_pages")
            big = torch.empty((pages,) + tuple(old.shape[1:]), dtype=old.dtype, device=cuda_device)
            big[pages - small:].view(torch.uint8).copy_(old.view(torch.uint8))
            setattr(p, name + "_pages", big)
            if e4m3:
                s = torch.empty((pages, hkv, 16), device=cuda_device)
                s[pages - small:] = getattr(p, name + "_scales")
                setattr(p, name + "_scales", s)
        p.page_table += pages - small
        got, st = attend(ts, p, ts.KERNEL_AUTO)
        assert torch.equal(got, want) and st & ~BAD_PAGE == 0
        q, k, v, qw, kw, f = append_inputs(cuda_device, p, 1, 128, True)
        ts.tree_chunk_append(q, k, v, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, q_norm=qw,
                             k_norm=kw, inv_freq=f, **p.scales())
        page, at = int(p.page_table[1, 1]), 15
        x = och.dequantise(p.v_pages[page:page + 1].view(torch.uint8).cpu().numpy(),
                           p.v_scales[page:page + 1].cpu().numpy())[0, at] if e4m3 else \
            p.v_pages[page, at].double().cpu().numpy()
        ref = v[9].double().cpu().numpy()
        assert (np.abs(x - ref) <= U_E4M3 * np.abs(ref).max()).all()
        del p, want, got
        torch.cuda.empty_cache()


def test_streams_graphs_and_shared_workspace(ts, cuda_device):
    """A captured append + attention replays on new values and lengths of the same sizes; two
    graphs share a workspace one after the other; a side stream gives the same bits."""
    p = make(cuda_device, [50, 700], [6, 3], 8, 2, 128, "bf16", True, seed=61)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 1, 128, True, fused=False)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)
    ws = torch.empty(ts.chunk_attn_workspace_bytes(prob), dtype=torch.uint8, device=cuda_device)
    q_out, out = torch.empty_like(q), torch.empty_like(q)

    def step():
        ts.tree_chunk_append(q, k, v, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, q_out,
                             q_norm=qw, k_norm=kw, inv_freq=f, workspace=ws, **p.scales())
        ts.tree_chunk_attn(q_out, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, out, workspace=ws,
                           **p.scales())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for turn, g in enumerate(graphs * 2):
        q.normal_()
        k.normal_()
        v.normal_()
        p.prefix_lens.copy_(ints([50 - 9 * turn, 700 - 100 * turn], cuda_device))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        with torch.cuda.stream(side):
            out.fill_(float("nan"))
        side.synchronize()
        res = ts.tree_chunk_attn(q_out, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, stream=side,
                                 **p.scales())
        side.synchronize()
        assert torch.equal(res, got)


# ------------------------------------------------------------------------------ trees over 8-bit pools

def tree_problem(device, sizes, N, prefix, hq, hkv, dim, dtype, seed=0):
    rng = np.random.default_rng([seed, 3])
    parents = trees.padded([trees.random_recursive(rng, n) for n in sizes], N)
    p = make(device, prefix, sizes, hq, hkv, dim, dtype, True, seed=seed)
    q = torch.from_numpy(rng.standard_normal((len(sizes), N, hq, dim)).astype(np.float32)).to(device).to(p.q.dtype)
    return p, q, parents


def tree_reference(p, q, parents):
    kp, vp = p.pools64()
    q64 = q.double().cpu().numpy()
    out, spread, reach = np.zeros(q64.shape), np.zeros(q64.shape), np.zeros(q64.shape[:3])
    table = p.page_table.cpu().numpy()
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        t = np.arange(S + n)
        pages = table[b][t // 16]
        K, V = kp[pages, t % 16], vp[pages, t % 16]
        for i in range(n):
            seen = t < S
            j = i
            while j >= 0:
                seen[S + j] = True
                j = parents[b, j]
            out[b, i], spread[b, i], reach[b, i] = och.attend(q64[b, i], K, V, seen)
    return out, spread, reach


TREES = [
    ([8], 8, [2000], 32, 8, 128),
    ([1], 1, [0], 4, 1, 64),
    ([64, 17, 1, 40], 64, [100, 37, 0, 300], 16, 2, 128),
    ([128, 65], 128, [10, 700], 8, 2, 64),
    ([20, 30, 16], 30, [63, 64, 65], 7, 1, 128),
    ([33] * 9, 33, [50 * i for i in range(9)], 12, 4, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"n{c[1]}-{c[3]}x{c[4]}-d{c[5]}")
def test_verify_e4m3(ts, cuda_device, case, dtype):
    sizes, N, prefix, hq, hkv, dim = case
    p, q, parents = tree_problem(cuda_device, sizes, N, prefix, hq, hkv, dim, dtype, seed=N)
    for kernel in (ts.KERNEL_AUTO, ts.KERNEL_SIMT):
        prob = ts.attn_problem(q, p.k_pages, p.page_table, kernel=kernel)
        ws = torch.full((ts.attn_e4m3_workspace_bytes(prob),), 0xff, dtype=torch.uint8, device=cuda_device)
        out = torch.full_like(q, float("nan"))
        got = ts.tree_attn_verify_e4m3(q, p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens,
                                       ints(parents, cuda_device), out, kernel=kernel, workspace=ws)
        assert ts.read_status(ws) == 0
        check_attention(got, *tree_reference(p, q, parents), max(a + b for a, b in zip(prefix, sizes)), dim, dtype,
                        dtype == "bf16")


def test_verify_e4m3_bad_input_sets_the_status(ts, cuda_device):
    p, q, parents = tree_problem(cuda_device, [12, 9], 12, [40, 40], 8, 2, 128, "bf16", seed=71)
    ws = torch.empty(ts.attn_e4m3_workspace_bytes(ts.attn_problem(q, p.k_pages, p.page_table)), dtype=torch.uint8,
                     device=cuda_device)

    def call(par):
        out = ts.tree_attn_verify_e4m3(q, p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens,
                                       ints(par, cuda_device), workspace=ws)
        return out, ts.read_status(ws)

    clean, st = call(parents)
    assert st == 0
    bad = parents.copy()
    bad[1, 3] = 7
    assert call(bad)[1] == 1                                   # BAD_PARENT
    p.prefix_lens[0] = -1
    out, st = call(parents)
    assert st == BAD_LENGTH and not out[0].any() and torch.equal(out[1], clean[1])
    p.prefix_lens[0] = 40
    p.page_table[1, 0] = -4
    out, st = call(parents)
    assert st == BAD_PAGE and torch.equal(out[0], clean[0])


def test_verify_e4m3_agrees_with_the_verification_of_the_same_values(ts, cuda_device):
    """Codes with scale 1 are bf16 values too: both verifications see the same numbers."""
    p, q, parents = tree_problem(cuda_device, [40, 64], 64, [500, 90], 16, 2, 128, "bf16", seed=73)
    p.k_scales.fill_(1.0)
    p.v_scales.fill_(1.0)
    p.k_pages.view(torch.uint8)[:] = torch.randint(0, 0x48, p.k_pages.shape, dtype=torch.uint8, device=cuda_device)
    p.v_pages.view(torch.uint8)[:] = torch.randint(0, 0x48, p.v_pages.shape, dtype=torch.uint8, device=cuda_device)
    q *= 0.1
    a = ts.tree_attn_verify_e4m3(q, p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens,
                                 ints(parents, cuda_device))
    b = ts.tree_attn_verify(q, p.k_pages.to(torch.bfloat16), p.v_pages.to(torch.bfloat16), p.page_table, p.prefix_lens,
                            ints(parents, cuda_device))
    # both round the weights and the result (2^-8 each) of positive values
    assert ((a.double() - b.double()).abs() <= 4.1 * U_BF16 * b.double().abs() + 1e-6).all()


@pytest.mark.parametrize("dim,hkv", [(128, 8), (64, 1)])
def test_commit_e4m3(ts, cuda_device, dim, hkv):
    N = 20
    prefix = [14, 0, 33, 5, 200]
    p = make(cuda_device, prefix, [N] * 5, hkv, hkv, dim, "bf16", True, seed=81)
    path = np.full((5, N), -1)
    for b, nodes in enumerate(([2, 5, 6, 19], [], list(range(1, 20)), [3, 2], [1])):
        path[b, :len(nodes)] = nodes
    length = np.array([4, 0, 19, 2, 1])
    table = p.page_table.cpu().numpy()
    codes = [t.view(torch.uint8).cpu().numpy() for t in (p.k_pages, p.v_pages)]
    scales = [np.nan_to_num(t.cpu().numpy()).transpose(0, 2, 1)[..., None] for t in (p.k_scales, p.v_scales)]
    ck, cv, lens, st = okc.kv_commit(codes[0], codes[1], table, np.array(prefix), path, length, num_nodes=N)
    sk, sv, _, _ = okc.kv_commit(scales[0], scales[1], table, np.array(prefix), path, length, num_nodes=N)
    ws = torch.empty(ts.commit_workspace_bytes(), dtype=torch.uint8, device=cuda_device)
    new = ts.tree_kv_commit_e4m3(p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens,
                                 ints(path, cuda_device), ints(length, cuda_device), workspace=ws)
    assert ts.read_status(ws) == st == 64                      # sequence 3's path does not increase
    assert new.cpu().numpy().tolist() == lens.tolist()
    assert np.array_equal(p.k_pages.view(torch.uint8).cpu().numpy(), ck)
    assert np.array_equal(p.v_pages.view(torch.uint8).cpu().numpy(), cv)
    assert np.array_equal(np.nan_to_num(p.k_scales.cpu().numpy()), sk[..., 0].transpose(0, 2, 1))
    assert np.array_equal(np.nan_to_num(p.v_scales.cpu().numpy()), sv[..., 0].transpose(0, 2, 1))


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_tree_accept_commit_and_decode(ts, cuda_device, e4m3):
    """As a serving loop runs them: append and attend the prompts in two chunks, append and verify
    a draft tree, walk it, commit the accepted path, append and attend one more token.  Each
    attention is checked against the definition over the cache as it then is, and the committed
    cache against one that only ever saw the accepted tokens."""
    hq, hkv, D, B, N = 8, 2, 128, 3, 12
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(5)
    lens = [70, 33, 5]
    pages_per = 8
    pool = B * pages_per + 1
    table = torch.randperm(pool, generator=gen, device=cuda_device)[:B * pages_per].view(B, -1).to(torch.int32)
    f = (10000.0 ** (-torch.arange(0, D, 2, device=cuda_device) / D)).float()
    w = 1 + 0.1 * torch.randn(D, generator=gen, device=cuda_device)

    def pools():
        if e4m3:
            return dict(k_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device).to(torch.float8_e4m3fn),
                        v_pages=torch.zeros((pool, 16, hkv, D), device=cuda_device).to(torch.float8_e4m3fn),
                        k_scales=torch.ones((pool, hkv, 16), device=cuda_device),
                        v_scales=torch.ones((pool, hkv, 16), device=cuda_device))
        z = torch.zeros((pool, 16, hkv, D), device=cuda_device, dtype=torch.bfloat16)
        return dict(k_pages=z.clone(), v_pages=z.clone())

    cache, plain = pools(), pools()

    def project(n):
        x = torch.randn((n, hq + 2 * hkv, D), generator=gen, device=cuda_device).to(torch.bfloat16)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    def append(c, qkv, prefix, offsets, positions=None):
        return ts.tree_chunk_append(*qkv, page_table=table, prefix_lens=prefix, chunk_offsets=offsets, positions=positions,
                                    q_norm=w, k_norm=w, inv_freq=f, **c)

    def check(c, q, prefix, offsets):
        from chunk_util import Problem
        s = (c.get("k_scales"), c.get("v_scales"))
        new = (offsets[1:] - offsets[:-1]).tolist()
        check_chunk(ts, Problem(prefix.tolist(), new, q, c["k_pages"], c["v_pages"], s[0], s[1], table, prefix, offsets),
                    ts.KERNEL_AUTO)

    prefix = ints([0] * B, cuda_device)
    for part in ([40, 20, 5], [30, 13, 0]):
        offsets = ints(np.concatenate(([0], np.cumsum(part))), cuda_device)
        qkv = project(sum(part))
        q = append(cache, qkv, prefix, offsets)
        append(plain, qkv, prefix, offsets)
        check(cache, q, prefix, offsets)
        prefix = prefix + ints(part, cuda_device)
    assert prefix.tolist() == lens
    rng = np.random.default_rng(9)
    parents = np.stack([trees.random_recursive(rng, N) for _ in range(B)])
    depth = np.zeros((B, N), dtype=np.int64)
    for b in range(B):
        for i in range(1, N):
            depth[b, i] = depth[b, parents[b, i]] + 1
    offsets = ints(np.arange(B + 1) * N, cuda_device)
    qkv = project(B * N)
    q = append(cache, qkv, prefix, offsets, ints((np.array(lens)[:, None] + depth).reshape(-1), cuda_device)).view(B, N, hq, D)
    if e4m3:
        out = ts.tree_attn_verify_e4m3(q, page_table=table, prefix_lens=prefix, tree_parents=ints(parents, cuda_device),
                                       **cache)
    else:
        out = ts.tree_attn_verify(q, cache["k_pages"], cache["v_pages"], table, prefix, ints(parents, cuda_device))
    from chunk_util import Problem
    p = Problem(lens, [N] * B, None, cache["k_pages"], cache["v_pages"], cache.get("k_scales"), cache.get("v_scales"), table,
                prefix, offsets)
    check_attention(out, *tree_reference(p, q, parents), max(lens) + N, D, "bf16", True)
    logits = torch.randn((B, N, 50), generator=gen, device=cuda_device)
    tokens = logits.argmax(-1)[torch.arange(B)[:, None], torch.from_numpy(np.maximum(parents, 0))].to(torch.int32)
    path, length, _bonus = ts.tree_accept(logits, tokens, None, ints(parents, cuda_device), None, 0.0)
    assert int(length.min()) >= 1
    if e4m3:
        new = ts.tree_kv_commit_e4m3(page_table=table, prefix_lens=prefix, accept_path=path, accept_len=length, **cache)
    else:
        new = ts.tree_kv_commit(cache["k_pages"], cache["v_pages"], table, prefix, path, length)
    # the same tokens appended in order by the plain route: their positions are the prefix and the depth
    order = [[0] + path[b, :int(length[b])].tolist() for b in range(B)]
    rows = torch.tensor([b * N + i for b in range(B) for i in order[b]], device=cuda_device)
    kept = ints(np.concatenate(([0], np.cumsum([len(o) for o in order]))), cuda_device)
    append(plain, tuple(t[rows] for t in qkv), prefix, kept)
    assert new.tolist() == [n + len(o) for n, o in zip(lens, order)]
    for b in range(B):
        t = torch.arange(int(new[b]), device=cuda_device)
        page, at = table[b].long()[t // 16], t % 16
        for name in cache:
            x, y = (c[name].transpose(1, 2) if "scales" in name else c[name] for c in (cache, plain))
            x, y = ((z.view(torch.uint8) if z.dtype == torch.float8_e4m3fn else z)[page, at] for z in (x, y))
            assert torch.equal(x, y), name
    offsets = ints(np.arange(B + 1), cuda_device)
    q = append(cache, project(B), new, offsets)
    check(cache, q, new, offsets)


# ------------------------------------------------------------------------------ uses that meet in one program

@pytest.mark.parametrize("e4m3", [False, True])
def test_two_calls_at_once_with_a_workspace_each(ts, cuda_device, e4m3):
    p = make(cuda_device, [3000, 10, 900], [1, 200, 64], 16, 2, 128, "bf16", e4m3, seed=91)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)
    want, _ = attend(ts, p, ts.KERNEL_AUTO)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(ts.chunk_attn_workspace_bytes(prob), dtype=torch.uint8, device=cuda_device) for _ in streams]
    outs = [[torch.empty_like(p.q) for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for st, ws, out in zip(streams, spaces, outs):
            ts.tree_chunk_attn(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, out[i], workspace=ws,
                               stream=st, **p.scales())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for out in outs for o in out)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
def test_sequences_that_share_the_pages_of_a_prefix(ts, cuda_device, dtype, e4m3):
    p = make(cuda_device, [64, 70, 64], [20, 5, 1], 8, 2, 128, dtype, e4m3, seed=93)
    p.page_table[1:, :4] = p.page_table[0, :4]                 # 64 tokens in four whole pages
    check_chunk(ts, p, ts.KERNEL_AUTO)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_and_negative_scales(ts, cuda_device, dtype):
    """Scales that a program made itself: any finite float32 multiplies its codes."""
    p = make(cuda_device, [150, 3], [70, 2], 8, 2, 128, dtype, True, seed=95)
    gen = torch.Generator(device=cuda_device)
    gen.manual_seed(1)
    for s in (p.k_scales, p.v_scales):
        s *= torch.randint(-1, 2, s.shape, generator=gen, device=cuda_device)
    check_chunk(ts, p, ts.KERNEL_AUTO)


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(ts, cuda_device, dtype, e4m3):
    p = make(cuda_device, [90], [40], 8, 2, 128, dtype, e4m3, seed=97)
    clean, _ = attend(ts, p, ts.KERNEL_AUTO)
    p.q[7, 3, 5], p.q[20, 6, 100] = float("nan"), float("inf")
    got, st = attend(ts, p, ts.KERNEL_AUTO)
    assert st == 0 and torch.isnan(got[7, 3]).all() and torch.isnan(got[20, 6]).all()
    keep = torch.ones(40, 8, dtype=torch.bool, device=cuda_device)
    keep[7, 3] = keep[20, 6] = False
    tol = (2 * U_BF16 if dtype == "bf16" else 1e-5) * clean.abs().amax().item()
    assert (got[keep].double() - clean[keep].double()).abs().max().item() <= tol


# ------------------------------------------------------------------------------ units of one and of two query tiles

MIXED = [
    # kind, prefix, new, rows of a sequence, hq, hkv, dim.  128 // (hq // hkv) tokens fill a query tile: every case has units
    # of one tile beside units of two, and more units than SMs, so that a CTA walks several of them
    ("tree", [1000 + 7 * b for b in range(32)], [40] * 32, 40, 64, 8, 128),
    ("tree", [1100 - 9 * b for b in range(32)], [20, 50] * 16, 50, 32, 8, 128),
    ("tree", [700 + 64 * (b % 5) for b in range(24)], [48, 3, 33, 17] * 6, 48, 64, 8, 64),
    ("chunk", [1500, 900, 2100, 1300], [488, 500, 484, 510], None, 64, 8, 128),
    ("chunk", [0] * 24, [35 + 11 * b for b in range(24)], None, 32, 8, 128),
    ("chunk", [900 + 130 * (b % 7) for b in range(48)], [10, 64] * 24, None, 32, 8, 128),
]


@pytest.mark.parametrize("case", MIXED, ids=lambda c: f"{c[0]}-{len(c[1])}x{max(c[2])}-{c[4]}x{c[5]}-d{c[6]}")
def test_8bit_units_of_one_and_two_query_tiles(ts, cuda_device, case):
    """The scales of V differ by up to two orders of magnitude from token to token, so a row that
    is weighed with another tile's scales is far off."""
    kind, prefix, new, width, hq, hkv, dim = case
    p = make_8bit(cuda_device, prefix, new, hq, hkv, dim, seed=len(new))
    table = (p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens)
    if kind == "tree":
        rng = np.random.default_rng(len(new))
        parents = trees.padded([trees.random_recursive(rng, n) for n in new], width)
        gen = torch.Generator(device=cuda_device)
        gen.manual_seed(7)
        q = torch.randn((len(new), width, hq, dim), generator=gen, device=cuda_device).to(torch.bfloat16)
        ws = torch.empty(ts.attn_e4m3_workspace_bytes(ts.attn_problem(q, p.k_pages, p.page_table, kernel=ts.KERNEL_TC_STREAM)),
                         dtype=torch.uint8, device=cuda_device)
        par = ints(parents, cuda_device)
        call = lambda: ts.tree_attn_verify_e4m3(q, *table, par, kernel=ts.KERNEL_TC_STREAM, workspace=ws)  # noqa: E731
        ref = tree64(p, q, parents)
    else:
        ws = torch.empty(ts.chunk_attn_workspace_bytes(ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)),
                         dtype=torch.uint8, device=cuda_device)
        call = lambda: ts.tree_chunk_attn(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets,  # noqa: E731
                                          kernel=ts.KERNEL_TC_STREAM, workspace=ws, **p.scales())
        ref = causal64(p)
    got = call()
    assert ts.read_status(ws) == 0
    check_attention(got, *ref, max(a + b for a, b in zip(prefix, new)), dim, "bf16", True)
    for _ in range(20):
        again = call()
        assert torch.equal(again.view(torch.int16), got.view(torch.int16)), "the same call gave other bits"
    assert ts.read_status(ws) == 0


# ------------------------------------------------------------------------------ hidden values that are not finite

def poison(p, tokens, columns):
    """A NaN in V of kv head h at new token tokens[b][h] of sequence b, in `columns` of the head (8-bit: the code)."""
    for b, of_head in enumerate(tokens):
        for h, i in enumerate(of_head):
            page, at = int(p.page_table[b, (p.prefix[b] + i) // 16]), (p.prefix[b] + i) % 16
            if p.k_scales is None:
                p.v_pages[page, at, h, columns] = float("nan")
            else:
                p.v_pages.view(torch.uint8)[page, at, h, columns] = 0x7f


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("prefix,new,hq,hkv,dim", [
    ([300, 40], [96, 64], 16, 2, 128),                         # few units: CTAs of their own, cut into pieces
    ([70] * 40, [34] * 40, 32, 4, 64),                         # more units than SMs
])
def test_all_rows_of_a_tile_beside_a_hidden_nan(ts, cuda_device, prefix, new, hq, hkv, dim, e4m3):
    """The last new token of every sequence holds a NaN: it shares a tile with every row, and all rows
    but its own are finite, stored whole and in pieces, in every call."""
    p = make(cuda_device, prefix, new, hq, hkv, dim, "bf16", e4m3, seed=101)
    poison(p, [[n - 1] * hkv for n in new], slice(3, 4))
    ref = causal64(p)
    assert np.isnan(ref[0]).sum() == len(new) * hq
    got, st = attend(ts, p, ts.KERNEL_TC_STREAM)
    assert st == 0
    check_attention(got, *ref, max(a + b for a, b in zip(prefix, new)), dim, "bf16", True)
    for _ in range(20):
        again, _ = attend(ts, p, ts.KERNEL_TC_STREAM)
        assert torch.equal(again.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("kind,e4m3", [("chunk", False), ("chunk", True), ("tree", True)])
def test_recomputed_rows_outlast_the_wait_limit(ts, cuda_device, kind, e4m3):
    """Rows that share a tile with a hidden NaN are recomputed for far longer than the limit of the
    waits, while the rest of the CTA waits for them: no wait runs out, and every row is right.  (The
    hand-offs of the fast path take microseconds, the limit is a millisecond.)"""
    prefix, new = ([1500, 900, 2100, 1300], [488, 500, 484, 510]) if kind == "chunk" else ([1500] * 24, [40] * 24)
    if e4m3:
        p = make_8bit(cuda_device, prefix, new, 64, 8, 128, seed=103, spread=0.3)
    else:
        p = make(cuda_device, prefix, new, 64, 8, 128, "bf16", seed=103)
    gen = np.random.default_rng(7)
    # the last token of a unit of 32 (a chunk), or the last leaf: every row before it in its unit is recomputed
    poison(p, [[31 + 32 * int(gen.integers(3)) for _ in range(8)] if kind == "chunk" else [39] * 8 for _ in new], slice(17, 18))
    ts.set_wait_limit_ns(1_000_000)
    try:
        if kind == "chunk":
            got, st = attend(ts, p, ts.KERNEL_TC_STREAM)
            ref = causal64(p)
        else:
            rng = np.random.default_rng(3)
            parents = np.stack([trees.random_recursive(rng, 40) for _ in new])
            q = p.q.view(len(new), 40, 64, 128)
            ws = torch.empty(ts.attn_e4m3_workspace_bytes(ts.attn_problem(q, p.k_pages, p.page_table)), dtype=torch.uint8,
                             device=cuda_device)
            got = ts.tree_attn_verify_e4m3(q, p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens,
                                           ints(parents, cuda_device), workspace=ws)
            st = ts.read_status(ws)
            ref = tree64(p, q, parents)
    finally:
        ts.set_wait_limit_ns(0)
    assert st == 0
    check_attention(got, *ref, max(a + b for a, b in zip(prefix, new)), 128, "bf16", True)


# ------------------------------------------------------------------------------ scores of minus infinity

MINUS_INF = [
    # prefix, new, tokens whose score is -inf for every row
    ([32], [1], [32]),                                         # alone in its slice of 32 tokens
    ([300], [20], list(range(32)) + list(range(128, 160))),    # whole slices, before and between finite ones
    ([0], [40], [0]),                                          # row 0 sees nothing else: NaN by definition
    ([70, 400], [50, 3], list(range(64))),                     # a whole tile
]


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("kernel,hidden", [("auto", False), ("auto", True), ("simt", False)])
@pytest.mark.parametrize("case", MINUS_INF, ids=["own", "slices", "first", "tile"])
def test_a_score_of_minus_infinity_weighs_nothing(ts, cuda_device, case, kernel, hidden, dtype, e4m3):
    """Such a token has weight 0, wherever it stands; `hidden`: beside a NaN that the rows do not see, which
    has the tensor-core form recompute them."""
    prefix, new, tokens = case
    if hidden and new[-1] == 1:
        pytest.skip("a row alone hides nothing")
    p = make(cuda_device, prefix, new, 8, 2, 128, dtype, e4m3, seed=sum(new))
    p.q[:] = p.q.abs() * 0.2 + 0.01                            # all products of the token are -inf or finite and positive
    where = [(int(p.page_table[b, t // 16]), t % 16) for b in range(len(prefix)) for t in tokens]
    if hidden:
        poison(p, [[n - 1] * 2 for n in new], slice(9, 10))
    finite = [x.copy() for x in p.pools64()]
    for page, at in where:
        finite[0][page, at] = 0
        if e4m3:
            p.k_pages.view(torch.uint8)[page, at] = 0x38
            p.k_scales[page, :, at] = -float("inf")
        else:
            p.k_pages[page, at, :, 5] = -float("inf")
    host = (p.page_table.cpu().numpy(), p.prefix_lens.cpu().numpy(), p.chunk_offsets.cpu().numpy())
    q64 = p.q.double().cpu().numpy()
    out, spread, _ = och.chunk_attention(q64, *p.pools64(), *host)
    reach = och.chunk_attention(q64, *finite, *host)[2]        # what errors of the finite scores scale with
    got, st = attend(ts, p, ts.KERNEL_AUTO if kernel == "auto" else ts.KERNEL_SIMT)
    assert st == 0
    check_attention(got, out, spread, reach, max(a + b for a, b in zip(prefix, new)), 128, dtype, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("splits", [1, 3])
def test_tree_verification_on_cuda_cores_with_scores_of_minus_infinity(ts, cuda_device, dtype, splits):
    sizes, N, prefix = [9, 12], 12, [400, 64]
    rng = np.random.default_rng(5)
    parents = trees.padded([trees.random_recursive(rng, n) for n in sizes], N)
    p = make(cuda_device, prefix, sizes, 8, 2, 128, dtype, seed=111)
    for t in (p.k_pages, p.v_pages):                           # tree_attn_verify reads a page's unused slots
        t.nan_to_num_()
    q = torch.rand((2, N, 8, 128), device=cuda_device).to(p.q.dtype)
    finite = p.k_pages.clone()
    for b in range(2):
        for t in list(range(32)) + list(range(300, 332)):
            if t < prefix[b]:
                page, at = int(p.page_table[b, t // 16]), t % 16
                p.k_pages[page, at, :, 5] = -float("inf")
                finite[page, at] = 0
    out, spread, _ = tree64(p, q, parents)
    got = ts.tree_attn_verify(q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, ints(parents, cuda_device),
                              kernel=ts.KERNEL_SIMT, num_splits=splits)
    p.k_pages = finite
    check_attention(got, out, spread, tree64(p, q, parents)[2], 412, 128, dtype, False)


def gpu_ms(call):
    """Milliseconds of a call on the device, the best of three after one that warms up."""
    call()
    best = float("inf")
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("what", ["v", "v_inf", "k", "both"])
def test_values_that_all_rows_see_do_not_have_them_recomputed(ts, cuda_device, what, e4m3):
    """One NaN (or infinity) near the start of a sequence reaches every later row by definition.  The rows
    are what the definition says, beside a NaN at a unit's end that the unit's other rows do not see, and
    the call does not take hundreds of times as long (a recomputed row costs some microseconds per 10
    tokens, and there are 65536 of them)."""
    prefix, new = [3000, 700], [512, 512]
    if e4m3:
        p = make_8bit(cuda_device, prefix, new, 64, 8, 128, seed=121, spread=0.3)
    else:
        p = make(cuda_device, prefix, new, 64, 8, 128, "bf16", seed=121)
    clean = gpu_ms(lambda: attend(ts, p, ts.KERNEL_TC_STREAM))
    page, at = int(p.page_table[0, 1]), 3                      # token 19 of sequence 0
    bad = float("inf") if what == "v_inf" else float("nan")
    if what != "k":
        if e4m3:
            p.v_scales[page, 2:6, at] = bad                    # kv heads 2 .. 5
        else:
            p.v_pages[page, at, 2:6, 77] = bad
    if what in ("k", "both"):
        if e4m3:
            p.k_pages.view(torch.uint8)[page, at, 4, 90] = 0xff
        else:
            p.k_pages[page, at, 4, 90] = bad
    spoiled = gpu_ms(lambda: attend(ts, p, ts.KERNEL_TC_STREAM))
    poison(p, [[63] * 8, [127] * 8], slice(100, 101))          # hidden from rows of their units
    got, st = attend(ts, p, ts.KERNEL_TC_STREAM)
    assert st == 0
    ref = causal64(p)
    g = got.double().cpu().numpy()
    # an infinity may come out as itself or as NaN (8-bit: codes of both signs); finite values have to be finite
    assert np.array_equal(np.isfinite(g), np.isfinite(ref[0]))
    got[~torch.isfinite(got)] = float("nan")
    check_attention(got, *ref, 3512, 128, "bf16", True)
    assert spoiled < 30 * clean + 1, (spoiled, clean)


# ------------------------------------------------------------------------------ the library's host side

def test_a_rejected_call_does_not_fail_the_next_one(ts, cuda_device):
    """A stream whose capture was made invalid (by waiting for it) refuses what is launched on it; the calls
    after that, on other streams, succeed."""
    import ctypes
    driver = ctypes.CDLL("libcuda.so.1")
    p = make(cuda_device, [20, 5], [4, 3], 8, 2, 128, "bf16", seed=131)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 1, 128, True)
    prob = ts.chunk_problem(p.q, p.k_pages, p.page_table, p.chunk_offsets)
    ws = torch.empty(ts.chunk_attn_workspace_bytes(prob), dtype=torch.uint8, device=cuda_device)
    q_out, out = torch.empty_like(p.q), torch.empty_like(p.q)
    path, length, lens = ints([[1, -1]] * 2, cuda_device), ints([1, 1], cuda_device), ints([0, 0], cuda_device)

    def calls(stream):
        yield lambda: ts.tree_chunk_append(q, k, v, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, q_out,
                                           q_norm=qw, k_norm=kw, inv_freq=f, workspace=ws, stream=stream)
        for kernel in (ts.KERNEL_AUTO, ts.KERNEL_SIMT):
            yield lambda: ts.tree_chunk_attn(p.q, p.k_pages, p.v_pages, p.page_table, p.prefix_lens, p.chunk_offsets, out,
                                             kernel=kernel, workspace=ws, stream=stream)
        yield lambda: ts.tree_kv_commit(p.k_pages, p.v_pages, p.page_table, p.prefix_lens, path, length, lens, workspace=ws,
                                        stream=stream)

    for c in calls(None):
        c()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    for n in range(4):
        assert driver.cuStreamBeginCapture_v2(handle, 1) == 0  # thread-local: nothing else is affected
        assert driver.cuStreamSynchronize(handle) != 0         # not allowed while capturing
        with pytest.raises(ts.TreespecError):
            list(calls(stream))[n]()
        graph = ctypes.c_void_p()
        assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0 and not graph.value
        for c in calls(None):
            c()
        assert ts.last_launch_error()[0] != 0                  # the rejected one's
    torch.cuda.synchronize()
    assert ts.read_status(ws) == 0


def test_an_argument_that_is_no_tensor_is_named(ts, cuda_device):
    import inspect
    p = make(cuda_device, [20, 5], [4, 4], 8, 2, 128, "bf16", True, seed=133)
    tree = ints([[-1, 0, 1, 1]] * 2, cuda_device)
    have = dict(q=p.q, k=p.q[:, :2], v=p.q[:, 2:4], k_pages=p.k_pages, v_pages=p.v_pages, k_scales=p.k_scales,
                v_scales=p.v_scales, page_table=p.page_table, prefix_lens=p.prefix_lens, chunk_offsets=p.chunk_offsets,
                tree_parents=tree, accept_path=tree, accept_len=ints([1, 1], cuda_device))
    extra = dict(positions=None, q_norm=None, k_norm=None, inv_freq=None, q_out=None, out=None, new_prefix_lens=None,
                 workspace=None)
    for fn in (ts.tree_chunk_append, ts.tree_chunk_attn, ts.tree_attn_verify_e4m3, ts.tree_kv_commit_e4m3):
        names = inspect.signature(fn).parameters
        args = {n: t for n, t in have.items() if n in names}
        if fn is ts.tree_attn_verify_e4m3:
            args["q"] = p.q.view(2, 4, 8, 128)
        for name in [n for n in (*have, *extra) if n in names]:
            with pytest.raises(ValueError, match=name.replace("_scales", "_scales|scales")):
                fn(**{**args, name: 3.5})
            if name in have:
                with pytest.raises(ValueError, match=name):
                    fn(**{**args, name: None})


@pytest.mark.parametrize("layout", [0, 1])
def test_append_angles_at_the_stated_limit_of_the_frequencies(ts, cuda_device, layout):
    """Frequencies up to the last float32 below 2^24 at positions up to 2^31 - 1."""
    p = make(cuda_device, [0], [6], 2, 1, 64, "f32", seed=2)
    q, k, v, qw, kw, _ = append_inputs(cuda_device, p, 4, 64, False)
    f = torch.tensor([2.0 ** 24 - 1, 1024.5, 65537.25, 1048577.0, 12345678.0, 333333.34, 4095.9998, 7.0] * 4,
                     device=cuda_device)
    pos = ints([0, 1, 65537, 123456789, (1 << 30) + 7, (1 << 31) - 1], cuda_device)
    assert check_append(ts, p, q, k, v, qw, kw, f, pos, layout) == 0
    assert check_append(ts, p, q, k, v, qw, kw, -f, pos, layout) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_waits_that_run_out_anywhere_leave_the_next_call_right(ts, cuda_device, e4m3):
    """Limits from below the first hand-off to about a call's whole time: the call ends with TIMEOUT or is
    right, and so is one without a limit after it."""
    p = make_8bit(cuda_device, [1500, 300, 0, 900], [200, 3, 129, 64], 32, 4, 128, seed=141)
    if not e4m3:
        p.k_pages, p.v_pages = ((x.float() * 0.01).to(torch.bfloat16) for x in (p.k_pages, p.v_pages))
        p.k_scales = p.v_scales = None
    want, st = attend(ts, p, ts.KERNEL_TC_STREAM)
    assert st == 0
    for limit in (1, 500, 1000, 1500, 2000, 3000, 5000, 8000, 15000, 25000, 60000):
        ts.set_wait_limit_ns(limit)
        try:
            got, st = attend(ts, p, ts.KERNEL_TC_STREAM)
        finally:
            ts.set_wait_limit_ns(0)
        assert st in (0, 16)
        if st == 0:
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        got, st = attend(ts, p, ts.KERNEL_TC_STREAM)
        assert st == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("tokens,hq,hkv,dim,dtype,e4m3", [
    (1217, 28, 4, 64, "bf16", True),                           # 8 tokens per SM and a last CTA with one token
    (1400, 60, 2, 128, "f32", False),
    (4863, 5, 5, 128, "bf16", False),                          # just below 32 tokens per SM, just above
    (4867, 3, 1, 64, "bf16", True),
])
def test_append_at_the_borders_of_the_launch_shapes(ts, cuda_device, tokens, hq, hkv, dim, dtype, e4m3):
    a = tokens // 3
    p = make(cuda_device, [5, 0, 40], [a, 7, tokens - a - 7], hq, hkv, dim, dtype, e4m3, seed=tokens, lead=1)
    q, k, v, qw, kw, f = append_inputs(cuda_device, p, 3, 48, True)
    assert check_append(ts, p, q, k, v, qw, kw, f, None, tokens % 2) == 0


@pytest.mark.parametrize("dtype,e4m3", KINDS, ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("kernel", ["auto", "simt"])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("prefix,new", [([3000], [1]), ([1500], [70]), ([900, 40], [5, 1]), ([1000] * 40, [1] * 40),
                                        ([100], [1])])
def test_a_nan_among_tokens_of_no_weight_is_not_lost(ts, cuda_device, prefix, new, where, kernel, dtype, e4m3):
    """The scores of the first 700 tokens lie hundreds below the others, so that whole pieces, splits and slices
    weigh 0 in 32 bits; a NaN that a row sees among them makes the row (K) or its column (V) NaN all the same."""
    p = make(cuda_device, prefix, new, 8, 1, 128, dtype, e4m3, seed=151)
    p.q[:] = p.q.abs() + 0.1
    for b, S in enumerate(prefix):
        t = torch.arange(min(700, S), device=cuda_device)
        page, at = p.page_table[b].long()[t // 16], t % 16
        if e4m3:
            p.k_pages.view(torch.uint8)[page, at] = 0xe0       # -32
            p.k_scales[page, :, at] = 1.0
        else:
            p.k_pages[page, at] = -32.0
    page, at = int(p.page_table[0, 0]), 10
    if e4m3:
        (p.k_pages if where == "k" else p.v_pages).view(torch.uint8)[page, at, 0, 77] = 0x7f
    else:
        (p.k_pages if where == "k" else p.v_pages)[page, at, 0, 77] = float("nan")
    ref = causal64(p)
    assert np.isnan(ref[0]).any()
    got, st = attend(ts, p, ts.KERNEL_AUTO if kernel == "auto" else ts.KERNEL_SIMT)
    assert st == 0
    check_attention(got, *ref, max(a + b for a, b in zip(prefix, new)), 128, dtype, dtype == "bf16")


def test_captured_tree_step_over_8bit_pools(ts, cuda_device):
    """Append, verification and commit of a batch of trees in one graph, replayed over other trees, lengths, values
    and paths of the same sizes; between replays the same step runs eagerly with a workspace of its own."""
    rng = np.random.default_rng(161)
    B, N, hq, hkv, D = 5, 20, 16, 2, 128
    p = make_8bit(cuda_device, [900, 30, 0, 400, 77], [N] * B, hq, hkv, D, seed=161)
    for t in (p.k_pages, p.v_pages):
        t.view(torch.uint8)[t.view(torch.uint8) == 0x7f] = 0
    for t in (p.k_scales, p.v_scales):
        t.nan_to_num_(0.01)
    qkv = torch.randn((B * N, hq + 2 * hkv, D), device=cuda_device).to(torch.bfloat16)
    f = (10000.0 ** (-torch.arange(0, D, 2, device=cuda_device) / D)).float()
    offsets = ints(np.arange(B + 1) * N, cuda_device)
    parents, pos = ints(np.zeros((B, N)), cuda_device), ints(np.zeros(B * N), cuda_device)
    path, length, lens = ints(np.zeros((B, N)), cuda_device), ints(np.zeros(B), cuda_device), ints(np.zeros(B), cuda_device)
    q = torch.empty((B * N, hq, D), dtype=torch.bfloat16, device=cuda_device)
    out = torch.empty((B, N, hq, D), dtype=torch.bfloat16, device=cuda_device)
    size = ts.attn_e4m3_workspace_bytes(ts.attn_problem(out, p.k_pages, p.page_table))
    spaces = [torch.empty(size, dtype=torch.uint8, device=cuda_device) for _ in range(2)]

    def step(ws):
        ts.tree_chunk_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], p.k_pages, p.v_pages, p.page_table,
                             p.prefix_lens, offsets, q, positions=pos, inv_freq=f, workspace=ws, **p.scales())
        ts.tree_attn_verify_e4m3(q.view(B, N, hq, D), p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table,
                                 p.prefix_lens, parents, out, workspace=ws)
        ts.tree_kv_commit_e4m3(p.k_pages, p.v_pages, p.k_scales, p.v_scales, p.page_table, p.prefix_lens, path, length, lens,
                               workspace=ws)

    def fill():
        sizes = [int(n) for n in rng.integers(1, N + 1, B)]
        tree = trees.padded([trees.random_recursive(rng, n) for n in sizes], N)
        depth, way, steps = np.full((B, N), -1), np.full((B, N), -1), []
        prefix = [int(rng.integers(0, m + 1)) for m in (900, 30, 0, 400, 77)]
        for b, n in enumerate(sizes):
            for i in range(n):
                depth[b, i] = prefix[b] if i == 0 else depth[b, tree[b, i]] + 1
            chain, node = [], int(rng.integers(n))
            while node > 0:
                chain.append(node)
                node = int(tree[b, node])
            way[b, :len(chain)] = chain[::-1]
            steps.append(len(chain))
        for t, a in ((parents, tree), (pos, depth.reshape(-1)), (path, way), (length, steps), (p.prefix_lens, prefix)):
            t.copy_(ints(a, cuda_device))
        qkv.normal_()

    state = lambda: [t.clone() for t in (p.k_pages.view(torch.uint8), p.v_pages.view(torch.uint8), p.k_scales, p.v_scales)]  # noqa: E731
    fill()
    step(spaces[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(spaces[0])
    for _ in range(4):
        fill()
        before = state()
        g.replay()
        torch.cuda.synchronize()
        assert ts.read_status(spaces[0]) == 0
        by_graph = [out.clone(), lens.clone(), *state()]
        for t, old in zip((p.k_pages.view(torch.uint8), p.v_pages.view(torch.uint8), p.k_scales, p.v_scales), before):
            t.copy_(old)
        out.fill_(float("nan"))
        step(spaces[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([out, lens, *state()], by_graph))
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kernel", ["tc", "simt"])
def test_offsets_that_give_rows_to_two_sequences(ts, cuda_device, kernel, e4m3):
    """0, 64, 0, 64, ...: every second sequence owns all rows.  The call is flagged and touches nothing but the rows;
    the tensor-core form, whose sums over the sequences could not hold such counts, computes none."""
    p = make(cuda_device, [40] * 300, [1] * 300, 8, 2, 128, "bf16", e4m3, seed=171, extra_pages=5)
    p.q = torch.randn((64, 8, 128), device=cuda_device).to(torch.bfloat16)
    p.chunk_offsets[0::2] = 0
    p.chunk_offsets[1::2] = 64
    room = torch.full((64 + 32, 8, 128), 3.0, dtype=torch.bfloat16, device=cuda_device)
    k = ts.KERNEL_TC_STREAM if kernel == "tc" else ts.KERNEL_SIMT
    _, st = attend(ts, p, k, out=room[16:80])
    assert st & BAD_LENGTH
    assert (room[:16] == 3.0).all() and (room[80:] == 3.0).all()
    if kernel == "tc":
        assert (room == 3.0).all()
