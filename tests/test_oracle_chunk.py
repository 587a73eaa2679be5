"""Pins of oracle.chunk: appending, 8-bit storage and causal attention of chunks (CPU only)."""
import inspect
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import chunk as och


def test_e4m3_codes_by_hand():
    v = och.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448.0
    assert math.isnan(v[0x7f]) and math.isnan(v[0xff]) and v[0xb8] == -1.0
    # ties go to the even code: 1.0625 lies between 1.0 (0x38) and 1.125 (0x39), 1.1875 between 0x39 and 0x3a
    assert och.to_e4m3([1.0625, 1.1875, -1.0625, 448.0, 0.0]).tolist() == [0x38, 0x3a, 0xb8, 0x7e, 0]


def test_e4m3_agrees_with_torch():
    import torch
    x = torch.linspace(-448, 448, 20011, dtype=torch.float64)
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(och.to_e4m3(x.float().double().numpy()), want)


def test_quantise_error_is_half_a_step_and_zero_rows_keep_a_scale():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 64)) * 10.0 ** rng.uniform(-3, 3, (50, 1))
    x[7] = 0
    codes, scale = och.quantise(x)
    back = och.e4m3_values()[codes] * scale[:, None]
    assert scale[7] == och.SCALE_MIN and not codes[7].any()
    # half a step of a normal value is 2^-4 of it; below 2^-6 (in units of the scale) it is 2^-10
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale[:, None]) * (1 + 1e-12)).all()


def test_angle_matches_plain_arithmetic_and_keeps_far_positions():
    for pos in (0, 1, 7, 4096):
        for f in (1.0, 0.25, np.float32(0.123456)):
            assert abs(math.remainder(och.angle(pos, f) - pos * float(f), 2 * math.pi)) < 1e-11
    # 113 x 2^20 positions at frequency 2: the product is exact in float64, and 3.8e7 turns of a
    # 2 pi that is off by 2^-52 give at most 1e-8
    pos, f = 113 * 2 ** 20, 2.0
    want = math.remainder(pos * f, 2 * math.pi)
    assert abs(math.remainder(och.angle(pos, f) - want, 2 * math.pi)) < 2e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_a_quarter_turn(interleaved):
    x = np.arange(1.0, 9.0)[None]                                      # one head, 8 elements
    f = [math.pi / 2]                                                  # one pair turns: rot_dim 2
    y = och.rotate(x, 1, f, interleaved)
    assert np.allclose(y[0, :2], [-2.0, 1.0]) and np.array_equal(y[0, 2:], x[0, 2:])
    y = och.rotate(x, 1, [math.pi / 2, 0.0], interleaved)
    want = [-2, 1, 3, 4] if interleaved else [-3, 2, 1, 4]
    assert np.allclose(y[0, :4], want) and np.array_equal(y[0, 4:], x[0, 4:])


def test_rotated_scores_depend_on_distance_only():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((2, 1, 16))
    f = 10.0 ** -np.arange(8)
    a = och.rotate(q, 1003, f, False)[0] @ och.rotate(k, 1000, f, False)[0]
    b = och.rotate(q, 3, f, False)[0] @ och.rotate(k, 0, f, False)[0]
    assert abs(a - b) < 1e-9


def test_append_places_rows_and_leaves_padding_out():
    q = k = v = np.ones((7, 1, 16))
    table = np.array([[4, 2], [9, 1]], dtype=np.int32)
    rows, slots = och.append(q, k, v, table, [15, 0], [1, 4, 6], 5, positions=[0, 15, -1, 17, 0, 1, 0])
    # rows 1..3 are sequence 0 at positions 15..17: page 4 slot 15, (padding), page 2 slot 1; sequence 1's page 9 is
    # outside the pool of 5; rows 0 and 6 belong to none
    assert sorted(rows) == [1, 3] and sorted(slots) == [(2, 1), (4, 15)]


def test_chunk_attention_is_the_tree_attention_of_a_chain():
    rng = np.random.default_rng(5)
    kp, vp = rng.standard_normal((2, 6, 16, 2, 8))
    table = np.array([[3, 1], [0, 5]], dtype=np.int32)
    q = rng.standard_normal((8, 4, 8))
    out, spread, reach = och.chunk_attention(q, kp, vp, table, [13, 2], [0, 3, 8])
    for b, (o0, o1, S) in enumerate(((0, 3, 13), (3, 8, 2))):
        n = o1 - o0
        ref = oatt.tree_attention(q[None, o0:o1], kp, vp, table[b:b + 1], np.array([S]),
                                  np.arange(-1, n - 1, dtype=np.int32)[None], 16)
        assert np.allclose(out[o0:o1], ref[0], atol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all() and (reach > 0).all()


def test_first_token_of_a_prompt_returns_its_own_value():
    rng = np.random.default_rng(6)
    kp, vp = rng.standard_normal((2, 1, 16, 1, 4))
    out, _, _ = och.chunk_attention(rng.standard_normal((2, 2, 4)), kp, vp, np.array([[0]]), [0], [0, 2])
    assert np.allclose(out[0], vp[0, 0, 0])


def test_a_planted_off_by_one_in_the_mask_is_seen():
    rng = np.random.default_rng(5)
    kp, vp = rng.standard_normal((2, 6, 16, 2, 8))
    args = (rng.standard_normal((3, 4, 8)), kp, vp, np.array([[3, 1]]), [13], [0, 3])
    ns = dict(vars(och))
    exec(inspect.getsource(och.chunk_attention).replace("t <= S + i", "t < S + i"), ns)
    assert not np.allclose(ns["chunk_attention"](*args)[0], och.chunk_attention(*args)[0])


def test_empty_and_invalid_sequences():
    rng = np.random.default_rng(8)
    kp, vp = rng.standard_normal((2, 3, 16, 1, 4))
    q = rng.standard_normal((5, 1, 4))
    out, _, _ = och.chunk_attention(q, kp, vp, np.array([[0], [1], [2]]), [3, -1, 16], [0, 2, 3, 4])
    assert np.isfinite(out[:2]).all() and not out[2:4].any() and np.isnan(out[4]).all()


def test_the_batched_reference_of_larger_problems_is_the_definition():
    """chunk_util.causal64 and tree64, which serve larger GPU cases, against the row-by-row oracle."""
    import torch
    from chunk_util import causal64, make, make_8bit, tree64
    for p in (make("cpu", [20, 3], [5, 18], 4, 2, 16, "f32", True, seed=2), make_8bit("cpu", [9, 0], [3, 7], 4, 1, 8, seed=4)):
        args = (p.q.double().numpy(), *p.pools64(), p.page_table.numpy(), p.prefix, p.chunk_offsets.tolist())
        for got, ref in zip(causal64(p), och.chunk_attention(*args)):
            assert np.allclose(got, ref, rtol=1e-12, atol=1e-12)
    parents = np.array([[-1, 0, 0, 2, -2], [-1, 0, 1, 1, 0]])
    p = make_8bit("cpu", [13, 2], [4, 5], 2, 1, 8, seed=5)
    q = torch.randn(2, 5, 2, 8, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out, _, _ = tree64(p, q, parents)
    kp, vp = p.pools64()
    for b in range(2):
        n = p.new[b]
        ref = oatt.tree_attention(q[b:b + 1, :n].double().numpy(), kp, vp, p.page_table[b:b + 1].numpy(),
                                  np.array(p.prefix[b:b + 1]), parents[b:b + 1, :n].astype(np.int32), 16)
        assert np.allclose(out[b, :n], ref[0], atol=1e-12) and not out[b, n:].any()
