"""Pins of the ragged-chunk definitions (oracle/chunk.py): hand-worked plans,
rotations against the block oracle's RoPE and by their invariants, attention
against the block oracle on uniform blocks.  CPU only."""
import numpy as np
import pytest

import oracle
from oracle import chunk


def test_plan_by_hand():
    # P = 4: request 0 has 5 keys on pages 9, 8 and brings 4 (keys 5..8: needs a
    # third page); request 1 is not live; request 2 is new and brings 5 (2 pages)
    table = np.array([[9, 8, -1, -1], [7, -1, -1, -1], [-1, -1, -1, -1]], np.int32)
    o = chunk.chunk_plan([4, 3, 5], [5, 2, 0], [2, 1, 0], table, [0, 1, 2, 3, 4], [1, 5],
                         [1, 0, 1], 1 << 30, n_rows=11, P=4, NP=10)
    assert o["flags"] == 0
    assert o["cu_rows"].tolist() == [0, 4, 4, 9]
    assert o["n_pages"].tolist() == [3, 0, 2]
    assert o["block_table"].tolist() == [[9, 8, 1, -1], [7, -1, -1, -1], [2, 3, -1, -1]]
    assert o["alloc_limit"].tolist() == [12, 0, 8] and o["seq_lens"].tolist() == [9, 0, 5]
    assert o["free_head"].tolist() == [4]
    assert o["row_req"].tolist() == [0, 0, 0, 0, 2, 2, 2, 2, 2, -1, -1]
    assert o["row_pos"].tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, -1, -1]
    assert o["row_page"].tolist() == [8, 8, 8, 1, 2, 2, 2, 2, 3, -1, -1]
    assert o["row_slot"].tolist() == [1, 2, 3, 0, 0, 1, 2, 3, 0, -1, -1]


def test_plan_runs_out():
    # one free page for two requests that need one each: the first gets it
    table = np.full((2, 2), -1, np.int32)
    o = chunk.chunk_plan([2, 2], [0, 0], [0, 0], table, [5], [0, 1], None, 1 << 30, n_rows=3, P=4,
                         NP=6)
    assert o["flags"] == 128 | 256  # 4 rows asked of 3; no page for request 1
    assert o["cu_rows"].tolist() == [0, 2, 3]
    assert o["row_page"].tolist() == [5, 5, -1] and o["row_pos"].tolist() == [0, 1, 0]
    assert o["seq_lens"].tolist() == [2, 0]


@pytest.mark.parametrize("hd", [64, 128])
def test_half_layout_is_the_block_rope(hd):
    rng = np.random.default_rng(3)
    x = oracle.f64_to_bf16(rng.standard_normal((1, 4, 2, hd)))
    gamma = oracle.f64_to_bf16(1 + 0.1 * rng.standard_normal(hd))
    pos = np.array([[0, 1, 4096, 393215]], np.int32)
    want = oracle.q_norm_rope(x, gamma, pos, 1e6, 1e-6)
    f64 = lambda b: (np.asarray(b).astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
    ang, mag = chunk.rope_angles(hd, 1e6)
    y, _ = chunk.turn(f64(x)[0], f64(gamma), pos[0], 1e-6, layout="half", rot=hd, angles=ang,
                      mag=mag)
    assert np.array_equal(oracle.f64_to_bf16(y)[None], want)


def test_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(4)
    rot, hd = 24, 64
    x = rng.standard_normal((5, 3, hd))
    perm = np.arange(hd)
    perm[0:rot:2], perm[1:rot:2] = np.arange(rot // 2), np.arange(rot // 2) + rot // 2
    ang, mag = chunk.rope_angles(rot, 1e4, "yarn", 4.0, 512)
    pos = np.array([0, 1, 7, 300, 5000])
    half, _ = chunk.turn(x, None, pos, 0.0, layout="half", rot=rot, angles=ang, mag=mag)
    pairs, _ = chunk.turn(x[..., perm], None, pos, 0.0, layout="pairs", rot=rot, angles=ang,
                          mag=mag)
    np.testing.assert_allclose(pairs, half[..., perm], atol=1e-13)
    np.testing.assert_array_equal(half[..., rot:], x[..., rot:])


def test_yarn_ends():
    # the fastest pairs keep their angle, the slowest are divided by the factor
    plain, _ = chunk.rope_angles(128, 1e6)
    ang, mag = chunk.rope_angles(128, 1e6, "yarn", 8.0, 8192)
    assert ang[0] == plain[0] and np.isclose(ang[-1], plain[-1] / 8.0, rtol=1e-14)
    assert np.all(ang <= plain) and np.all(ang >= plain / 8.0 * (1 - 1e-14))
    assert np.isclose(mag, 1 + 0.1 * np.log(8.0))


@pytest.mark.parametrize("window,sinks,causal", [(0, False, True), (7, True, True), (0, True, False)])
def test_attention_on_uniform_blocks_is_the_block_oracle(window, sinks, causal):
    from context_kv_update_gb300 import inputs
    prob = inputs.make_problem(inputs.workload("tiny", B=2, ctx=[21, 40], n_acc=[1, 1],
                                               alloc_pages=[3, 4]), seed=5, with_weights=False)
    g = prob["g"]
    T = g["T"]
    kv = np.array([21 + T, 40 + T], np.int32)
    sk = prob["sinks"][0] if sinks else None
    want = oracle.attention_gqa(g, 0, prob["q"][0], prob["pool"], prob["pages"], kv, window=window,
                                sinks=sk, mask_mode=0 if causal else 1)
    f64 = lambda b: (np.asarray(b).astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
    q = f64(prob["q"][0]).reshape(2 * T, g["hq"], g["hd"])
    got, size = chunk.chunk_attention(q, f64(prob["pool"])[0], prob["pages"], [0, T, 2 * T],
                                      [21, 40], kv, scale=1 / np.sqrt(g["hd"]), window=window,
                                      sinks=sk, causal=causal)
    np.testing.assert_allclose(got.reshape(want.shape), want, atol=1e-9)
    assert np.all(np.abs(got) <= size + 1e-12)
