"""Pins of the oracles for a step's index arrays and for the norm and rotation (no GPU)."""
import math

import numpy as np
import pytest

import oracle


def test_plan_by_hand():
    # pages of 4: a sequence of 3 that gets 3 more (its page, then a new one), an idle one, a new one of 5
    got = oracle.plan_step([3, 0, 5], [3, 9, 0], [[7, -1, -1], [1, 2, 3], [-1, -1, -1]], [10, 11, 12, 13], 4, 4, 10, 20,
                           refcount=np.zeros(20))
    assert got["block_table"].tolist() == [[7, 13, -1], [1, 2, 3], [12, 11, -1]]
    assert got["slot_mapping"].tolist() == [31, 52, 53, 48, 49, 50, 51, 44, -1, -1]
    assert got["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 0, 0]
    assert got["cu_q_lens"].tolist() == [0, 3, 3, 8] and got["seq_lens"].tolist() == [6, 9, 5]
    assert got["free_count"] == 1 and got["status"] == 0 and got["held_blocks"].tolist() == [2, 3, 2]
    assert np.flatnonzero(got["refcount"]).tolist() == [11, 12, 13]


def test_plan_pages_already_named_are_kept():
    # a prompt whose full pages a prefix lookup dealt out: 8 of its 11 tokens are cached
    got = oracle.plan_step([3], [8], [[5, 6, 9]], [1], 1, 4, 3, 10, held=[3])
    assert got["slot_mapping"].tolist() == [36, 37, 38] and got["free_count"] == 1


def test_plan_flags():
    run = oracle.plan_step
    assert run([-2], [4], [[0, 1]], [], 0, 4, 2, 4)["status"] == 8
    out = run([3], [3], [[0, 9]], [], 0, 4, 4, 4)
    assert out["status"] == 32 and out["slot_mapping"].tolist() == [3, -1, -1, -1] and out["block_table"][0, 1] == -1
    out = run([3], [3], [[0]], [2], 1, 4, 4, 4)
    assert out["status"] == 2 and out["seq_lens"].tolist() == [6]
    out = run([3, 3], [0, 0], [[-1], [-1]], [2, 3], 2, 4, 4, 4)
    assert out["status"] == 64 and out["cu_q_lens"].tolist() == [0, 3, 4] and out["seq_lens"].tolist() == [3, 1]
    assert run([1], [0], [[-1]], [77], 1, 4, 1, 4)["status"] == 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 8))
    angle = rng.uniform(-3, 3, (5, 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    out, _ = oracle.norm_rope(x, None, table, [4, 0, 2], 0.0, interleaved)
    a, b = ([0, 2], [1, 3]) if interleaved else ([0, 1], [2, 3])
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle[[4, 0, 2]])[:, None]
    assert np.allclose(out[..., a], z.real, atol=1e-14) and np.allclose(out[..., b], z.imag, atol=1e-14)
    assert (out[..., 4:] == x[..., 4:]).all()


def test_scores_depend_on_distance_only():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    turn = np.arange(50)[:, None] * 10000.0 ** (-2 * np.arange(8) / 16)
    table = np.concatenate([np.cos(turn), np.sin(turn)], 1)
    at = lambda x, p: oracle.norm_rope(x, None, table, [p], 0.0, False)[0].ravel()
    assert math.isclose(at(q, 7) @ at(k, 3), at(q, 44) @ at(k, 40), rel_tol=1e-12)


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((4, 3, 64)) * 50
    out, _ = oracle.norm_rope(x, np.full(64, 2.0), None, None, 0.0, False)
    assert np.allclose((out ** 2).mean(2), 4.0, rtol=1e-12)
    assert np.allclose(oracle.norm_rope(x * 0, np.ones(64), None, None, 1e-6, False)[0], 0.0)
