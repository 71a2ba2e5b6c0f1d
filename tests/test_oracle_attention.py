"""Pins of the attention and sampling oracles (CPU): closed forms, torch compositions, brute force."""
import numpy as np
import pytest
import torch

from oracle import attention, sampling


def test_tables_worked_example():
    # page 4; request 0 has 5 cached + 4 new (pages 7, 2 -> one more), request 1 rests, request 2 starts with 3
    table, start, seq, pos, slot, head = attention.tables(
        [5, 8, 0], [4, 0, 3], [[7, 2, -1], [1, 3, -1], [-1, -1, -1]], [9, 8, 6, 5], 1, 4, 9)
    assert table.tolist() == [[7, 2, 8], [1, 3, -1], [6, -1, -1]]
    assert start.tolist() == [0, 4, 4, 7] and seq.tolist() == [9, 8, 3] and head == 3
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 0, 0]
    assert slot.tolist() == [9, 10, 11, 32, 24, 25, 26, -1, -1]


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(pairs):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    f = 100.0 ** (-np.arange(16) / 16)

    def at(x, p):
        return attention.norm_rotate(x, None, 0.0, np.cos(p * f), np.sin(p * f), pairs)
    assert np.allclose(np.linalg.norm(at(q, 9)), np.linalg.norm(q))
    assert np.allclose(at(q, 9) @ at(k, 4), at(q, 25) @ at(k, 20))       # only the distance counts
    assert np.allclose(at(q, 0), q) and np.allclose(at(q, 9)[32:], q[32:])


def test_norm_has_unit_mean_square_times_weight():
    x = np.arange(1.0, 65.0)
    y = attention.norm_rotate(x, np.full(64, 3.0), 0.0, np.zeros(0), np.zeros(0), False)
    assert np.allclose(np.mean(y * y), 9.0)


def test_attend_matches_torch_and_masks():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal(64), rng.standard_normal((20, 64)), rng.standard_normal((20, 64))
    out, _ = attention.attend(q, k, v, 19, 0.125, 0)
    ref = torch.softmax(torch.tensor(k @ q * 0.125), 0) @ torch.tensor(v)
    assert np.allclose(out, ref.numpy())
    assert np.allclose(attention.attend(q, k, v, 7, 0.125, 1)[0], v[7])
    assert np.allclose(attention.attend(q, k, v, 0, 0.125, 0)[0], v[0])
    assert not attention.attend(q, k, v, -1, 0.125, 0)[0].any()


def test_keep_set_cases():
    x = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))
    def kept(*a):
        return sampling.keep_set(x, 1.0, *a)[0].tolist()
    assert kept(0, 1.0, 0.0) == [0, 1, 2, 3, 4]
    assert kept(2, 1.0, 0.0) == [1, 3]
    assert kept(3, 1.0, 0.0) == [0, 1, 3]                 # ties go to the lowest index
    assert kept(0, 0.65, 0.0) == [1, 3]
    assert kept(0, 0.75, 0.0) == [0, 1, 3]
    assert kept(0, 0.0, 0.0) == [1]                       # the first always
    assert kept(2, 0.5, 0.0) == [1]                       # of the top-k's mass 0.7: 0.4 >= 0.35
    assert kept(0, 1.0, 0.5) == [1, 3]


def test_sample_frequencies_follow_the_weights():
    x = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))
    ids = [sampling.sample(x, 1.0, 0, 1.0, 0.0, (i + 0.5) / 1000)[0] for i in range(1000)]
    assert np.bincount(ids).tolist() == [100, 400, 100, 300, 100]
    assert sampling.sample(x, 0.0, 0, 1.0, 0.0, 0.9)[0] == 1
    assert sampling.sample(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0, 0.9)[0] == -1
    assert sampling.sample(np.array([np.nan, 1.0, -np.inf]), 1.0, 0, 1.0, 0.0, 0.9)[:2] == (1, 0.0)
