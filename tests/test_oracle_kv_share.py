"""Pins of the restatement of the operators on shared pages: hand-worked values and invariants."""
import numpy as np
import pytest

from oracle import kv_oracle as KO
from oracle import kv_share_oracle as SO


def test_fork_hand_worked():
    # pages of 4 tokens.  Request 0 has 10 tokens in pages 5, 3, 0; ring: 7, 2, 6 from counter 9 on (9 mod 8 = 1)
    table = np.array([[5, 3, 0, -1], [-1] * 4, [-1] * 4, [-1] * 4, [1, -1, -1, -1]], np.int32)
    holders = np.array([1, 1, 0, 1, 0, 1, 0, 0], np.int32)
    ring = np.array([9, 7, 2, 6, 9, 9, 9, 9], np.int32)
    got = SO.fork([10, 0, 0, 0, 3], [-1, 0, 0, 0, 0], [0, 10, 8, 5, 2], table, holders, ring, [9, 10], 4)
    # request 1 takes page 7 for tokens 8 and 9; request 2 needs none; for request 3 the ring is empty; 4 has tokens
    assert got["new_lens"].tolist() == [10, 10, 8, 0, 3] and got["free_range"].tolist() == [10, 10]
    assert got["table"].tolist() == [[5, 3, 0, -1], [5, 3, 7, -1], [5, 3, -1, -1], [-1] * 4, [1, -1, -1, -1]]
    assert got["holders"].tolist() == [1, 1, 0, 3, 0, 3, 0, 1]
    assert got["copies"].tolist() == [[-1, 0, -1, -1, -1], [-1, 7, -1, -1, -1], [0, 2, 0, 0, 0]]


def test_release_hand_worked():
    # pages of 4; requests 0 and 1 share pages 5 and 3; 1 has page 7 of its own; 2 shares page 5 with 2 tokens in it
    table = np.array([[5, 3, -1], [5, 3, 7], [5, -1, -1]], np.int32)
    holders = np.array([0, 0, 0, 2, 0, 3, 0, 1], np.int32)
    ring = np.array([0, 1, 2, 4, 6, 9, 9, 9], np.int32)
    got = SO.pages_held([8, 10, 2], [9, 0, 3], table, ring, [0, 5], 4, 4, holders)
    # 0 grows into page 0, 1 ends: 7 is free, 5 and 3 go on; 2 may not write into page 5
    assert got["new_lens"].tolist() == [9, 0, 2] and got["slots"].tolist() == [0, -1, -1, -1]
    assert got["table"][0].tolist() == [5, 3, 0] and got["holders"].tolist() == [1, 0, 0, 1, 0, 2, 0, 0]
    assert got["ring"].tolist() == [0, 1, 2, 4, 6, 7, 9, 9] and got["free_range"].tolist() == [1, 6]
    # the last one that lets go gives the page back, in the order of the requests
    got = SO.pages_held([8, 10, 2], [0, 0, 0], table, ring, [0, 5], 4, 0, holders)
    assert got["ring"].tolist() == [0, 1, 2, 4, 6, 3, 7, 5] and got["holders"].sum() == 0


def test_pages_without_sharing_are_those_of_the_other_call():
    rng = np.random.default_rng(3)
    for _ in range(30):
        B, P, width = 6, 4, 5
        lens, target = rng.integers(0, 21, B), rng.integers(0, 24, B)
        have = -(-lens // P)
        ids = rng.permutation(int(have.sum()) + 8)
        table, holders = np.full((B, width), -1, np.int32), np.zeros(len(ids), np.int32)
        at = 0
        for b in range(B):
            table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        holders[ids[:at]] = 1
        ring = np.full(len(ids), 99, np.int32)
        ring[:8] = ids[at:]
        one = KO.pages(lens, target, table, ring, [0, 8], P, 60)
        two = SO.pages_held(lens, target, table, ring, [0, 8], P, 60, holders)
        for name in one:
            assert np.array_equal(one[name], two[name]), name


def test_compact_hand_worked():
    holders = np.array([0, 2, 0, 1, 0, 1, 3], np.int32)  # four in use: 5 and 6 move to 0 and 2
    got = SO.compact([8, 3, 0], np.array([[1, 6, 4], [5, 6, 6], [6, 6, 6]], np.int32), holders, [11, 14], 4)
    assert got["copies"].tolist() == [[5, 6, -1], [0, 2, -1], [4, 4, 0]]
    assert got["holders"].tolist() == [1, 2, 3, 1, 0, 0, 0]
    assert got["table"].tolist() == [[1, 2, 4], [0, 6, 6], [6, 6, 6]]
    assert got["ring"].tolist() == [-1, -1, -1, -1, 4, 5, 6] and got["free_range"].tolist() == [11, 14]


def test_norm_hand_worked():
    got = SO.norm(np.array([[[3.0, 4.0, 0.0, 0.0]]]), np.array([1.0, 0.5, 1.0, 1.0]), 0.0, False)
    assert np.allclose(got, [[[1.2, 0.8, 0, 0]]])  # the root of 25 / 4 is 2.5
    got = SO.norm(np.array([[[3.0, 4.0, 0.0, 0.0]]]), np.array([0.0, -0.5, 0.0, 0.0]), 0.0, True)
    assert np.allclose(got, [[[1.2, 0.8, 0, 0]]])


@pytest.mark.parametrize("paired", [False, True])
def test_size_of_a_turn(paired):
    rng = np.random.default_rng(5)
    y, angle = rng.normal(size=(4, 2, 12)), rng.uniform(-3, 3, (9, 4))
    pos = rng.integers(0, 9, (1, 4))
    args = (pos, np.cos(angle), np.sin(angle), (4,), False, paired)
    size = SO.turned_size(y, *args)
    assert (size >= np.abs(KO.rotate(y, *args)) - 1e-12).all() and np.array_equal(size[..., 8:], np.abs(y[..., 8:]))
    pair = np.hypot(y[..., 0], y[..., 1 if paired else 4])
    assert (size[..., 0] <= np.sqrt(2) * pair + 1e-12).all()


def test_tokens_of_a_shared_prefix():
    table, prefix = np.array([[8, 9, 4], [7, -1, -1]]), np.array([[1, 2]])
    got = SO.token_rows(table, [5, 1], 2, [(0, 3), None], prefix)
    assert got.tolist() == [[2, 3, 4, 19, 8], [14, -1, -1, -1, -1]]
