"""Pins of the paged key-value cache's restatement: hand-worked values, invariants, and the gradient of the rotation."""
import numpy as np
import pytest

from oracle import kv_oracle as KO


def test_pages_hand_worked():
    # pages of 4 tokens; the ring holds free pages 7, 5, 2 from counter 6 on (6 mod 8 = 6, 7, 0)
    table = np.array([[0, 1, -1], [3, -1, -1], [4, 6, -1]], np.int32)
    ring = np.array([2, 9, 9, 9, 9, 9, 7, 5], np.int32)
    got = KO.pages([5, 4, 8], [9, 5, 3], table, ring, [6, 9], 4, 6)
    assert got["table"].tolist() == [[0, 1, 7], [3, 5, -1], [4, 6, -1]]
    assert got["starts"].tolist() == [0, 4, 5, 5] and got["new_lens"].tolist() == [9, 5, 3]
    assert got["slots"].tolist() == [1 * 4 + 1, 1 * 4 + 2, 1 * 4 + 3, 7 * 4, 5 * 4, -1]
    assert got["positions"].tolist() == [5, 6, 7, 8, 4, 0]
    assert got["free_range"].tolist() == [8, 10] and got["ring"][9 % 8] == 6


def test_pages_short_pool_hand_worked():
    table, ring = np.full((3, 2), -1, np.int32), np.array([1, 0, 2], np.int32)
    got = KO.pages([0, 0, 0], [4, 8, 4], table, ring, [0, 2], 4, 16)
    # the second asks for pages 2 and 3 of two; the third then asks for the fourth
    assert got["new_lens"].tolist() == [4, 0, 0] and got["free_range"].tolist() == [1, 2]
    assert got["slots"].tolist() == [4, 5, 6, 7] + [-1] * 12


@pytest.mark.parametrize("sections,cycled,axes", [
    ((2, 1, 1), False, [0, 0, 1, 2]), ((2, 1, 1), True, [0, 1, 2, 0]), ((1, 0, 3), True, [0, 2, 2, 2]), ((3,), True, [0, 0, 0]),
])
def test_axes_hand_worked(sections, cycled, axes):
    assert KO.axis_of(sections, cycled) == axes


@pytest.mark.parametrize("paired", [False, True])
def test_rotation_keeps_lengths_and_its_gradient_is_the_turn_back(paired):
    rng = np.random.default_rng(1)
    x, g = rng.normal(size=(3, 2, 12)), rng.normal(size=(3, 2, 12))
    angle = rng.uniform(-3, 3, (7, 4))
    pos = rng.integers(0, 7, (2, 3))
    args = (pos, np.cos(angle), np.sin(angle), (1, 3), True, paired)
    y = KO.rotate(x, *args)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 8:], x[..., 8:])
    back = KO.rotate(g, pos, np.cos(angle), -np.sin(angle), (1, 3), True, paired)
    e = rng.normal(size=x.shape)
    step = (KO.rotate(x + 1e-6 * e, *args) - KO.rotate(x - 1e-6 * e, *args)) / 2e-6
    assert np.isclose((g * step).sum(), (back * e).sum(), rtol=1e-7)


def test_rtn8_hand_worked():
    codes, d = KO.rtn8(np.array([[127.0, -127.0, 0.5, 1.5, 2.5], [0, 0, 0, 0, 0], [np.inf, 1, 2, 3, 4]]))
    assert codes.tolist() == [[127, -127, 0, 2, 2], [0] * 5, [0] * 5]
    assert d[0] == 1.0 and d[1] == 0.0 and np.isnan(d[2])


def test_attention_of_one_and_two_tokens():
    q = np.array([[[1.0, 0.0]]])
    k = np.array([[[[0.0, 3.0]], [[np.log(3.0), 5.0]]]])  # one page of two tokens, one head
    v = np.array([[[[2.0, -2.0]], [[6.0, 10.0]]]])
    one, _, _ = KO.attention(q, k, v, np.array([[0]]), [1], [0, 1], 1.0)
    two, spread, _ = KO.attention(q, k, v, np.array([[0]]), [2], [0, 1], 1.0)
    last, _, _ = KO.attention(q, k, v, np.array([[0]]), [2], [0, 1], 1.0, window=1)
    assert np.allclose(one, [[[2, -2]]]) and np.allclose(two, [[[5, 7]]]) and np.allclose(spread, [[[5, 8]]])
    assert np.allclose(last, [[[6, 10]]])


def test_attention_rows_before_the_first_token_are_zeros():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 2, 4)), rng.normal(size=(2, 4, 1, 4)), rng.normal(size=(2, 4, 1, 4))
    out, _, _ = KO.attention(q, k, v, np.array([[1]]), [2], [0, 3], 0.5)
    assert (out[0] == 0).all() and np.allclose(out[1], v[1, 0, 0])


def test_floor_of_format_8_hand_worked():
    q = np.array([[[1.0, 0.0]], [[1.0, 0.0]]])
    k = np.array([[[[0.0, 3.0]], [[np.log(3.0), 5.0]]]])
    codes, d = np.array([[[[2.0, -2.0]], [[6.0, 10.0]]]]), np.array([[[8.0], [4.0]]])
    # weights 1, and 1/4 and 3/4: products 8, and 2 and 3
    got = KO.attention8_floor(q, k, codes, d, np.array([[0]]), [2], [0, 2], 1.0)
    assert np.allclose(got * 2.0 ** 32, [[[16, 16]], [[24, 36]]])
    last = KO.attention8_floor(q[1:], k, codes, d, np.array([[0]]), [2], [0, 1], 1.0, window=1)
    assert np.allclose(last * 2.0 ** 32, [[[24, 40]]])
