"""Pins of the attention oracle: a worked table, closed forms of the softmax,
and the paged form against the plain one."""

import math

import numpy as np
import pytest

import oracle


def test_tables_worked_example():
    # pages of 16: request 0 has 15 tokens in block 7 and gets 2 (one new
    # block), request 1 has none and gets 17 (two), request 2 idles
    table = [[7, -1, -1], [-1, -1, -1], [3, -1, -1]]
    t, lens, starts, slots, taken = oracle.kv_tables([15, 0, 16], [2, 17, 0], [9, 4, 5, 6], table, 16, 20)
    assert t.tolist() == [[7, 9, -1], [4, 5, -1], [3, -1, -1]]
    assert lens.tolist() == [17, 17, 16] and starts.tolist() == [0, 2, 19, 19] and taken == 3
    assert slots.tolist() == [7 * 16 + 15, 9 * 16] + [4 * 16 + i for i in range(16)] + [5 * 16, -1]


def test_tables_run_out_of_blocks_and_of_width():
    t, lens, starts, slots, taken = oracle.kv_tables([0, 30], [20, 5], [8], [[-1, -1], [2, 3]], 16, 25)
    assert t.tolist() == [[8, -1], [2, 3]] and taken == 2
    assert lens.tolist() == [20, 32]
    assert slots.tolist() == [128 + i for i in range(16)] + [-1] * 4 + [3 * 16 + 14, 3 * 16 + 15, -1, -1, -1]


def test_attend_closed_forms():
    v = np.array([[1.0, 2.0], [3.0, -2.0], [5.0, 6.0]])
    # equal scores: the mean; one key: its value; log weights: their ratio
    assert np.allclose(oracle.attend([0.0, 0.0], np.ones((3, 2)), v, 1.0), v.mean(axis=0), rtol=1e-15)
    assert oracle.attend([1.0, 2.0], np.ones((1, 2)), v[:1], 0.3).tolist() == v[0].tolist()
    k = np.array([[0.0, 0.0], [math.log(2), 0.0], [math.log(5), 0.0]])
    assert np.allclose(oracle.attend([1.0, 0.0], k, v, 1.0), (v[0] + 2 * v[1] + 5 * v[2]) / 8, rtol=1e-15)


def test_attend_rows_without_weight_are_zero():
    v = np.ones((2, 4))
    assert not oracle.attend(np.ones(4), np.zeros((0, 4)), np.zeros((0, 4)), 1.0).any()
    assert not oracle.attend(np.ones(4), np.full((2, 4), -np.inf), v, 1.0).any()
    one = np.vstack([np.full(4, -np.inf), np.zeros(4)])
    assert oracle.attend(np.ones(4), one, np.vstack([v[:1] * 7, v[:1]]), 1.0).tolist() == [1.0] * 4
    assert np.isnan(oracle.attend(np.ones(4), np.full((2, 4), np.nan), v, 1.0)).all()


@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (3, 3), (6, 1)])
def test_paged_equals_cross_on_one_query(heads, kv_heads):
    rng = np.random.default_rng(heads)
    page, dim, lens = 16, 8, [0, 5, 33]
    cache = rng.standard_normal((2, 9, kv_heads, page, dim))
    table = np.array([[-1, -1, -1], [4, -1, -1], [8, 0, 5]])
    q = rng.standard_normal((3, heads, dim))
    k = np.zeros((2, 3, 48, kv_heads, dim))
    for b in range(3):
        for t in range(lens[b]):
            k[:, b, t] = cache[:, table[b, t // page], :, t % page]
    paged = oracle.paged_attention(q, cache[0], cache[1], table, lens, 40, 0.35)
    cross = oracle.cross_attention(q[:, None], k[0], k[1], lens, 0.35)[:, 0]
    assert np.array_equal(paged, cross)
    # a head reads its own group's keys: heads of one group, same query
    q[:, :] = q[:, :1]
    same = oracle.paged_attention(q, cache[0], cache[1], table, lens, 40, 0.35)
    group = heads // kv_heads
    for h in range(heads):
        assert np.array_equal(same[:, h], same[:, h // group * group])


def test_paged_leaves_out_missing_blocks():
    rng = np.random.default_rng(5)
    cache = rng.standard_normal((2, 3, 1, 16, 4))
    q = rng.standard_normal((1, 1, 4))
    out = oracle.paged_attention(q, cache[0], cache[1], [[1, -1, 7, 2]], [64], 64, 0.5)
    k, v = (np.concatenate([c[1, 0], c[2, 0]]) for c in cache)
    assert np.array_equal(out[0, 0], oracle.attend(q[0, 0], k, v, 0.5))
