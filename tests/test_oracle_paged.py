"""Pins of the paged cache's oracle: hand-worked tables, bounds that bound,
selections worked out by hand, attention against torch's softmax."""
import numpy as np
import torch

from oracle import paged


def test_resize_by_hand():
    table = np.array([[0, 1, 2, -1], [3, -1, -1, -1], [4, 5, -1, -1]], dtype=np.int32)
    free = np.array([-1] * 6 + [6, 7], dtype=np.int32)
    # sequence 0 ends (pages 0, 1, 2 go back to places 3, 4, 5); 1 grows by two pages, 2 by none
    lens, used, slots = paged.resize(table, free, 6, [40, 16, 20], [0, 40, 23], 16, 24)
    assert lens == [0, 40, 23] and used == 5
    assert free.tolist() == [-1, -1, -1, 0, 1, 2, 6, 7]
    assert table.tolist() == [[0, 1, 2, -1], [3, 0, 1, -1], [4, 5, -1, -1]]
    assert slots[0].tolist() == [-1] * 24
    assert slots[1].tolist() == list(range(0, 16)) + list(range(16, 24))
    assert slots[2].tolist() == [5 * 16 + 4, 5 * 16 + 5, 5 * 16 + 6] + [-1] * 21


def test_resize_keeps_its_order_when_pages_run_out():
    table = np.full((4, 4), -1, dtype=np.int32)
    free = np.arange(3, dtype=np.int32)
    lens, used, slots = paged.resize(table, free, 0, [0, 0, 0, 0], [16, 48, 16, 0], 16, 48)
    # the second does not get its three pages, and the third, which would get its one, does not pass it
    assert lens == [16, 0, 0, 0] and used == 1 and (slots[1:] == -1).all()


def test_resize_refuses_lengths_and_a_stack_that_cannot_be():
    table, free = np.zeros((2, 2), dtype=np.int32), np.arange(4, dtype=np.int32)
    lens, used, _ = paged.resize(table, free, 1, [0, 40], [33, 0], 16, 64)
    assert lens == [0, 40] and used == 1
    lens, used, _ = paged.resize(table, free, 1, [32, 0], [0, 1], 16, 64)
    assert lens == [32, 0] and used == 1 and free.tolist() == [0, 1, 2, 3]


def test_bounds_bound_and_are_bf16():
    rng = np.random.default_rng(0)
    for scale in (1e-30, 1e-3, 1.0, 1e6, 1e28):
        k = torch.from_numpy(rng.standard_normal((16, 64)) * scale).to(torch.bfloat16).double().numpy()
        b = paged.bounds(k)
        assert (b[0] >= k.max(0)).all() and (b[1] <= k.min(0)).all()
        assert np.array_equal(torch.from_numpy(b).to(torch.bfloat16).double().numpy(), b)
        unit = 2.0 ** max(np.floor(np.log2(np.abs(k).max())) - 7, -100)
        assert (b[0] - k.max(0) < unit).all() and np.abs(b / unit).max() <= 256
        q = rng.standard_normal((3, 64))
        qc = np.rint(q / 2.0 ** (np.floor(np.log2(np.abs(q).max())) - 6))
        assert paged.scores(q, b[None])[0] >= (k @ qc.T).max()


def test_bounds_of_keys_that_are_no_numbers():
    k = np.ones((3, 64))
    for x in (np.nan, np.inf, -np.inf, 2.0 ** 100):
        k[1, 5] = x
        assert np.isinf(paged.bounds(k)).all()
        assert paged.scores(np.ones((1, 64)), paged.bounds(k)[None])[0] == np.inf
    assert not paged.bounds(np.zeros((2, 64))).any()


def test_selection_by_hand():
    b = np.zeros((6, 2, 64))
    b[:, 0, 0] = [1, 5, 3, 5, 2, 0]
    q = np.zeros((2, 64))
    q[0, 0] = 1.0
    assert paged.select(q, b, 3, 1, 1).tolist() == [0, 1, 5]          # 1 and 3 tie: the lower one
    assert paged.select(q, b, 4, 1, 1).tolist() == [0, 1, 3, 5]
    assert paged.select(q, b, 2, 0, 0).tolist() == [1, 3]
    assert paged.select(-q, b, 2, 0, 0).tolist() == [0, 1]            # all score 0: max(-hi, -lo) with lo = 0
    assert paged.select(q, b, 8, 1, 1).tolist() == [0, 1, 2, 3, 4, 5, -1, -1]
    assert paged.select(q, b[:0], 2, 1, 1).tolist() == [-1, -1]


def test_first_key():
    assert [paged.first_key(p, left=3) for p in (0, 2, 3, 9)] == [0, 0, 0, 6]
    assert [paged.first_key(p, chunk=4) for p in (0, 3, 4, 9)] == [0, 0, 4, 8]
    assert paged.first_key(7) == 0 and paged.first_key(7, left=-1) == 0


def test_attention_against_softmax():
    rng = np.random.default_rng(1)
    q, k, v, z = rng.standard_normal(64), rng.standard_normal((9, 64)), rng.standard_normal((9, 64)), rng.standard_normal(2)
    o, lse, mass, _ = paged.attend(q, k, v, 0.125)
    p = torch.softmax(torch.from_numpy(k @ q * 0.125), 0).numpy()
    assert np.allclose(o, p @ v) and np.isclose(lse, np.log(np.exp(k @ q * 0.125).sum())) and (mass >= np.abs(o)).all()
    o, lse, _, _ = paged.attend(q, k, v, 0.125, cap=2.0, sinks=z)
    s = 2 * np.tanh(k @ q * 0.0625)
    p = torch.softmax(torch.from_numpy(np.concatenate((s, z))), 0).numpy()[:9]
    assert np.allclose(o, p @ v)
    assert paged.attend(q, k[:0], v[:0], 0.125)[1] == -np.inf
    assert np.isclose(paged.attend(q, k[:0], v[:0], 0.125, sinks=z)[1], np.log(np.exp(z).sum()))
