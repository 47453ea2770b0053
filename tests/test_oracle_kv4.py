"""Pins of the 4-bit cache's oracle: hand-computed codes, the row order as a
bijection, rounding against torch, attention against torch in fp64, eviction
on hand-built weights."""
import numpy as np
import pytest
import torch

from oracle import kv4


def test_bf16_rounding_equals_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.integers(-40, 38, 4000), [0.0, 1e-41, 3e-40, 9.2e-41]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).to(torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(kv4.bf16(x), want)


def test_hand_computed_group():
    x = np.zeros((1, 64))
    x[0, :6] = [7, -7, 3.5, 2.5, 0.49, -1.5]       # amax 7: s = 1
    codes, s = kv4.quantise(x)
    assert s.tolist() == [[1.0, 0.0]]
    assert codes[0, :7].tolist() == [15, 1, 12, 10, 8, 6, 8]   # 3.5 -> 4, 2.5 -> 2, -1.5 -> -2
    assert (codes[0, 32:] == 8).all()
    x[0, 40] = np.inf
    codes, s = kv4.quantise(x)
    assert s[0, 0] == 1.0 and np.isnan(s[0, 1])
    assert np.isnan(kv4.values(codes, s)[0, 32:]).all() and not np.isnan(kv4.values(codes, s)[0, :32]).any()


@pytest.mark.parametrize("D", [64, 128])
def test_quantisation_error_is_within_half_a_step(D):
    x = torch.randn((50, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).double().numpy()
    codes, s = kv4.quantise(x)
    assert codes.min() >= 1 and codes.max() <= 15
    # 7 s is within 2^-8 of the largest magnitude: that element alone may be clipped by the scale's rounding
    assert (np.abs(kv4.values(codes, s) - x) <= np.repeat(s, 32, -1) * 0.5 * (1 + 2.0 ** -4)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", ["k", "v"])
def test_row_order_is_a_bijection(D, name):
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 16, (2, 8, D)).astype(np.uint8)
    rows = kv4.pack(codes, name, np.arange(8))
    assert np.array_equal(kv4.unpack(rows, name), codes)
    one = np.full((4, D), 8, np.uint8)
    one[:, 37] = 3
    rows = kv4.pack(one, name, np.arange(4))
    word = (5 // 8 * (D // 32) + 1) * 4 + 5 // 2 if name == "k" else (5 // 4 * (D // 32) + 1) * 2 + 1 // 2
    for slot in range(4):
        at = word ^ (32 if name == "v" and D == 128 and slot & 2 else 0)
        want = np.full(D // 2, 0x88, np.uint8)
        want[at] = 0x38
        assert np.array_equal(rows[slot], want)


def test_forward_equals_torch_attention():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((2, 4, 3, 64), (2, 2, 9, 64), (2, 2, 9, 64)))
    lens = [9, 5]
    o, lse, w, _, _ = kv4.forward(q.numpy(), k.numpy(), v.numpy(), lens)
    for b, n in enumerate(lens):
        mask = torch.arange(n)[None, :] <= torch.arange(3)[:, None] + n - 3
        kk, vv = (x[b, :, :n].repeat_interleave(2, 0) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q[b], kk, vv, attn_mask=mask)
        assert np.abs(o[b] - want.numpy()).max() < 1e-12
        s = (q[b] @ kk.transpose(1, 2) / 8).masked_fill(~mask, -np.inf)
        assert np.abs(lse[b] - torch.logsumexp(s, -1).numpy()).max() < 1e-12
        assert np.abs(w[b, :, :n] - torch.softmax(s, -1).sum(1).reshape(2, 2, n).sum(1).numpy()).max() < 1e-12
        assert (w[b, :, n:] == 0).all()
    assert np.abs(w.sum(-1) - 6).max() < 1e-12          # 2 heads x 3 rows, each of probability 1


def test_forward_of_empty_rows_and_sinks():
    z = np.zeros((1, 1, 2, 64))
    o, lse, w, _, _ = kv4.forward(z, np.ones((1, 1, 16, 64)), np.ones((1, 1, 16, 64)), [0])
    assert (o == 0).all() and np.isneginf(lse).all() and (w == 0).all()
    o, lse, _, _, _ = kv4.forward(z, np.ones((1, 1, 16, 64)), np.ones((1, 1, 16, 64)), [1], sinks=np.zeros(3))
    assert lse[0, 0, 0] == pytest.approx(np.log(3)) and (o[0, 0, 0] == 0).all()   # token 0 of 2 sees nothing
    assert lse[0, 0, 1] == pytest.approx(np.log(4)) and np.allclose(o[0, 0, 1], 0.25)


def test_evict_by_hand():
    w = np.array([[[5.0, 1.0, np.nan, 1.0, 0.0, 1.0, 7.0, 0.0]]])
    idx, n = kv4.evict(w, None, [7], 4)
    assert idx.tolist() == [[[0, 1, 2, 6]]] and n.tolist() == [4]      # ties at 1.0: the lowest slot
    idx, _ = kv4.evict(w, None, [7], 4, recent=3)
    assert idx.tolist() == [[[2, 4, 5, 6]]]
    idx, _ = kv4.evict(w, None, [7], 4, in_place=True)
    assert idx.tolist() == [[[0, 1, 2, 6]]]
    idx, n = kv4.evict(w, None, [3], 4)
    assert idx.tolist() == [[[0, 1, 2, -1]]] and n.tolist() == [3]
    pos = np.array([[[0, 9, 2, 3, 4, 5, 6, 7]]])
    idx, _ = kv4.evict(w, pos, [7], 3, recent=1, seen=[10], in_place=True)
    assert idx.tolist() == [[[6, 1, 2]]]                                # slot 0 freed for slot 6
